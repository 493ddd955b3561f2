// What the attention kernels share: tensor-memory moves of 32 columns, products whose first operand lies
// in tensor memory, packed fp32 arithmetic, loads of a tile and the zeroing of rows past a sequence.
#pragma once

#include "tc_ptx.cuh"

namespace lora {

// Tensor map of a [rows, cols] bf16 matrix with ld elements from row to row, in boxes of box_rows x 64 (attention.cu).
bool attn_map(CUtensorMap* map, const void* ptr, int64_t cols, int64_t rows, int64_t ld, int box_rows = kAttnTile);

namespace attn {

using namespace tc;

constexpr int kRows = kAttnTile;
// The forward pass and k_attn_dq have 384 threads: eight warps that compute, then a warpgroup that loads and issues and
// leaves them its registers; k_attn_dkv 640, sixteen of them.
template <int THREADS, int LAUNCH, int ISSUE, int COMPUTE>
struct Split {
  static constexpr int kThreads = THREADS, kLaunch = LAUNCH, kIssue = ISSUE, kCompute = COMPUTE;   // registers per thread
  static_assert(128 * ISSUE + (THREADS - 128) * COMPUTE <= THREADS * LAUNCH, "setmaxnreg draws on the block's own registers");
  __device__ static void issue() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(ISSUE)); }
  __device__ static void compute() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(COMPUTE)); }
};
using SplitFwd = Split<384, 168, 56, 224>;
using SplitBwd = Split<640, 96, 64, 104>;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// ---- packed fp32 pairs ----
using f2 = uint64_t;
__device__ __forceinline__ f2 mk2(float a, float b) {
  f2 v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(a), "f"(b));
  return v;
}
__device__ __forceinline__ float2 un2(f2 v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
  f2 d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
  f2 d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
  f2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ float exp2_(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// A value of shared memory, read where this stands: what is computed from it is not moved ahead of the
// arrivals before it.
__device__ __forceinline__ float read_here(const float* p) {
  float v;
  asm volatile("ld.volatile.shared.f32 %0, [%1];" : "=f"(v) : "r"(smem_u32(p)) : "memory");
  return v;
}

// ---- tensor memory, 32 columns of this thread's lane ----
__device__ __forceinline__ void tmem_ld32_nw(uint32_t taddr, uint32_t* r) {   // valid after tmem_wait_ld_n
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
      "%12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, "
      "%30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
      "%12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, "
      "%30, %31, %32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
      "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]),
      "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
      "%12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
// 32 columns of 16 lanes, spread over the warp: register 4 b + 2 i + j is lane (thread / 4) + 8 i, column
// 8 b + 2 (thread % 4) + j.
__device__ __forceinline__ void tmem_ld16x32_nw(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
      "%12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
// 16 columns of 16 lanes: register 2 b + i is lane (thread / 4) + 8 i, column 4 b + thread % 4.
__device__ __forceinline__ void tmem_st16x16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x128b.x4.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// The same as tmem_wait_ld for a run of registers.
template <int N>
__device__ __forceinline__ void tmem_wait_ld_n(uint32_t* r) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+r"(r[i])::"memory");
}

// ---- products. The whole warp runs the issuing loop, so that operands stay in uniform registers, and its
// elected lane (`one` nonzero) issues: a single lane's branch moves every operand there first, and then eight
// instructions of 64 cycles take 720 to 1040 to issue.
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t one;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}\n" : "=r"(one));
  return one;
}
// D (+)= A B^T, both in shared memory
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t acc, uint32_t one) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(id), "r"(acc), "r"(one));
}
// with A [128, 16] in tensor memory: lane = row, two bf16 of k per 32-bit column
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t id, uint32_t acc, uint32_t one) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(id), "r"(acc), "r"(one));
}
__device__ __forceinline__ void commit(uint64_t* bar, uint32_t one) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}\n" ::"r"(smem_u32(bar)),
      "r"(one)
      : "memory");
}
// A value that is the same in all lanes, known as such to the compiler.
__device__ __forceinline__ int uniform(int v) { return __shfl_sync(0xffffffffu, v, 0); }

__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}
// A flag between two kernels that run side by side: what the setting thread has seen is seen by a thread that has
// found the flag set.
__device__ __forceinline__ void flag_set(int32_t* flag) {
  asm volatile("st.release.gpu.global.b32 [%0], %1;" ::"l"(flag), "r"(1) : "memory");
}
// false (and an error bit) if the flag is not set within `limit` cycles
__device__ __forceinline__ bool flag_wait(const int32_t* flag, uint32_t bit, uint32_t* err, unsigned long long limit) {
  const unsigned long long t0 = clock64();
  for (;;) {
    int32_t v;
    asm volatile("ld.acquire.gpu.global.b32 %0, [%1];" : "=r"(v) : "l"(flag) : "memory");
    if (v) return true;
    if (clock64() - t0 > limit) {
      atomicOr(err, bit);
      return false;
    }
  }
}
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// A tile: 128 rows of D bf16, as D / 64 boxes of 128 rows of 128 swizzled bytes.
template <int D>
struct Tile {
  static constexpr int kBoxes = D / 64;
  static constexpr int kBoxBytes = kRows * 128;
  static constexpr int kBytes = kBoxes * kBoxBytes;
  // rows x columns as they lie (k along the columns) and turned (k along the rows)
  __device__ static void load(uint8_t* dst, const CUtensorMap* map, uint64_t* bar, int col, int row) {
#pragma unroll
    for (int b = 0; b < kBoxes; ++b) tma_load_2d(dst + b * kBoxBytes, map, bar, col + 64 * b, row);
  }
  // D[128, 128] = A B^T over the tiles' D columns
  __device__ static void mma_nt(uint32_t d, uint32_t sa, uint32_t sb, uint32_t id, uint32_t one) {
#pragma unroll
    for (int b = 0; b < kBoxes; ++b) {
      const uint64_t da = smem_desc_sw128(sa + b * kBoxBytes), db = smem_desc_sw128(sb + b * kBoxBytes);
#pragma unroll
      for (int k = 0; k < 4; ++k) mma_ss(d, da + 2 * k, db + 2 * k, id, (b || k) ? 1u : 0u, one);
    }
  }
  // D[128, D] += A B over the tile's 128 rows, A in tensor memory in runs of RUN rows' columns, which start RUN
  // columns apart (a thread's fp32 values and over them its bf16 ones)
  // (rows 16 K0 .. 16 K1 - 1 of them)
  template <int RUN, int K0 = 0, int K1 = 8>
  __device__ static void mma_tn(uint32_t d, uint32_t a, uint32_t sb, uint32_t id, bool acc, uint32_t one) {
    const uint64_t db = smem_desc_sw128_mn(sb, kBoxBytes);
#pragma unroll
    for (int k = K0; k < K1; ++k)
      mma_ts(d, a + 16 * k / RUN * RUN + 16 * k % RUN / 2, db + 128 * k, id, (acc || k) ? 1u : 0u, one);
  }
  // Zeros in the rows from `rows` on, by a whole warp (the swizzle moves 16-byte pieces within a row only).
  __device__ static void zero_rows(uint8_t* tile, int rows, int lane) {
    const int n = (kRows - rows) * 8;
#pragma unroll
    for (int b = 0; b < kBoxes; ++b)
      for (int i = lane; i < n; i += 32)
        *reinterpret_cast<uint4*>(tile + b * kBoxBytes + rows * 128 + i * 16) = make_uint4(0, 0, 0, 0);
  }
};

// A kernel's attributes. A build that launches with fewer registers would wait for them forever.
template <typename Split, typename F>
cudaError_t set_up(F* kernel, int smem) {
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  cudaFuncAttributes fa;
  if (e == cudaSuccess) e = cudaFuncGetAttributes(&fa, kernel);
  if (e == cudaSuccess && fa.numRegs != Split::kLaunch) e = cudaErrorInvalidConfiguration;
  return e;
}

// What other kernels wrote, the plan's lists and the rows' statistics, is read by plain loads: the non-coherent path is
// for data that nothing writes while the kernel lives, and with programmatic launch a CTA may be there before its
// producer is done. (As the language's own load these 16 bytes cost k_attn_dq at head_dim 128 36 bytes of spills more.)
__device__ __forceinline__ int4 load_plain(const void* p) {
  int4 v;
  asm volatile("ld.global.v4.s32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p) : "memory");
  return v;
}

// One of a plan's lists. A plan of other tokens or sequences than the call's has none of its items: nothing is
// computed, and nothing outside the call's tensors is touched.
struct PlanRef {
  const int32_t* head;     // tiles of 128 rows, of 256 rows, tokens, sequences
  const AttnTile* tiles;
  int32_t list, tokens, n_seq;
  __device__ int items(int groups) const {
    const int4 v = load_plain(head);
    return uniform(v.z == tokens && v.w == n_seq ? (list ? v.y : v.x) * groups : 0);
  }
};
inline PlanRef plan_ref(const AttnArgs& a, int list) {
  return PlanRef{a.plan.count, a.plan.tiles[list], list, (int32_t)a.T, a.plan.n_seq};
}

// The work of a persistent CTA: items of the plan's list (a tile and one of its `groups` groups of heads), the
// longest first, dealt out to and fro so that every CTA's sum comes out alike. Every role of a CTA walks the
// same items; the loading warp comes to each first, so that the others find its tile in L1.
struct Items {
  const AttnTile* tiles;
  int groups, n, round, b, grid;
  __device__ Items(const PlanRef& p, int g, int cluster = 1)
      : tiles(p.tiles), groups(g), n(p.items(g)), round(0), b((int)blockIdx.x / cluster), grid((int)gridDim.x / cluster) {}
  // the next item, false if there is none
  __device__ bool take(AttnTile& t, int& group) {
    const int64_t i = (int64_t)round * grid + ((round & 1) ? grid - 1 - b : b);
    ++round;
    if (i >= n) return false;
    const int li = (int)i / groups;
    group = (int)i - li * groups;
    const int4 v = load_plain(tiles + li);
    t = AttnTile{uniform(v.x), uniform(v.y), uniform(v.z), 0};
    return true;
  }
};

// Two tiles of 128 queries that read the same keys: two heads of a group, or, where a group's heads do not pair
// up, two neighbouring tiles of one head. Tile s: head h(s), queries from qi(s) * 128, n(s) key tiles (0: there
// is no such tile).
struct Pair {
  int h0, h1, q0, q1, n0, n1, most;
  __device__ Pair(const AttnTile& t, int group, bool by_heads) {
    h0 = by_heads ? 2 * group : group;
    h1 = by_heads ? h0 + 1 : h0;
    q0 = by_heads ? t.index : 2 * t.index;
    q1 = by_heads ? q0 : q0 + 1;
    n0 = q0 + 1;
    n1 = (int64_t)q1 * kRows < t.len ? q1 + 1 : 0;
    most = n1 > n0 ? n1 : n0;
  }
  __device__ int h(int s) const { return s ? h1 : h0; }
  __device__ int qi(int s) const { return s ? q1 : q0; }
  __device__ int n(int s) const { return s ? n1 : n0; }
};

// 32 lanes' COLS columns of tensor memory, scaled by each lane's f, as bf16 rows in `stage`, the warp's own
// 32 x COLS bf16 of shared memory, in the swizzle of a bulk tensor store of that box.
template <int COLS>
__device__ __forceinline__ uint32_t piece_at(int row, int c) {   // byte of 16-byte piece c of a row
  constexpr int NC = COLS / 8;
  return row * (COLS * 2) + ((c ^ ((NC == 8 ? row : row >> 1) & (NC - 1))) << 4);
}
template <int COLS>
__device__ __forceinline__ void read_rows(uint32_t taddr, float f, uint32_t (&u)[COLS / 2]) {
  uint32_t v[COLS];
  if constexpr (COLS >= 32) {
#pragma unroll
    for (int k = 0; k < COLS / 32; ++k) tmem_ld32_nw(taddr + 32 * k, v + 32 * k);
  } else {
    tmem_ld16_nw(taddr, v);
  }
  tmem_wait_ld_n<COLS>(v);
  const f2 ff = mk2(f, f);
#pragma unroll
  for (int i = 0; i < COLS / 2; ++i) {
    const float2 e = un2(mul2(mk2(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1])), ff));
    u[i] = pack_bf16(e.x, e.y);
  }
}
template <int COLS>
__device__ __forceinline__ void stage_rows(uint8_t* stage, const uint32_t (&u)[COLS / 2], int lane) {
#pragma unroll
  for (int c = 0; c < COLS / 8; ++c)
    *reinterpret_cast<uint4*>(stage + piece_at<COLS>(lane, c)) = make_uint4(u[4 * c], u[4 * c + 1], u[4 * c + 2], u[4 * c + 3]);
}
// The staged rows, `live` of them, to `out` (row 0, first column; ld elements apart), a store covering whole runs
// of a row. (A lane's row written piece by piece, 32 rows to a store, filled the load and store queue for 3500 cycles
// per tile and held up the next item's first loads and waits for 2300 more.)
template <int COLS>
__device__ __forceinline__ void write_rows(const uint8_t* stage, __nv_bfloat16* out, int64_t ld, int live, int lane) {
  constexpr int NC = COLS / 8, RPI = 32 / NC;   // 16-byte pieces of a row, rows of a store
  __syncwarp();
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int row = i * RPI + lane / NC, c = lane % NC;
    const uint4 u = *reinterpret_cast<const uint4*>(stage + piece_at<COLS>(row, c));
    if (row < live) *reinterpret_cast<uint4*>(out + row * ld + 8 * c) = u;
  }
  __syncwarp();
}
// The same as a bulk tensor store of all 32 rows, which the warp need not wait for: 8 pairs of a read and a store
// take it 700 to 1200 cycles.
__device__ __forceinline__ void send_rows(const CUtensorMap* map, const uint8_t* stage, int col, int64_t row, int lane) {
  fence_async();
  __syncwarp();
  if (lane == 0) {
    tma_store_2d(map, stage, col, (int32_t)row);
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
  }
}
// Lane 0's bulk stores have read their stages.
__device__ __forceinline__ void rows_read(int lane) {
  if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
  __syncwarp();
}

// Bounded wait of a whole warp: the same answer in every lane. Under a bound below the default (a test's) an
// attempt that succeeds too late counts as failed. Short, since the issuing warp's loop runs through it several
// times for each tile.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, uint32_t bit, uint32_t* err,
                                          unsigned long long limit) {
  if (limit >= kWaitCycles && __all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  const unsigned long long t0 = clock64();
  do {
    if (__any_sync(0xffffffffu, clock64() - t0 > limit)) {
      atomicOr(err, bit);
      return false;
    }
  } while (!__all_sync(0xffffffffu, mbar_try_wait(bar, parity)));
  return true;
}

// Tiles whose rows behind the sequence are zeroed before the products see them: P and dS are zero there, but zero
// times another sequence's or padding's NaN is not. The copy lands on the buffer's `landed` barrier, and a warp of its
// own zeroes the rows and passes the tile on (`full`), so that the loading warp need not wait (1500 cycles a tile;
// dK and dV meet one for every query head). Both warps walk the same tiles and count each buffer's uses.
struct Partial {
  static constexpr unsigned long long kLongest = 1ull << 40;   // cycles: minutes
  uint32_t parity = 0, used = 0;   // by buffer: the next use's parity, whether there was one
  uint32_t n = 0;                  // tiles so far
  __device__ void next(int s) {
    parity ^= 1u << s;
    used |= 1u << s;
    ++n;
  }
  // the zeroing warp, which has passed `before` tiles: false where the copy does not land. Its next tile may be many
  // items away, so that its wait has no short bound of its own: the loading warp, whose waits have one, leaves 1 + the
  // tiles it asked for in `ended`, and what was asked for lands.
  template <int D>
  __device__ bool pass(uint8_t* tile, int s, int rows, uint64_t* landed, uint64_t* full, int lane, uint32_t* err,
                       const uint32_t* ended, uint32_t before) {
    const uint32_t par = parity >> s & 1u;
    const unsigned long long t0 = clock64();
    while (!__all_sync(0xffffffffu, mbar_try_wait(&landed[s], par))) {
      const uint32_t v = __shfl_sync(0xffffffffu, *static_cast<const volatile uint32_t*>(ended), 0);
      if (v != 0u || __any_sync(0xffffffffu, clock64() - t0 > kLongest)) {
        if ((v != 0u && before + 1u >= v) || !warp_wait(&landed[s], par, 1u, err, kWaitCycles)) return false;
        break;
      }
    }
    next(s);
    Tile<D>::zero_rows(tile, rows, lane);
    fence_async();
    __syncwarp();
    if (lane == 0) mbar_arrive(&full[s]);
    return true;
  }
  // the loading warp's lane 0, at its end: every copy has landed
  __device__ void drain(uint64_t* landed, int n, uint32_t* err) const {
    for (int s = 0; s < n; ++s)
      if (used >> s & 1u) mbar_wait(&landed[s], (parity >> s & 1u) ^ 1u, 1u, err);
  }
};

}  // namespace attn
}  // namespace lora
