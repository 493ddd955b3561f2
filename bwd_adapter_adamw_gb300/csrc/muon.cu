// Orthogonalised update of the adapter matrices: momentum, then a Newton-Schulz sequence
// X <- (a I + b G + c G^2) X, G = X X^T over the smaller side s (at most 64), from X = u / ||u||_F.
//
// The smaller side is the adapter's rank, so the sequence acts on the small Gram matrix G alone:
// with P = a I + b G + c G^2 (a polynomial in G, so they commute) one step maps G to P G P and
// multiplies X by P. Several steps then cost one Gram matrix, small products, and one product
// Q X = P_m .. P_1 X on the long axis. A rounding of G, relative to its largest eigenvalue, is
// amplified by about a^2 per step at the smallest ones, so after at most kStageSteps steps (five
// steps: two, then three) the Gram matrix is formed again from Q X, which brings the error down
// to that of iterating on X itself (the CPU oracle's bound in the tests).
//
// One cluster of CTAs per matrix, its long axis spread over the CTAs, u held on chip: the arenas
// are read and written once (20 bytes per element: p and m both ways, g in). The Gram matrices of
// the CTAs are added through distributed shared memory in rank order (bitwise reproducible), and
// every CTA repeats the small products.
//
// s <= 16: CUDA cores, u in fp32 (k_muon_simt). Larger s: the two long products on tensor cores
// (k_muon_tc), u as a two-term bf16 split, all four products of the terms kept.
//
// Measured: 22 layers of rank 8 (2048 + 256 columns) 15 us, a chain of passes and cluster barriers;
// 32 layers of rank 64 (4096 + 14336 columns) 365 us, 755 MB at the least, 1.00 GB moved (the tiles
// beyond those that a CTA holds go through L2): bound by the latency of a tile's steps (load,
// split, MMA, drain), one after the other, and by the small products, during which no tile moves.
#include <algorithm>
#include <atomic>

#include "tc_ptx.cuh"

namespace lora {

namespace {
using namespace tc;

constexpr int kMuonThreads = 256;
constexpr int kStageSteps = 3;

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

__device__ __forceinline__ float dsmem_ld(const float* local, uint32_t rank) {
  uint32_t remote;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(smem_u32(local)), "r"(rank));
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(remote) : "memory");
  return v;
}

__device__ __forceinline__ void cluster_sync() {
  __syncwarp();
  cluster_sync_all();
}

// The power of two that brings the cluster's largest |u| to about one when its squares could
// leave the fp32 range; one otherwise. `sh` holds a float per warp (16 at most) and the CTA's maximum.
template <int Threads>
__device__ __forceinline__ float range_scale(float mx, float* sh, int C) {
  mx = warp_max(mx);
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = mx;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < Threads / 32; ++w) mx = fmaxf(mx, sh[w]);
    sh[16] = mx;
  }
  if (C > 1) cluster_sync();
  else __syncthreads();
  mx = sh[16];
  for (int r = 0; r < C; ++r) mx = C > 1 ? fmaxf(mx, dsmem_ld(sh + 16, (uint32_t)r)) : mx;
  if (C > 1) cluster_sync();   // sh may be written again
  if (!(mx > 0.f) || !isfinite(mx) || (mx > 0x1p-30f && mx < 0x1p30f)) return 1.f;
  return exp2f((float)-min(max(ilogbf(mx), -126), 126));
}

// ---- s <= 16 on CUDA cores ----------------------------------------------------------------------
// S = 4 S4. u [columns][SP] fp32 in shared memory (SP keeps 4-way bank conflicts at most for a
// column-wise walk); columns past the cap are computed again from g and m in every pass.
template <int S4>
struct SimtCfg {
  static constexpr int S = 4 * S4;
  static constexpr int SP = S % 8 == 0 ? S + 4 : S;
  static constexpr int kBlocks = S4 * S4;                      // 4 x 4 blocks of the Gram matrix
  static constexpr int kLanes = kBlocks == 9 ? 16 : kBlocks;   // threads of one column group
  static constexpr int kGroups = kMuonThreads / kLanes;
  static constexpr int kSmallFloats = 8 * S * S + 5 * S * S + 20;
  static constexpr int kCap = (200 * 1024 - kSmallFloats * 4) / (SP * 4) / 4 * 4;
};

template <int S4>
__device__ __forceinline__ void simt_mm(float* C, const float* A, const float* B) {
  constexpr int S = 4 * S4;
  const int i = threadIdx.x / S, j = threadIdx.x % S;
  float d = 0.f;
  if (threadIdx.x < S * S) {
#pragma unroll
    for (int k = 0; k < S; ++k) d = fmaf(A[i * S + k], B[k * S + j], d);
  }
  __syncthreads();
  if (threadIdx.x < S * S) C[threadIdx.x] = d;
  __syncthreads();
}

template <int S4>
__global__ void __launch_bounds__(kMuonThreads) k_muon_simt(float* __restrict__ P, float* __restrict__ G,
                                                            float* __restrict__ M,
                                                            const __grid_constant__ MuonTab tab,
                                                            const MuonK hp,
                                                            const double* __restrict__ scale_norm,
                                                            const int32_t* __restrict__ status,
                                                            int zero_grads, int C) {
  grid_dep_sync();
  using F = SimtCfg<S4>;
  constexpr int S = F::S, SP = F::SP;
  extern __shared__ float sm[];
  float* part = sm;               // [8][S S] warps' Gram matrices; then [0] the CTA's
  float* g0 = part + 8 * S * S;   // Gram matrix
  float* qs = g0 + S * S;         // product of this stage's steps
  float* qt = qs + S * S;         // product of all steps (columns past the cap)
  float* t1 = qt + S * S;
  float* t2 = t1 + S * S;
  float* sh = t2 + S * S;
  float* u = sh + 20;             // [cap][SP]
  const int rank = C > 1 ? (int)cluster_ctarank() : 0;
  const int tid = threadIdx.x;
  for (int mi = (int)blockIdx.x / C; mi < tab.n; mi += (int)gridDim.x / C) {
    const MuonMat mt = tab.m[mi];
    if (status[mt.group] != LORA_OK) continue;
    const float c = (float)scale_norm[2 * mt.group], mu = hp.mu;
    const int64_t n4 = mt.n / 4;   // columns are shared out by fours
    const int64_t j0 = n4 * rank / C * 4, j1 = n4 * (rank + 1) / C * 4;
    const int cols = (int)(j1 - j0), held = min(cols, F::kCap);
    const int64_t sj = mt.tall ? S : 1, si = mt.tall ? 1 : mt.n;   // element (i, j): i si + j sj
    float* p = P + mt.offset + j0 * sj;
    float* g = G + mt.offset + j0 * sj;
    float* m = M + mt.offset + j0 * sj;
    auto make_u = [&](float gv, float mv) {   // mv: the new momentum
      return hp.nesterov ? fmaf(mu, mv, c * gv) : mv;
    };
    // momentum and u
    const int units = cols * S4;
    for (int e0 = tid; e0 < units; e0 += 4 * kMuonThreads) {
      float4 gv[4], mv[4];
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const int e = e0 + v * kMuonThreads;
        if (e < units) {
          // tall: four rows' entries of one column; wide: four columns' entries of one row
          const int64_t at = mt.tall ? (int64_t)e * 4 : (int64_t)(e / (cols / 4)) * si + e % (cols / 4) * 4;
          gv[v] = *reinterpret_cast<const float4*>(g + at);
          mv[v] = *reinterpret_cast<const float4*>(m + at);
        }
      }
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const int e = e0 + v * kMuonThreads;
        if (e >= units) break;
        const int i = mt.tall ? e % S4 * 4 : e / (cols / 4);
        const int j = mt.tall ? e / S4 : e % (cols / 4) * 4;
        const int64_t at = i * si + j * sj;
        float* a = &gv[v].x;
        float* b = &mv[v].x;
        float w[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          b[q] = fmaf(mu, b[q], c * a[q]);
          w[q] = make_u(a[q], b[q]);
        }
        *reinterpret_cast<float4*>(m + at) = mv[v];
        if (mt.tall) {
          if (j < held) *reinterpret_cast<float4*>(u + j * SP + i) = make_float4(w[0], w[1], w[2], w[3]);
        } else {
#pragma unroll
          for (int q = 0; q < 4; ++q)
            if (j + q < held) u[(j + q) * SP + i] = w[q];
        }
      }
    }
    if (tid < S * S) qt[tid] = tid / S == tid % S ? 1.f : 0.f;
    __syncthreads();
    // G, summed over the cluster, in g0
    auto gram = [&]() {
      // a thread adds a 4 x 4 block over its group's columns
      {
        float acc[4][4] = {};
        const int b = tid % F::kLanes, grp = tid / F::kLanes;
        const int bi = b / S4 * 4, bk = b % S4 * 4;
        if (b < F::kBlocks) {
          for (int j = grp; j < held; j += F::kGroups) {
            const float4 a = *reinterpret_cast<const float4*>(u + j * SP + bi);
            const float4 d = *reinterpret_cast<const float4*>(u + j * SP + bk);
            const float av[4] = {a.x, a.y, a.z, a.w}, dv[4] = {d.x, d.y, d.z, d.w};
#pragma unroll
            for (int y = 0; y < 4; ++y)
#pragma unroll
              for (int z = 0; z < 4; ++z) acc[y][z] = fmaf(av[y], dv[z], acc[y][z]);
          }
          for (int j = held + grp; j < cols; j += F::kGroups) {
            float av[4] = {}, dv[4] = {};
            for (int k = 0; k < S; ++k) {
              const int64_t at = k * si + j * sj;
              const float w = make_u(g[at], m[at]);
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                av[q] = fmaf(qt[(bi + q) * S + k], w, av[q]);
                dv[q] = fmaf(qt[(bk + q) * S + k], w, dv[q]);
              }
            }
#pragma unroll
            for (int y = 0; y < 4; ++y)
#pragma unroll
              for (int z = 0; z < 4; ++z) acc[y][z] = fmaf(av[y], dv[z], acc[y][z]);
          }
        }
#pragma unroll
        for (int y = 0; y < 4; ++y)
#pragma unroll
          for (int z = 0; z < 4; ++z) {
#pragma unroll
            for (int o = F::kLanes; o < 32; o *= 2) acc[y][z] += __shfl_xor_sync(0xffffffffu, acc[y][z], o);
            if (b < F::kBlocks && (tid & 31) < F::kLanes)
              part[(tid >> 5) * S * S + (bi + y) * S + bk + z] = acc[y][z];
          }
      }
      __syncthreads();
      float d = 0.f;
      if (tid < S * S) {
#pragma unroll
        for (int w = 0; w < kMuonThreads / 32; ++w) d += part[w * S * S + tid];
      }
      if (C > 1) {
        __syncthreads();
        if (tid < S * S) part[tid] = d;
        cluster_sync();
        if (tid < S * S) {
          d = 0.f;
          for (int r = 0; r < C; ++r) d += dsmem_ld(part + tid, (uint32_t)r);
        }
        cluster_sync();   // the peers have read part
      }
      if (tid < S * S) g0[tid] = d;
      __syncthreads();
    };
    for (int done = 0; done < hp.steps;) {
      const int left = hp.steps - done;
      const int now = left % kStageSteps ? left % kStageSteps : kStageSteps;
      gram();
      float inv = 1.f;
      if (done == 0) {   // X = u / ||u||, ||u||^2 = trace G
        auto trace = [&]() {
          float tr = 0.f;
#pragma unroll
          for (int i = 0; i < S; ++i) tr += g0[i * S + i];
          return tr;
        };
        float tr = trace();
        if (!(tr > 1e-18f && tr < 1e30f)) {
          // the squares may have left the fp32 range (or u is zero): scale u by a power of two that
          // brings its largest magnitude to about one, and sum again
          float mx = 0.f;
          for (int e = tid; e < cols * S; e += kMuonThreads) {
            const int j = e / S, i = e % S;
            mx = fmaxf(mx, fabsf(j < held ? u[j * SP + i] : make_u(g[i * si + j * sj], m[i * si + j * sj])));
          }
          const float pre = range_scale<kMuonThreads>(mx, sh, C);
          if (pre != 1.f) {
            for (int e = tid; e < held * S; e += kMuonThreads) u[e / S * SP + e % S] *= pre;
            if (tid < S * S) qt[tid] *= pre;
            __syncthreads();
            gram();
            tr = trace();
          }
        }
        inv = tr > 0.f ? 1.f / sqrtf(tr) : 0.f;
        __syncthreads();
        if (tid < S * S) g0[tid] *= inv * inv;
        __syncthreads();
      }
      if (tid < S * S) qs[tid] = tid / S == tid % S ? inv : 0.f;
      for (int k = 0; k < now; ++k) {
        simt_mm<S4>(t1, g0, g0);                                        // G^2
        if (tid < S * S)
          t1[tid] = hp.c * t1[tid] + hp.b * g0[tid] + (tid / S == tid % S ? hp.a : 0.f);   // P
        __syncthreads();
        simt_mm<S4>(qs, t1, qs);                                        // Q <- P Q
        if (k + 1 < now) {                                              // G <- P (G P)
          simt_mm<S4>(t2, g0, t1);
          simt_mm<S4>(g0, t1, t2);
        }
      }
      done += now;
      if (cols > held) simt_mm<S4>(qt, qs, qt);
      // X <- Q X on the held columns
      for (int j = tid; j < held; j += kMuonThreads) {
        float x[S];
#pragma unroll
        for (int i = 0; i < S; i += 4) *reinterpret_cast<float4*>(x + i) = *reinterpret_cast<const float4*>(u + j * SP + i);
#pragma unroll 1   // (all of Q at once does not fit the registers)
        for (int i = 0; i < S; i += 4) {
          float y[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            y[q] = 0.f;
#pragma unroll
            for (int k = 0; k < S; k += 4) {
              const float4 w = *reinterpret_cast<const float4*>(qs + (i + q) * S + k);
              y[q] = fmaf(w.x, x[k], fmaf(w.y, x[k + 1], fmaf(w.z, x[k + 2], fmaf(w.w, x[k + 3], y[q]))));
            }
          }
          *reinterpret_cast<float4*>(u + j * SP + i) = make_float4(y[0], y[1], y[2], y[3]);
        }
      }
      __syncthreads();
    }
    const float step = mt.step, dec = mt.lr * mt.decay;
    const int hunits = held * S4;
    for (int e = tid; e < hunits; e += kMuonThreads) {
      const int i = mt.tall ? e % S4 * 4 : e / (held / 4);
      const int j = mt.tall ? e / S4 : e % (held / 4) * 4;
      const int64_t at = i * si + j * sj;
      float4 pv = *reinterpret_cast<const float4*>(p + at);
      float* a = &pv.x;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float x = mt.tall ? u[j * SP + i + q] : u[(j + q) * SP + i];
        a[q] = a[q] - step * x - dec * a[q];
      }
      *reinterpret_cast<float4*>(p + at) = pv;
      if (zero_grads) *reinterpret_cast<float4*>(g + at) = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    // the other columns: (all steps) u
    for (int e = tid; e < (cols - held) * S4; e += kMuonThreads) {
      const int j = held + e / S4, i = e % S4 * 4;
      float x[4] = {};
      for (int k = 0; k < S; ++k) {
        const float w = make_u(g[k * si + j * sj], m[k * si + j * sj]);
#pragma unroll
        for (int q = 0; q < 4; ++q) x[q] = fmaf(qt[(i + q) * S + k], w, x[q]);
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int64_t at = (i + q) * si + j * sj;
        p[at] = p[at] - step * x[q] - dec * p[at];
      }
    }
    if (zero_grads && cols > held) {   // read by every thread above
      __syncthreads();
      for (int e = tid; e < (cols - held) * S; e += kMuonThreads)
        g[(e % S) * si + (held + e / S) * sj] = 0.f;
    }
    __syncthreads();   // u, part and sh are free for the next matrix
  }
}

// ---- s <= 64 on tensor cores --------------------------------------------------------------------
// A tile is 128 columns of u as two arrays of 128 rows x 64 bf16 (hi, lo; rows past s are zero),
// 128-byte rows in the 128-byte swizzle. One layout serves both products:
//   Gram   [hi; lo] [hi; lo]^T: M = N = 128 over the columns, MN-major operands whose second
//          64-row block is the lo array: the four products of the split are the quadrants of D
//   Q X    rows are K-major A operands, B = [Q_hi; Q_lo] (N = 128): hi and lo into one
//          accumulator, the two halves of its columns added in the epilogue
constexpr int kTcThreads = 512;
// A CTA has room for six tiles. Up to five are held (the sixth's room serves the small matrices). Of
// more, three are held and the others go through `spill` and the three rooms left, two of them on
// their way while one is in use.
constexpr int kTcSlots = 6;
constexpr int kTcHeld = 3;
constexpr int kTcScr = kTcSlots - kTcHeld;
constexpr int kTcTileBytes = 32 * 1024;
constexpr int kTcAhead = 4;                    // tiles prefetched to L2 ahead of the one in use
constexpr int kTcSmem = kTcSlots * kTcTileBytes + 2 * 16 * 1024 + 256 + 1024;
static_assert(kTcSmem <= 227 * 1024, "shared memory per CTA");

__device__ __forceinline__ bool mbar_test(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Eight values as 16 bytes of hi and of lo at chunk c (8 values) of row `row` of a 64-wide split
__device__ __forceinline__ void put_split8(uint8_t* hi, uint8_t* lo, int row, int c, const float* v) {
  uint32_t h[4], l[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    h[q] = pack_bf16(v[2 * q], v[2 * q + 1]);
    l[q] = pack_bf16(v[2 * q] - __uint_as_float(h[q] << 16), v[2 * q + 1] - __uint_as_float(h[q] & 0xFFFF0000u));
  }
  const int at = row * 128 + ((c ^ (row & 7)) << 4);
  *reinterpret_cast<uint4*>(hi + at) = make_uint4(h[0], h[1], h[2], h[3]);
  *reinterpret_cast<uint4*>(lo + at) = make_uint4(l[0], l[1], l[2], l[3]);
}

// The same for the four values from column col of the split
__device__ __forceinline__ void put_split4(uint8_t* hi, uint8_t* lo, int row, int col, const float* v) {
  uint32_t h[2], l[2];
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    h[q] = pack_bf16(v[2 * q], v[2 * q + 1]);
    l[q] = pack_bf16(v[2 * q] - __uint_as_float(h[q] << 16), v[2 * q + 1] - __uint_as_float(h[q] & 0xFFFF0000u));
  }
  const int at = row * 128 + (((col >> 3) ^ (row & 7)) << 4) + (col & 4) * 2;
  *reinterpret_cast<uint2*>(hi + at) = make_uint2(h[0], h[1]);
  *reinterpret_cast<uint2*>(lo + at) = make_uint2(l[0], l[1]);
}

struct TcArgs {
  float* P;
  float* G;
  float* M;
  const double* scale_norm;
  const int32_t* status;
  uint8_t* spill;        // [CTA][spill_tiles][kTcTileBytes]
  int32_t spill_tiles;
  int32_t held;          // tiles held per CTA: kTcSlots - 1, or kTcHeld where there are more
  int32_t zero_grads, C;
  uint32_t* err;
  unsigned long long wait_limit;   // bound of the pipeline waits (cycles); the drains keep kWaitCycles
};

// The small matrices are [64][64] fp32 with the 16-byte chunks of a row spread by the row (no bank
// conflicts for the fragment reads below): element (i, j) at mat_at(i, j).
__device__ __forceinline__ int mat_at(int i, int j) { return i * 64 + (j ^ ((i & 7) << 2)); }

__device__ __forceinline__ void mma_tf32(float (&d)[4], const float (&a)[4], float b0, float b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(__float_as_uint(a[0])), "r"(__float_as_uint(a[1])), "r"(__float_as_uint(a[2])),
        "r"(__float_as_uint(a[3])), "r"(__float_as_uint(b0)), "r"(__float_as_uint(b1)));
}

// D = gamma A B + beta E + alpha I (alpha on the first s of the diagonal) for commuting symmetric
// matrices, D one of them or another, 16 warps: warp w the rows 16 (w % 4) .. and columns
// 16 (w / 4) .., three tf32 products of a two-term split (about 2^-21). Thread-level tensor-core
// instructions fit here: the operands are fp32 in shared memory already (tcgen05 would need split
// operands written out and a trip through tensor memory each time). Bound by their latency: 4700
// cycles a product at s = 64; the upper triangle alone (two blocks in turn for some warps) took
// 5600, fp32 FMAs 6000, three chains of accumulators instead of one 5000. Not inlined: one copy of
// its code serves the fourteen products of an update.
__device__ __noinline__ void small_product(float* D, const float* A, const float* B, const float* E, int s,
                                           float alpha, float beta, float gamma) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int r = (warp & 3) * 16 + (lane >> 2), n = (warp >> 2) * 16 + (lane >> 2), kq = lane & 3;
  float acc[2][4] = {};
  // every row a lane reads has the same spread, (lane >> 2) << 2, so eight offsets cover a row
  const int spread = (lane >> 2) << 2;
  const float* pa = A + r * 64;
  const float* pb = B + n * 64;
#pragma unroll
  for (int k = 0; k < 64; k += 8) {
    if (k >= s) break;
    const int o0 = (k & 32) + (((k & 24) + kq) ^ spread), o1 = o0 ^ 4;
    const float xa[4] = {pa[o0], pa[o0 + 8 * 64], pa[o1], pa[o1 + 8 * 64]};
    const float xb[4] = {pb[o0], pb[o1], pb[o0 + 8 * 64], pb[o1 + 8 * 64]};
    float ah[4], al[4], bh[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      ah[q] = tf32_hi(xa[q]);
      al[q] = xa[q] - ah[q];
      bh[q] = tf32_hi(xb[q]);
    }
#pragma unroll
    for (int v = 0; v < 2; ++v) {
      mma_tf32(acc[v], al, bh[2 * v], bh[2 * v + 1]);
      mma_tf32(acc[v], ah, xb[2 * v] - bh[2 * v], xb[2 * v + 1] - bh[2 * v + 1]);
      mma_tf32(acc[v], ah, bh[2 * v], bh[2 * v + 1]);
    }
  }
#pragma unroll
  for (int v = 0; v < 2; ++v)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int i = r + (q >> 1) * 8, j = (warp >> 2) * 16 + v * 8 + kq * 2 + (q & 1);
      acc[v][q] = gamma * acc[v][q] + beta * E[mat_at(i, j)] + (i == j && i < s ? alpha : 0.f);
    }
  __syncthreads();
#pragma unroll
  for (int v = 0; v < 2; ++v)
#pragma unroll
    for (int q = 0; q < 4; q += 2)
      *reinterpret_cast<float2*>(D + mat_at(r + (q >> 1) * 8, (warp >> 2) * 16 + v * 8 + kq * 2)) =
          make_float2(acc[v][q], acc[v][q + 1]);
  __syncthreads();
}

__global__ void __launch_bounds__(kTcThreads, 1) k_muon_tc(const __grid_constant__ MuonTab tab,
                                                             const MuonK hp, const TcArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* tiles = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* scratch = tiles + kTcHeld * kTcTileBytes;    // kTcScr spilled tiles
  uint8_t* small = tiles + (kTcSlots - 1) * kTcTileBytes;   // two small matrices, over the last room
  uint8_t* qop = tiles + kTcSlots * kTcTileBytes;       // [Q_hi; Q_lo] operand, or Q in fp32
  float* g0 = reinterpret_cast<float*>(qop + 16 * 1024);   // Gram matrix
  float* sh = g0 + 64 * 64;                         // [20]
  uint64_t* bar_apply = reinterpret_cast<uint64_t*>(sh + 20);   // [2]
  uint64_t* bar_gram = bar_apply + 2;
  uint64_t* bar_load = bar_gram + 1;        // [kTcScr]: a spilled tile is back
  uint64_t* bar_used = bar_load + kTcScr;   // [kTcScr]: a spilled tile's Gram products are done
  uint64_t* bar_done = bar_used + kTcScr;   // every MMA of this CTA is done
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bar_done + 1);
  volatile uint32_t* failed = tmem_slot + 1;
  float* t1 = reinterpret_cast<float*>(small);
  float* t2 = t1 + 64 * 64;
  float* qf = reinterpret_cast<float*>(qop);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int C = a.C;
  const int rank = C > 1 ? (int)cluster_ctarank() : 0;
  if (tid == 0) {
    mbar_init(&bar_apply[0], 1);
    mbar_init(&bar_apply[1], 1);
    *failed = 0u;
    mbar_init(bar_gram, 1);
    mbar_init(bar_done, 1);
    for (int b = 0; b < kTcScr; ++b) {
      mbar_init(&bar_load[b], 1);
      mbar_init(&bar_used[b], 1);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  grid_dep_sync();
  if (warp == 0) tmem_alloc(tmem_slot, 512);
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint32_t tm_gram = tmem, tm_apply = tmem + 128;   // apply buffers at +128 and +256
  // Spilled tiles should live in L2 (each CTA writes its own room again and again); the arenas pass
  // through it once.
  uint64_t keep;
  asm("createpolicy.fractional.L2::evict_last.b64 %0, 1.0;" : "=l"(keep));
  uint8_t* spill = a.spill + (size_t)blockIdx.x * a.spill_tiles * kTcTileBytes;
  constexpr uint32_t id_gram = idesc(kFmtBF16, 128, 128, true, true);
  constexpr uint32_t id_apply = idesc(kFmtBF16, 128, 128);
  uint32_t ph_apply[2] = {0, 0}, ph_gram = 0;   // the same in every thread
  uint32_t ph_load = 0, ph_used = 0;   // a bit per room, of thread 0, which alone waits on them
  uint32_t fetching = 0;               // thread 0: rooms with a copy on its way
  const int held = a.held;
  // A wait that runs out of its bound marks its CTA: once a thread knows of it (`ok`), it begins no copy and
  // no product, waits no more and writes no parameters, but keeps up with the cluster's barriers. With the
  // next Gram matrix the whole cluster learns of it and leaves (`gone`), so that an invalid matrix is never
  // used: each element of the parameters holds its update or is as it was.
  bool ok = true, gone = false;
  // One warp polls, the others wait at the barrier: polling by all of them took most of the issue slots.
  auto wait = [&](uint64_t* bar, uint32_t ph) {
    if (warp == 0 && !(ok && mbar_wait_strict(bar, ph, 2u, a.err, a.wait_limit))) *failed = 1u;
    __syncthreads();
    ok = *failed == 0u;
    fence_after();
  };
  // whether a CTA of the cluster is marked; after a barrier of the cluster, and none waits before the next
  auto marked = [&]() {
    const float* f = reinterpret_cast<const float*>(const_cast<const uint32_t*>(failed));
    return __any_sync(0xffffffffu, lane < C && __float_as_uint(dsmem_ld(f, (uint32_t)lane)) != 0u);
  };
  // every thread's writes to shared memory become visible to the tensor cores and bulk copies
  auto publish = [&]() {
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    fence_before();
    __syncthreads();
    fence_after();
  };

  for (int mi = (int)blockIdx.x / C; mi < tab.n; mi += (int)gridDim.x / C) {
    const MuonMat mt = tab.m[mi];
    if (a.status[mt.group] != LORA_OK) continue;
    const float c = (float)a.scale_norm[2 * mt.group], mu = hp.mu;
    const int s = mt.s;
    const int64_t all = (mt.n + 127) / 128;
    const int64_t first = all * rank / C;
    const int nt = (int)(all * (rank + 1) / C - first);
    const int64_t sj = mt.tall ? s : 1, si = mt.tall ? 1 : mt.n;
    float* p = a.P + mt.offset;
    float* g = a.G + mt.offset;
    float* m = a.M + mt.offset;
    const bool nesterov = hp.nesterov;
    const float mu_u = nesterov ? mu : 1.f, c_u = nesterov ? c : 0.f;   // u = c_u g + mu_u m
    // Tile t of this CTA: held, or, while it is in use, in room (t - held) % kTcScr of the scratch.
    // Spilled tiles move by bulk copies of thread 0.
    auto room = [&](int t) { return (t - held) % kTcScr; };
    auto place = [&](int t) { return t < held ? tiles + t * kTcTileBytes : scratch + room(t) * kTcTileBytes; };
    auto wait0 = [&](uint64_t* bars, uint32_t& ph, int b) {   // thread 0
      const bool done = mbar_wait_strict(&bars[b], (ph >> b) & 1u, 2u, a.err, a.wait_limit);
      if (done) {
        ph ^= 1u << b;
      } else {
        *failed = 1u;
        ok = false;
      }
      fence_after();
      return done;
    };
    auto begin_fetch = [&](int t) {
      fetching |= 1u << room(t);
      uint64_t* bar = &bar_load[room(t)];
      mbar_expect_tx(bar, kTcTileBytes);
      asm volatile(
          "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], %4;" ::"r"(
              smem_u32(place(t))),
          "l"(spill + (size_t)(t - held) * kTcTileBytes), "r"(kTcTileBytes), "r"(smem_u32(bar)), "l"(keep)
          : "memory");
    };
    auto end_fetch = [&](int t) {
      if (wait0(bar_load, ph_load, room(t))) fetching &= ~(1u << room(t));
    };
    auto begin_flush = [&](int t) {   // after publish
      asm volatile("cp.async.bulk.global.shared::cta.bulk_group.L2::cache_hint [%0], [%1], %2, %3;" ::"l"(
                       spill + (size_t)(t - held) * kTcTileBytes),
                   "r"(smem_u32(place(t))), "r"(kTcTileBytes), "l"(keep)
                   : "memory");
      asm volatile("cp.async.bulk.commit_group;" ::: "memory");
    };
    auto end_flushes = [&]() {   // the spilled tiles are in global memory
      asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
      asm volatile("fence.proxy.async;" ::: "memory");
    };
    // The room of a pass's spilled tile is free: its user kTcScr spilled tiles earlier in the pass has
    // been copied out and its Gram products are done. In the first pass one later copy has begun by
    // then, in the others none.
    auto room_free = [&](int t, bool first_pass) {
      if (first_pass) asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
      else asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
      wait0(bar_used, ph_used, room(t));
    };
    // the last uses of the rooms, at the end of a pass
    auto drain_used = [&]() {
      for (int k = 0; k < min(nt - held, kTcScr); ++k) wait0(bar_used, ph_used, k);
    };
    auto gram_mma = [&](const uint8_t* tile, bool begin) {   // thread 0
      const uint64_t d = smem_desc_sw128_mn(smem_u32(tile), 16 * 1024);
#pragma unroll
      for (int k = 0; k < 8; ++k) umma_f16(tm_gram, d + 128 * k, d + 128 * k, id_gram, (begin && k == 0) ? 0u : 1u);
    };
    auto apply_mma = [&](const uint8_t* tile, int buf) {     // thread 0
      const uint64_t dq = smem_desc_sw128(smem_u32(qop));
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint64_t d = smem_desc_sw128(smem_u32(tile) + h * 16 * 1024);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          umma_f16(tm_apply + 128u * (uint32_t)buf, d + 2 * k, dq + 2 * k, id_apply, (h || k) ? 1u : 0u);
      }
      umma_commit(&bar_apply[buf]);
    };

    // ---- momentum and u. A thread's part of a tile: four 16-byte vectors of the arena, 512 threads
    // apart (tall: whole lines per request), or two units of 8 rows of a column, one column per lane
    // (wide).
    int row[2], ch[2], live[2];   // wide: column, chunk of 8 rows, how many of them exist
    int64_t at0[2];               // wide: where the unit starts in the first tile
#pragma unroll
    for (int un = 0; un < 2; ++un) {
      const int e = un * 16 + warp;   // 32 units of (chunk, 32 columns)
      row[un] = (e & 3) * 32 + lane;
      ch[un] = e >> 2;
      live[un] = min(8, max(0, s - ch[un] * 8));
      at0[un] = first * 128 + row[un] + (int64_t)(ch[un] * 8) * si;
    }
    const int vrow = tid >> 4, vq = (tid & 15) * 4;   // tall: column vrow + 32 v, rows vq ..
    const int64_t v0 = (first * 128 + vrow) * (int64_t)s + vq;
    const int left0 = (int)(mt.n - first * 128);   // columns from the first tile to the end
    float gv[16], mv[16];
    auto load = [&](int t) {
      if (mt.tall) {
        const float4 z = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const bool in = t < nt && vq < s && t * 128 + vrow + 32 * v < left0;
          const int64_t at = v0 + ((int64_t)t * 128 + 32 * v) * s;
          *reinterpret_cast<float4*>(gv + 4 * v) = in ? __ldcs(reinterpret_cast<const float4*>(g + at)) : z;
          *reinterpret_cast<float4*>(mv + 4 * v) = in ? __ldcs(reinterpret_cast<const float4*>(m + at)) : z;
        }
      } else {
#pragma unroll
        for (int un = 0; un < 2; ++un) {
          const int k = t < nt && t * 128 + row[un] < left0 ? live[un] : 0;
          const float* gp = g + at0[un] + (int64_t)t * 128;
          const float* mp = m + at0[un] + (int64_t)t * 128;
#pragma unroll
          for (int q = 0; q < 8; ++q, gp += si, mp += si) {
            gv[un * 8 + q] = q < k ? __ldcs(gp) : 0.f;
            mv[un * 8 + q] = q < k ? __ldcs(mp) : 0.f;
          }
        }
      }
    };
    // Lines of later tiles to L2, one per thread and array (a tile is at most 256 lines): registers
    // hold one tile ahead, which covers L2's latency but not memory's.
    auto prefetch = [&](const float* base, int t, int l) {
      const int64_t j0 = (first + t) * 128;
      if (t >= nt) return;
      int64_t at;
      if (mt.tall) {
        at = j0 * s + (int64_t)l * 32;
        if (l >= 4 * s || at >= mt.n * s) return;
      } else {
        at = (int64_t)(l >> 2) * si + j0 + (l & 3) * 32;
        if ((l >> 2) >= s || j0 + (l & 3) * 32 >= mt.n) return;
      }
      asm volatile("prefetch.global.L2 [%0];" ::"l"(base + at));
    };
    for (int t = 1; t < kTcAhead; ++t) prefetch(tid < 256 ? g : m, t, tid & 255);
    load(0);
    for (int t = 0; t < nt; ++t) {
      prefetch(tid < 256 ? g : m, t + kTcAhead, tid & 255);
      uint8_t* hi = place(t);
      uint8_t* lo = hi + 16 * 1024;
      float w[16];
#pragma unroll
      for (int q = 0; q < 16; ++q) {
        mv[q] = fmaf(mu, mv[q], c * gv[q]);
        w[q] = fmaf(mu_u, mv[q], c_u * gv[q]);
      }
      if (mt.tall) {
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          if (vq >= s || t * 128 + vrow + 32 * v >= left0) continue;
          const int64_t at = v0 + ((int64_t)t * 128 + 32 * v) * s;
          __stcs(reinterpret_cast<float4*>(m + at), *reinterpret_cast<const float4*>(mv + 4 * v));
          if (a.zero_grads) __stcs(reinterpret_cast<float4*>(g + at), make_float4(0.f, 0.f, 0.f, 0.f));
        }
      } else {
#pragma unroll
        for (int un = 0; un < 2; ++un) {
          const int k = t * 128 + row[un] < left0 ? live[un] : 0;
          float* mp = m + at0[un] + (int64_t)t * 128;
#pragma unroll
          for (int q = 0; q < 8; ++q, mp += si)
            if (q < k) __stcs(mp, mv[un * 8 + q]);
          if (a.zero_grads) {
            float* gp = g + at0[un] + (int64_t)t * 128;
            for (int q = 0; q < k; ++q, gp += si) *gp = 0.f;
          }
        }
      }
      load(t + 1);   // on its way while this tile is split and stored
      if (mt.tall) {
#pragma unroll
        for (int v = 0; v < 4; ++v) put_split4(hi, lo, vrow + 32 * v, vq, w + 4 * v);
      } else {
#pragma unroll
        for (int un = 0; un < 2; ++un) put_split8(hi, lo, row[un], ch[un], w + 8 * un);
      }
      // the next tile's room, checked while this tile is finished; publish tells the other threads
      if (tid == 0 && ok && t + 1 < nt && t + 1 >= held + kTcScr) room_free(t + 1, true);
      publish();
      if (tid == 0 && ok) {
        gram_mma(hi, t == 0);
        if (t >= held) {
          umma_commit(&bar_used[room(t)]);
          begin_flush(t);
        }
        if (t + 1 == nt) {
          umma_commit(bar_gram);
          end_flushes();
          drain_used();
        }
      }
    }

    // G of the tiles (the Gram products in D_gram), summed over the cluster, in g0; invalid once `gone`
    auto gram_all = [&]() {
      if (nt > 0) {
        wait(bar_gram, ph_gram);
        ph_gram ^= 1u;
      }
      // ---- G = the sum of D's quadrants, then over the cluster
      if (warp < 4) {
        const uint32_t d = tm_gram + ((uint32_t)(warp * 32) << 16);
        const int grow = (warp & 1) * 32 + lane;
#pragma unroll
        for (int h = 0; h < 64; h += 32) {
          float v[32];
          if (nt > 0) {
            float x[32];
            tmem_ld32(d + (uint32_t)h, v);
            tmem_ld32(d + 64u + (uint32_t)h, x);
#pragma unroll
            for (int q = 0; q < 32; ++q) v[q] += x[q];
          } else {
#pragma unroll
            for (int q = 0; q < 32; ++q) v[q] = 0.f;
          }
          if (warp < 2) {
#pragma unroll
            for (int q = 0; q < 32; q += 4) store4(g0 + mat_at(grow, h + q), v + q);
          }
          asm volatile("bar.sync 1, 128;" ::: "memory");
          if (warp >= 2) {
#pragma unroll
            for (int q = 0; q < 32; q += 4) {
              float4* at = reinterpret_cast<float4*>(g0 + mat_at(grow, h + q));
              const float4 o = *at;
              *at = make_float4(o.x + v[q], o.y + v[q + 1], o.z + v[q + 2], o.w + v[q + 3]);
            }
          }
        }
        fence_before();
      }
      __syncthreads();
      if (C == 1) {
        gone = *failed != 0u;
      } else {
        // CTA r adds an r-th of the matrix over the ranks, then every CTA gathers the parts
        const int per = 1024 / C;
        cluster_sync();
        gone = marked();
        for (int e = tid; e < per; e += kTcThreads) {
          const int at = rank * per + e;
          float4 v = dsmem_ld4(g0 + at * 4, 0);
          for (int r = 1; r < C; ++r) {
            const float4 o = dsmem_ld4(g0 + at * 4, (uint32_t)r);
            v.x += o.x; v.y += o.y; v.z += o.z; v.w += o.w;
          }
          *reinterpret_cast<float4*>(t1 + at * 4) = v;
        }
        cluster_sync();
        for (int at = tid; at < 1024; at += kTcThreads) {
          const float4 v = dsmem_ld4(t1 + at * 4, (uint32_t)(at / per));
          *reinterpret_cast<float4*>(g0 + at * 4) = v;
        }
        cluster_sync();   // the peers have read t1
      }
    };

    bool backwards = false;
    for (int done = 0; done < hp.steps;) {
      const int left = hp.steps - done;
      const int now = left % kStageSteps ? left % kStageSteps : kStageSteps;
      gram_all();
      if (gone) break;
      float inv = 1.f;
      if (done == 0) {   // X = u / ||u||, ||u||^2 = trace G
        auto trace = [&]() {
          float tr = g0[mat_at(lane, lane)] + g0[mat_at(lane + 32, lane + 32)];   // zeros past s
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) tr += __shfl_xor_sync(0xffffffffu, tr, o);
          return tr;   // the same in every lane
        };
        float tr = trace();
        if (!(tr > 1e-18f && tr < 1e30f)) {
          // the squares may have left the fp32 range (or u is zero): scale u by a power of two that
          // brings its largest magnitude to about one, and sum again
          float mx = 0.f, pre = 1.f;
          for (int pass = 0; pass < 2; ++pass) {
            if (pass == 1 && pre == 1.f) break;
            publish();
            for (int t = 0; t < nt; ++t) {
              uint32_t* w = reinterpret_cast<uint32_t*>(place(t));
              if (tid == 0 && ok && t >= held) {
                begin_fetch(t);
                end_fetch(t);
              }
              __syncthreads();
              if (pass == 0) {
                for (int e = tid; e < kTcTileBytes / 8; e += kTcThreads)   // the hi terms
                  mx = fmaxf(mx, fmaxf(fabsf(__uint_as_float(w[e] << 16)), fabsf(__uint_as_float(w[e] & 0xFFFF0000u))));
                publish();
                continue;
              }
              for (int e = tid; e < kTcTileBytes / 4; e += kTcThreads)
                w[e] = pack_bf16(__uint_as_float(w[e] << 16) * pre, __uint_as_float(w[e] & 0xFFFF0000u) * pre);
              publish();
              if (tid == 0 && ok) {
                gram_mma(place(t), t == 0);
                if (t >= held) {
                  umma_commit(&bar_used[room(t)]);
                  begin_flush(t);
                  end_flushes();
                  wait0(bar_used, ph_used, room(t));
                }
                if (t + 1 == nt) umma_commit(bar_gram);
              }
              __syncthreads();
            }
            if (pass == 0) {
              pre = range_scale<kTcThreads>(mx, sh, C);
              if (C > 1) cluster_sync();
              gone = marked();
              if (C > 1) cluster_sync();
              else __syncthreads();
              if (gone) break;
            }
          }
          if (!gone && pre != 1.f) {
            gram_all();
            tr = trace();
          }
          if (gone) break;
        }
        inv = tr > 0.f ? 1.f / sqrtf(tr) : 0.f;
        __syncthreads();
        for (int e = tid; e < 64 * 64; e += kTcThreads) g0[e] *= inv * inv;
        __syncthreads();
      }
      // ---- the stage's steps on G: P = a I + b G + c G^2, Q <- P Q, G <- P^2 G
      float* q_now = t1;   // the first step's P is the product so far
      for (int k = 0; k < now; ++k) {
        float* pk = k == 0 ? t1 : t2;
        small_product(pk, g0, g0, g0, s, hp.a, hp.b, hp.c);
        if (k > 0) {
          small_product(qf, pk, q_now, g0, s, 0.f, 0.f, 1.f);
          q_now = qf;
        }
        if (k + 1 < now) {
          // P^2 goes where neither P nor Q is: over the other small matrix
          float* sq = k == 0 ? t2 : t1;
          small_product(sq, pk, pk, g0, s, 0.f, 0.f, 1.f);
          small_product(g0, g0, sq, g0, s, 0.f, 0.f, 1.f);
        }
      }
      done += now;
      // [Q_hi; Q_lo] as the B operand: 8 elements of a row per thread
      {
        const int row = tid >> 3, ch = tid & 7;
        float v[8];
        *reinterpret_cast<float4*>(v) = *reinterpret_cast<const float4*>(q_now + mat_at(row, ch * 8));
        *reinterpret_cast<float4*>(v + 4) = *reinterpret_cast<const float4*>(q_now + mat_at(row, ch * 8 + 4));
#pragma unroll
        for (int q = 0; q < 8; ++q) v[q] *= inv;
        __syncthreads();   // Q may lie where the operand goes
        put_split8(qop, qop + 64 * 128, row, ch, v);
      }
      publish();
      // ---- X <- Q X: into the tiles, with the next Gram matrix, or into the parameters
      const bool last = done >= hp.steps;
      const int quad = warp & 3, ih = warp >> 2;   // TMEM lanes, 16 of the 64 rows of X
      const int jrow = quad * 32 + lane;
      // Passes go through the tiles in turn forwards (the first, over g and m) and backwards, so that
      // a pass begins with the spilled tiles that were written last.
      backwards = !backwards;
      auto order = [&](int i) { return backwards ? nt - 1 - i : i; };
      if (tid == 0 && ok && nt > 0) {
        for (int k = 0; k < min(nt - held, kTcScr - 1); ++k) begin_fetch(backwards ? nt - 1 - k : held + k);
        if (order(0) < held) apply_mma(place(order(0)), 0);
      }
      // The parameters of a tile are on their way while the tile before it is updated. A thread's are
      // four 16-byte vectors, 512 threads apart (tall), or 16 rows of a column, four apart (wide).
      float pn[16];
      const int prow = mt.tall ? tid >> 4 : tid & 127, pq = mt.tall ? (tid & 15) * 4 : tid >> 7;
      float* p0 = p + (first * 128 + prow) * sj + pq * si;
      const bool pcol = pq < s;
      auto load_p = [&](int t) {
        const float* pp = p0 + (int64_t)t * 128 * sj;
        if (mt.tall) {
#pragma unroll
          for (int v = 0; v < 4; ++v)
            if (t < nt && pcol && t * 128 + prow + v * 32 < left0)
              *reinterpret_cast<float4*>(pn + 4 * v) = __ldcs(reinterpret_cast<const float4*>(pp + v * 32 * sj));
        } else {
          const int k = t < nt && t * 128 + prow < left0 ? s - pq : 0;
#pragma unroll
          for (int v = 0; v < 16; ++v, pp += 4 * si)
            if (4 * v < k) pn[v] = __ldcs(pp);
        }
      };
      if (last && nt > 0) {
        load_p(order(0));
        if (tid >= 256)
          for (int i = 1; i < min(kTcAhead, nt); ++i) prefetch(p, order(i), tid & 255);
      }
      bool early = false;   // thread 0: a spilled tile's products have begun
      for (int i = 0; i < nt; ++i) {
        const int t = order(i), next = i + 1 < nt ? order(i + 1) : INT32_MAX;   // the latter: none
        if (last && tid >= 256 && i + kTcAhead < nt) prefetch(p, order(i + kTcAhead), tid & 255);
        const int buf = i & 1;
        uint8_t* tile = place(t);
        if (tid == 0 && ok) {
          if (t >= held) {
            if (!early) {
              end_fetch(t);
              apply_mma(tile, buf);
            }
            // the tile kTcScr - 1 ahead, into the room of the spilled tile before this one
            const int k = backwards ? nt - 1 - t : t - held, f = order(i + kTcScr - 1);
            if (k + kTcScr - 1 < nt - held) {
              if (!last && k >= 1) room_free(f, false);
              begin_fetch(f);
            }
          }
          // the next tile's products run while this one is read, if it is there
          early = false;
          if (next < held) {
            apply_mma(place(next), buf ^ 1);
          } else if (next < nt && mbar_test(&bar_load[room(next)], (ph_load >> room(next)) & 1u)) {
            end_fetch(next);
            apply_mma(place(next), buf ^ 1);
            early = true;
          }
        }
        wait(&bar_apply[buf], ph_apply[buf]);
        ph_apply[buf] ^= 1u;
        float x[16];
        {
          float y[16];
          const uint32_t d = tm_apply + 128u * (uint32_t)buf + ((uint32_t)(quad * 32) << 16) + (uint32_t)(ih * 16);
          tmem_ld16(d, x);
          tmem_ld16(d + 64u, y);
#pragma unroll
          for (int q = 0; q < 16; ++q) x[q] += y[q];
        }
        if (!last) {
#pragma unroll
          for (int q = 0; q < 2; ++q) put_split8(tile, tile + 16 * 1024, jrow, ih * 2 + q, x + q * 8);
          publish();
          if (tid == 0 && ok) {
            gram_mma(tile, i == 0);
            if (t >= held) {
              umma_commit(&bar_used[room(t)]);
              begin_flush(t);
            }
            if (i + 1 == nt) {
              umma_commit(bar_gram);
              end_flushes();
              drain_used();
            }
          }
        } else {
          // X [128][64] fp32 over the tile, 16-byte chunks spread by the row
#pragma unroll
          for (int q = 0; q < 4; ++q)
            store4(reinterpret_cast<float*>(tile + jrow * 256 + (((ih * 4 + q) ^ (jrow & 15)) << 4)), x + q * 4);
          fence_before();
          __syncthreads();
          fence_after();
          const float step = mt.step, dec = mt.lr * mt.decay;
          float pc[16];
#pragma unroll
          for (int v = 0; v < 16; ++v) pc[v] = pn[v];
          load_p(next);
          float* pp = p0 + (int64_t)t * 128 * sj;
          if (mt.tall) {
            if (pcol && ok) {
#pragma unroll
              for (int v = 0; v < 4; ++v) {
                const int j = prow + v * 32;
                if (t * 128 + j >= left0) continue;
                const float4 xv = *reinterpret_cast<const float4*>(tile + j * 256 + (((pq >> 2) ^ (j & 15)) << 4));
                const float xs[4] = {xv.x, xv.y, xv.z, xv.w};
#pragma unroll
                for (int z = 0; z < 4; ++z) pc[4 * v + z] = pc[4 * v + z] - step * xs[z] - dec * pc[4 * v + z];
                __stcs(reinterpret_cast<float4*>(pp + v * 32 * sj), *reinterpret_cast<const float4*>(pc + 4 * v));
              }
            }
          } else {
            const int k = ok && t * 128 + prow < left0 ? s - pq : 0;
            const uint8_t* xrow = tile + prow * 256 + pq * 4;
#pragma unroll
            for (int v = 0; v < 16; ++v, pp += 4 * si) {
              if (4 * v >= k) continue;
              const float xv = *reinterpret_cast<const float*>(xrow + ((v ^ (prow & 15)) << 4));
              __stcs(pp, pc[v] - step * xv - dec * pc[v]);
            }
          }
          publish();   // a spilled tile's room is the next one's
        }
      }
    }
    __syncthreads();
    if (gone) break;
  }
  // every copy and every MMA is done before the tensor memory is freed (after a failed wait nothing else
  // says so); the peers are done with this CTA's memory
  if (tid == 0) {
    for (int b = 0; b < kTcScr; ++b)
      if (fetching >> b & 1u) mbar_wait(&bar_load[b], (ph_load >> b) & 1u, 2u, a.err);
    asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    umma_commit(bar_done);
    mbar_wait(bar_done, 0u, 2u, a.err);
  }
  fence_before();
  __syncthreads();
  fence_after();
  if (warp == 0) tmem_dealloc(tmem, 512);
}

// One launch of `kernel` over the table's matrices, a cluster of C CTAs each, persistent.
template <typename K, typename... Args>
cudaError_t launch_clusters(K kernel, int threads, int smem, int n, int C, int most, cudaStream_t st, const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = st;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)C;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = add_pdl_attr(at, 1);
  cfg.gridDim = dim3((unsigned)C);
  if (most < (1 << 20)) {   // persistent: as many clusters as are resident at a time
    static DeviceValues<17> fits;   // by cluster size
    cudaError_t e = cudaSuccess;
    const int fit = fits.get(current_device(), C, [&] {
      int n = 0;
      e = cudaOccupancyMaxActiveClusters(&n, kernel, &cfg);
      return e == cudaSuccess ? std::max(n, 1) : -1;
    });
    if (e != cudaSuccess) return e;
    most = std::min(most / C, fit);
  }
  cfg.gridDim = dim3((unsigned)(std::max(1, std::min(n, most)) * C));
  prof_begin(0, st);
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <typename K>
cudaError_t set_attrs(K kernel, int smem) {
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  return e;
}

template <int S4>
cudaError_t run_simt(float* p, float* g, float* m, const MuonTab& tab, const MuonK& hp,
                     const double* scale_norm, const int32_t* status, int zero_grads, int C,
                     int held, cudaStream_t st) {
  using F = SimtCfg<S4>;
  static std::atomic<uint64_t> set{0};
  const cudaError_t e =
      once_on_device(set, [] { return set_attrs(k_muon_simt<S4>, (F::kSmallFloats + F::kCap * F::SP) * 4); });
  if (e != cudaSuccess) return e;
  const int smem = (F::kSmallFloats + std::min(held, F::kCap) * F::SP) * 4;
  return launch_clusters(k_muon_simt<S4>, kMuonThreads, smem, tab.n, C, 1 << 20, st, p, g, m, tab, hp, scale_norm,
                         status, zero_grads, C);
}

}  // namespace

// CTAs of a matrix's cluster on CUDA cores: 512 columns a CTA, fewer while there are SMs left.
int muon_cluster_simt(const MuonMat& m, int n_mats) {
  int C = 1;
  while (C < 16 && (m.n > 512 * (int64_t)C || (n_mats * C * 2 <= 152 && m.n > 128 * C))) C *= 2;
  return C;
}

// On tensor cores, for the `count` matrices of a call with long axes n in falling order: the size
// whose first cluster, which takes every R-th matrix (R: clusters resident at once), is done first. A
// matrix costs a tile's time for each tile of a CTA and about six more, the chain of its small
// products and cluster barriers, which every CTA repeats (us with the next power of two that filled
// the SMs / with this rule: 24 matrices of 2560 and 1024 112 / 78, 44 of 2048 116 / 90, 64 of 4096 219 / 180, 4
// layers of 4096 and 14336 161 / 147; 32 such layers 370 either way).
int muon_cluster_tc(const int64_t* n, int count) {
  constexpr int kResident[5] = {152, 76, 37, 17, 5};   // of 1, 2, 4, 8, 16 CTAs
  int best = 1;
  int64_t least = INT64_MAX;
  for (int k = 0; k < 5; ++k) {
    const int C = 1 << k;
    int64_t cost = 0;
    for (int i = 0; i < count; i += kResident[k]) cost += 6 + ((n[i] + 127) / 128 + C - 1) / C;
    if (cost < least) {
      least = cost;
      best = C;
    }
  }
  return best;
}

size_t muon_spill_bytes(const MuonMat& m, int C, int n) {
  if (m.s <= 16) return 0;
  const int64_t tiles = ((m.n + 127) / 128 + C - 1) / C;
  if (tiles < kTcSlots) return 0;
  const int64_t ctas = (int64_t)std::max(1, std::min(n, kMuonMaxCtas / C)) * C;
  return (size_t)ctas * (tiles - kTcHeld) * kTcTileBytes;
}

cudaError_t launch_muon(float* p, float* g, float* m, const MuonTab& tab, const MuonK& hp,
                        const double* scale_norm, const int32_t* status, int zero_grads, int C,
                        void* spill, cudaStream_t st) {
  int64_t n = 0;
  for (int i = 0; i < tab.n; ++i) n = std::max(n, tab.m[i].n);
  if (tab.m[0].s <= 16) {
    const int held = (int)std::min<int64_t>((n / 4 + C - 1) / C * 4, 1 << 20);
    switch (tab.m[0].s / 4) {
      case 1: return run_simt<1>(p, g, m, tab, hp, scale_norm, status, zero_grads, C, held, st);
      case 2: return run_simt<2>(p, g, m, tab, hp, scale_norm, status, zero_grads, C, held, st);
      case 3: return run_simt<3>(p, g, m, tab, hp, scale_norm, status, zero_grads, C, held, st);
      default: return run_simt<4>(p, g, m, tab, hp, scale_norm, status, zero_grads, C, held, st);
    }
  }
  static std::atomic<uint64_t> set{0};
  const cudaError_t e = once_on_device(set, [] { return set_attrs(k_muon_tc, kTcSmem); });
  if (e != cudaSuccess) return e;
  TcArgs a{};
  a.P = p; a.G = g; a.M = m;
  a.scale_norm = scale_norm; a.status = status;
  a.spill = static_cast<uint8_t*>(spill);
  const int64_t tiles = ((n + 127) / 128 + C - 1) / C;
  a.held = tiles < kTcSlots ? kTcSlots - 1 : kTcHeld;
  a.spill_tiles = (int32_t)std::max<int64_t>(0, tiles - a.held);
  a.zero_grads = zero_grads; a.C = C;
  a.err = error_word();
  if (!a.err) return cudaErrorInvalidDevice;
  a.wait_limit = tc_wait_limit();
  return launch_clusters(k_muon_tc, kTcThreads, kTcSmem, tab.n, C, kMuonMaxCtas, st, tab, hp, a);
}

}  // namespace lora
