// Frozen product over E4M3 codes with one scale per block of 128, on sm_103a tensor cores:
//
//   Y[t, n] = sum_kb sx[t, kb] sw[n / 128, kb] D_kb[t, n] (+ mask (P Q^T)[t, n]),
//   D_kb[t, n] = sum_{k in block kb} x8[t, k] w8[n, k]
//
// The scales change along the contraction, so one accumulator cannot run over it: every block of
// 128 is summed on the tensor cores (kind::f8f6f4) into one of two TMEM buffers, and the epilogue
// warps add it, scaled, to fp32 accumulators in their registers while the next block's MMAs run
// into the other buffer. The LoRA term (kind::tf32) is one more such block per 32 of the rank, with
// scale one.
//
// For the input gradient the weight's codes are read in place: the operand is [out, in] with the
// contraction along the rows, an MN-major tile in the 128-byte swizzle.
//
// Two kernels. k_block_tile: 128 tokens x BN outputs, tokens as the M side. k_block_stream: 128
// outputs x NT tokens, the weight as the M side and the contraction split over a cluster, for few
// tokens, where the weight's bytes bound the product.
#include <cstring>
#include <mutex>

#include "block_e4m3.cuh"
#include "tc_ptx.cuh"

namespace lora {

namespace {
using namespace tc;

constexpr int kBlk = LORA_SCALE_BLOCK;
constexpr int kTileBytes = 128 * 128;   // 128 rows of 128 bytes

__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

__device__ __forceinline__ void tmem_ld32_nw(uint32_t taddr, uint32_t (&r)[32]) {
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

constexpr uint64_t kNan2 = 0x7FFFFFFF7FFFFFFFull;   // a pair of NaNs

__device__ __forceinline__ void tmem_ldc(uint32_t taddr, uint32_t (&r)[32]) { tmem_ld32_nw(taddr, r); }
__device__ __forceinline__ void tmem_ldc(uint32_t taddr, uint32_t (&r)[16]) { tmem_ld16_nw(taddr, r); }

// Two floats in a 64-bit register pair; a += s * (d0, d1), two FMAs in one instruction. The
// accumulators stay packed, so that no moves pair them up.
__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(a), "f"(b));
  return v;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ void fma2(uint64_t& a, uint64_t s, uint32_t d0, uint32_t d1) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(d0), "r"(d1));
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(a) : "l"(s), "l"(d));
}

// ---- 128 tokens x BN outputs ------------------------------------------------------------------
// Warps: 0 TMA, 1 and 2 MMA (one thread each, taking the blocks in turn, so that one waits for its
// operands and its accumulator while the other's MMAs run), 3 relay, 4 .. 11 epilogue: warp w takes
// TMEM lanes 32 (w % 4) .. and columns (w - 4) / 4 * BN / 2 .., so that a thread holds BN / 2
// accumulators of one row and, BN / 2 dividing 128, one weight scale per block.
//
// The relay waits for a block's sums on the mbarrier and passes them on through a named barrier,
// with the products of the two scales in shared memory: the epilogue's loop is then free of
// polling, branches and global loads (with them the compiler moved every accumulator between
// registers once per block, and the loop took three times as long).
//
// Bound by the epilogue's reads of tensor memory: a block takes about 950 cycles against the
// MMAs' 512, and the epilogue warps wait 14 of them for their next block and read for 790, beside
// MMAs that themselves read and write the other accumulator. Wider reads (32 columns), scalar FMAs,
// sixteen epilogue warps of 64 columns (436 us) and a fourth stage of operands measured the same or
// slower. 8192 x 4096 -> 14336 403 us a
// call, the quantisation's 16 included, in a series of tens (2390 TF/s), 430 to 441 in series of hundreds, at
// the power limit (the per-row-scaled product, which reads its accumulator once per tile, runs at 2690).
constexpr int kTileThreads = 384;
constexpr int kEpiWarps = 8;
constexpr int kLaunchRegs = 168, kIssueRegs = 72, kEpiRegs = 216;   // per thread
static_assert(128 * kIssueRegs + 32 * kEpiWarps * kEpiRegs <= kTileThreads * kLaunchRegs,
              "setmaxnreg draws on the block's own registers");
constexpr int kBox = 32 * 64;   // 32 rows x 32 bf16 columns, 64-byte swizzle

template <int BN>
struct TileCfg {
  static_assert(BN == 256 || BN == 128, "columns of one warp lie in one block of 128");
  static constexpr int kStageBytes = kTileBytes + BN * 128;
  // three stages feed the MMAs as well as four (404 us against 407, 8192 x 4096 -> 14336); the
  // fourth's room holds a whole tile's output, so that the epilogue never waits for its own stores
  static constexpr int kStages = BN == 256 ? 3 : 5;
  static constexpr int kSlots = 512 / BN;            // accumulators in TMEM
  static constexpr int kScaleBytes = 2 * kSlots * 2 * 128 * 4;   // [2 kSlots][half][128 rows]
  static constexpr int kEpiBytes = kEpiWarps * (BN / 64) * kBox;
  static constexpr int kSmem = kStages * kStageBytes + kEpiBytes + kScaleBytes + 512 + 1024;
  static_assert(kSmem <= 227 * 1024, "shared memory per CTA");
};

struct TileParams {
  CUtensorMap ta;     // codes [T, K], box {128, 128}
  CUtensorMap tb;     // W8 [out, in], box {128, BN} (forward) or {128, 128} (transposed)
  CUtensorMap to;     // Y [T, N] bf16, box {32, 32}
  CUtensorMap tp;     // P [T, rank] fp32, box {32, 128}
  CUtensorMap tq;     // Q [N, rank] fp32, box {32, BN}
  const float* sx;
  const float* sw;
  int64_t ld_sx;
  int64_t sw_n, sw_k;           // strides of sw over blocks of N and of K
  int64_t T, N;
  int32_t nk, n_lora;           // K-blocks; 32-wide LoRA blocks (0: none)
  int32_t n_tiles, m_tiles, group_m, total;
  int32_t splits;               // CTAs (of a cluster) that share a tile's blocks
  __nv_bfloat16* Y;
  uint32_t* err;
  unsigned long long wait_limit;
  DropParams drop;
};

// The relay's and the epilogue's threads, once per block.
__device__ __forceinline__ void epi_barrier() {
  asm volatile("barrier.cta.sync 1, %0;" ::"n"(kEpiWarps * 32 + 32) : "memory");
}

__device__ __forceinline__ void tile_at(const TileParams& p, int t, int32_t& m0, int32_t& nt) {
  const int per_group = p.group_m * p.n_tiles;
  const int group = t / per_group, first = group * p.group_m;
  const int gsize = min(p.group_m, p.m_tiles - first);
  const int idx = t - group * per_group;
  nt = idx / gsize;
  m0 = (first + idx % gsize) * 128;
}

// MASK: the LoRA blocks are masked by dropout at (t, n); otherwise they are added like any other
// block, with scale one.
template <int BN, bool TR, bool MASK, bool SPLIT>
__global__ void __launch_bounds__(kTileThreads, 1) k_block_tile(const __grid_constant__ TileParams p) {
  using C = TileCfg<BN>;
  constexpr int kStages = C::kStages;
  constexpr int kSlots = C::kSlots;
  // An odd number of stages and two MMA warps: a stage has a barrier for either, since a warp that
  // has not seen a barrier's last phase (the other warp's load) cannot tell it from its own.
  constexpr int kFull = 2 * kStages;
  static_assert(kStages % 2 == 1 && kSlots % 2 == 0, "a barrier belongs to one MMA warp");
  constexpr int HC = BN / 2;   // columns of an epilogue warp
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* boxes = base + kStages * C::kStageBytes;
  float* scales = reinterpret_cast<float*>(boxes + C::kEpiBytes);   // [2 kSlots][2][128]
  uint64_t* full_bar = reinterpret_cast<uint64_t*>(boxes + C::kEpiBytes + C::kScaleBytes);
  uint64_t* empty_bar = full_bar + kFull;
  uint64_t* acc_full = empty_bar + kStages;   // [kSlots]
  uint64_t* acc_empty = acc_full + kSlots;    // [kSlots]
  uint64_t* mma_done = acc_empty + kSlots;    // [2]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mma_done + 2);
  uint32_t* failed = tmem_slot + 1;           // the relay gave up waiting
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    *failed = 0;
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full_bar[s], 1);
      mbar_init(&full_bar[s + kStages], 1);
      mbar_init(&empty_bar[s], 1);
    }
    for (int b = 0; b < kSlots; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], kEpiWarps);
    }
    mbar_init(&mma_done[0], 1);
    mbar_init(&mma_done[1], 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  if (warp == 1) tmem_alloc(tmem_slot, 512);
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = *tmem_slot;
  grid_dep_sync();

  // this CTA's blocks of its tiles: all, or a share of them
  const int nblk = p.nk + p.n_lora, splits = SPLIT ? p.splits : 1;
  const int split = SPLIT ? (int)blockIdx.x % splits : 0;
  const int kb0 = SPLIT ? nblk * split / splits : 0, kb1 = SPLIT ? nblk * (split + 1) / splits : nblk;
  if (warp < 4) {
    // the epilogue takes the registers that these four warps leave
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kIssueRegs));
    if (warp == 0) {
      if (lane == 0) {
        int g = 0;
        bool ok = true;
        for (int t = (int)blockIdx.x / splits; t < p.total && ok; t += (int)gridDim.x / splits) {
          int32_t m0, nt;
          tile_at(p, t, m0, nt);
          const int n0 = nt * BN;
          for (int kb = kb0; kb < kb1; ++kb, ++g) {
            const int s = g % kStages;
            const uint32_t ph = (uint32_t)(g / kStages) & 1u;
            if (g >= kStages && !mbar_wait_for(&empty_bar[s], ph ^ 1u, 1u, p.err, p.wait_limit)) {
              ok = false;
              break;
            }
            uint8_t* sa = base + s * C::kStageBytes;
            uint8_t* sb = sa + kTileBytes;
            uint64_t* full = &full_bar[g % kFull];
            mbar_expect_tx(full, C::kStageBytes);
            if (kb < p.nk) {
              tma_load_2d(sa, &p.ta, full, kb * kBlk, m0);
              if constexpr (TR) {
#pragma unroll
                for (int c = 0; c < BN / 128; ++c)
                  tma_load_2d(sb + c * kTileBytes, &p.tb, full, n0 + c * 128, kb * kBlk);
              } else {
                tma_load_2d(sb, &p.tb, full, kb * kBlk, n0);
              }
            } else {
              tma_load_2d(sa, &p.tp, full, (kb - p.nk) * 32, m0);
              tma_load_2d(sb, &p.tq, full, (kb - p.nk) * 32, n0);
            }
          }
        }
        // every issued load has landed before the CTA may exit
        for (int gg = (g > kStages ? g - kStages : 0); gg < g; ++gg)
          if (!mbar_wait(&full_bar[gg % kFull], (uint32_t)(gg / kFull) & 1u, 1u, p.err)) break;
      }
    } else if (warp <= 2) {
      if (lane == 0) {
        constexpr uint32_t id8 = idesc(kFmtE4M3, 128, BN, false, TR);
        constexpr uint32_t id32 = idesc(kFmtTF32, 128, BN);
        int j = 0;
        bool ok = true;
        for (int t = (int)blockIdx.x / splits; t < p.total && ok; t += (int)gridDim.x / splits) {
          for (int kb = kb0; kb < kb1; ++kb, ++j) {
            if ((j & 1) != warp - 1) continue;   // the other MMA warp's block
            const int b = j % kSlots, use = j / kSlots, s = j % kStages;
            if (!mbar_wait_for(&full_bar[j % kFull], (uint32_t)(j / kFull) & 1u, 2u, p.err, p.wait_limit) ||
                (use >= 1 &&
                 !mbar_wait_for(&acc_empty[b], (uint32_t)(use - 1) & 1u, 2u, p.err, p.wait_limit))) {
              ok = false;
              break;
            }
            fence_after();
            const uint32_t d = tmem + (uint32_t)(BN * b);
            const uint32_t sa = smem_u32(base + s * C::kStageBytes);
            const uint64_t da = smem_desc_sw128(sa);
            if (kb < p.nk) {
              // K = 32 codes per instruction: 32 bytes along a K-major row, four 8-row groups
              // of the MN-major tile
              const uint64_t db = TR ? smem_desc_sw128_mn(sa + kTileBytes, kTileBytes)
                                     : smem_desc_sw128(sa + kTileBytes);
#pragma unroll
              for (int k = 0; k < 4; ++k)
                umma_f8(d, da + 2 * k, db + (TR ? 256 : 2) * k, id8, k > 0 ? 1u : 0u);
            } else {
              const uint64_t db = smem_desc_sw128(sa + kTileBytes);
#pragma unroll
              for (int k = 0; k < 4; ++k)
                umma_tf32(d, da + 2 * k, db + 2 * k, id32, k > 0 ? 1u : 0u);
            }
            umma_commit(&empty_bar[s]);
            umma_commit(&acc_full[b]);
          }
        }
        umma_commit(&mma_done[warp - 1]);
        mbar_wait(&mma_done[warp - 1], 0u, 2u, p.err);
      }
    } else {
      // Block j's scale products go to buffer j % (2 kSlots), whose last reader (block j - 2 kSlots)
      // had released its accumulator before block j - kSlots, already passed on, was begun.
      int j = 0;
      bool ok = true;
      for (int t = (int)blockIdx.x / splits; t < p.total; t += (int)gridDim.x / splits) {
        int32_t m0, nt;
        tile_at(p, t, m0, nt);
        const float4* sx = reinterpret_cast<const float4*>(p.sx + m0) + lane;   // 4 rows per lane
        const int64_t nb0 = (int64_t)nt * BN / kBlk, nb1 = nb0 * kBlk + HC < p.N ? ((int64_t)nt * BN + HC) / kBlk : nb0;
        const int kf = kb0 < p.nk ? kb0 : 0;
        float4 x = __ldg(sx + kf * (p.ld_sx / 4));
        float w0 = __ldg(p.sw + nb0 * p.sw_n + kf * p.sw_k), w1 = __ldg(p.sw + nb1 * p.sw_n + kf * p.sw_k);
        for (int kb = kb0; kb < kb1; ++kb, ++j) {
          float4* dst = reinterpret_cast<float4*>(scales + (j % (2 * kSlots)) * 256) + lane;
          if (kb < p.nk) {
            dst[0] = make_float4(x.x * w0, x.y * w0, x.z * w0, x.w * w0);
            dst[32] = make_float4(x.x * w1, x.y * w1, x.z * w1, x.w * w1);
          } else {   // the LoRA term
            dst[0] = dst[32] = make_float4(1.f, 1.f, 1.f, 1.f);
          }
          if (kb + 1 < p.nk) {   // the next block's scales arrive while this one is awaited
            x = __ldg(sx + (kb + 1) * (p.ld_sx / 4));
            w0 = __ldg(p.sw + nb0 * p.sw_n + (kb + 1) * p.sw_k);
            w1 = __ldg(p.sw + nb1 * p.sw_n + (kb + 1) * p.sw_k);
          }
          if (ok) {
            ok = __all_sync(0xffffffffu, mbar_wait_for(&acc_full[j % kSlots], (uint32_t)(j / kSlots) & 1u,
                                                       4u, p.err, p.wait_limit));
            if (!ok && lane == 0) *reinterpret_cast<volatile uint32_t*>(failed) = 1u;
          }
          fence_after();
          fence_before();
          __syncwarp();
          // both sides wait, so that the relay never runs ahead of the epilogue (after a timeout
          // neither waits for the tensor cores any more: the tile runs out on invalid sums)
          epi_barrier();
        }
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kEpiRegs));
    const int q = warp & 3, h = (warp - 4) >> 2;
    uint8_t* box0 = boxes + (warp - 4) * (BN / 64) * kBox;
    int j = 0;
    for (int t = (int)blockIdx.x / splits; t < p.total; t += (int)gridDim.x / splits) {
      int32_t m0, nt;
      tile_at(p, t, m0, nt);
      const int64_t n0 = (int64_t)nt * BN + h * HC;
      // the row's mask, a bit per column: hashed while the first blocks' MMAs run and no accumulator
      // is live (in the LoRA blocks it spilled, and cost twice: 8192 x 4096 x 4096, rank 64,
      // forward and backward 612 us against 582)
      uint32_t keep[MASK ? HC / 32 : 1];
      if constexpr (MASK) {
        const int64_t m = m0 + q * 32 + lane;
        const DropRow drow = drop_row(p.drop, m < p.T ? m : 0);
#pragma unroll
        for (int c = 0; c < HC / 32; ++c) {
          keep[c] = 0u;
#pragma unroll 4
          for (int i = 0; i < 32; ++i)
            keep[c] |= (uint32_t)drop_keep_at(drow, p.drop.tau, n0 + c * 32 + i) << i;
        }
      }
      uint64_t acc[HC / 2];
#pragma unroll
      for (int c = 0; c < HC / 2; ++c) acc[c] = 0;
      const uint32_t tcol = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(h * HC);
      const int plain = MASK && kb1 > p.nk ? p.nk : kb1;
      for (int kb = kb0; kb < plain; ++kb, ++j) {
        epi_barrier();
        fence_after();
        const float sf = scales[(j % (2 * kSlots)) * 256 + h * 128 + q * 32 + lane];
        const uint64_t s = pack2(sf, sf);
        const uint32_t d = tcol + (uint32_t)(BN * (j % kSlots));
        uint32_t r0[16], r1[16];
        tmem_ldc(d, r0);
#pragma unroll
        for (int c = 0; c < HC / 16; c += 2) {
          tmem_wait_ld(r0);
          tmem_ldc(d + (uint32_t)((c + 1) * 16), r1);
#pragma unroll
          for (int i = 0; i < 8; ++i) fma2(acc[c * 8 + i], s, r0[2 * i], r0[2 * i + 1]);
          tmem_wait_ld(r1);
          if (c + 2 < HC / 16) {
            tmem_ldc(d + (uint32_t)((c + 2) * 16), r0);
          } else {   // this warp has read its part of the buffer
            fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&acc_empty[j % kSlots]);
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) fma2(acc[(c + 1) * 8 + i], s, r1[2 * i], r1[2 * i + 1]);
        }
      }
      if constexpr (MASK) {
        for (int kb = kb0 > p.nk ? kb0 : p.nk; kb < kb1; ++kb, ++j) {
          epi_barrier();
          fence_after();
          const uint32_t d = tcol + (uint32_t)(BN * (j % kSlots));
#pragma unroll
          for (int c = 0; c < HC / 16; ++c) {
            uint32_t r[16];
            tmem_ldc(d + (uint32_t)(c * 16), r);
            tmem_wait_ld(r);
#pragma unroll
            for (int i = 0; i < 16; ++i)
              if (!(keep[c / 2] >> (16 * (c & 1) + i) & 1u)) r[i] = 0u;
#pragma unroll
            for (int i = 0; i < 8; ++i) fma2(acc[c * 8 + i], pack2(1.f, 1.f), r[2 * i], r[2 * i + 1]);
          }
          fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&acc_empty[j % kSlots]);
        }
      }
      if constexpr (SPLIT) {   // the partial tile [BN][128], over the stages that every MMA has read
        float* part = reinterpret_cast<float*>(base) + h * HC * 128 + q * 32 + lane;
        // after a wait that ran out a NaN, which no sum with it hides
        const bool lost = *reinterpret_cast<volatile uint32_t*>(failed) != 0u;
#pragma unroll
        for (int c = 0; c < HC / 2; ++c) {
          float a, b;
          unpack2(lost ? kNan2 : acc[c], a, b);
          part[2 * c * 128] = a;
          part[(2 * c + 1) * 128] = b;
        }
        break;
      }
      // rows past T and columns past N are clipped by the bulk store
      const int32_t wrow = m0 + q * 32;
      if (wrow < p.T && *reinterpret_cast<volatile uint32_t*>(failed) == 0u) {
        if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");   // the last tile's
        __syncwarp();
#pragma unroll
        for (int c = 0; c < HC / 32; ++c) {
          uint8_t* box = box0 + c * kBox;
#pragma unroll
          for (int gq = 0; gq < 4; ++gq) {
            float v[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) unpack2(acc[c * 16 + gq * 4 + i], v[2 * i], v[2 * i + 1]);
            store8(reinterpret_cast<__nv_bfloat16*>(box + lane * 64 + ((gq ^ ((lane >> 1) & 3)) << 4)), v);
          }
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) {
#pragma unroll
          for (int c = 0; c < HC / 32; ++c)
            if (n0 + c * 32 < p.N) tma_store_2d(&p.to, box0 + c * kBox, (int32_t)(n0 + c * 32), wrow);
          asm volatile("cp.async.bulk.commit_group;" ::: "memory");
        }
      }
    }
    if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    __syncwarp();
    fence_before();
  }
  if constexpr (SPLIT) {
    __syncwarp();
    // The partial tiles meet in distributed shared memory: this CTA adds an S-th of the tile, 4 rows
    // x 8 columns per thread, in split order, so that reruns are bitwise equal.
    cluster_sync_all();
    if (warp >= 4 && *reinterpret_cast<volatile uint32_t*>(failed) == 0u) {
      int32_t m0, nt;
      tile_at(p, (int)blockIdx.x / splits, m0, nt);
      const float* part = reinterpret_cast<const float*>(base);
      for (int e = split * (kEpiWarps * 32) + (int)threadIdx.x - 128; e < 32 * (BN / 8);
           e += p.splits * (kEpiWarps * 32)) {
        // 8 lanes along the rows, so that their loads cover the banks once; 4 along the columns
        const int r = (e >> 5) % 4 * 32 + (e & 7) * 4, c = ((e >> 5) / 4 * 4 + (e >> 3 & 3)) * 8;
        const int64_t n = (int64_t)nt * BN + c;
        if (m0 + r >= p.T || n >= p.N) continue;
        float4 f[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = dsmem_ld4(part + (c + i) * 128 + r, 0);
        for (int k = 1; k < p.splits; ++k) {
          float4 o[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) o[i] = dsmem_ld4(part + (c + i) * 128 + r, (uint32_t)k);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            f[i].x += o[i].x; f[i].y += o[i].y; f[i].z += o[i].z; f[i].w += o[i].w;
          }
        }
        float v[4][8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          v[0][i] = f[i].x; v[1][i] = f[i].y; v[2][i] = f[i].z; v[3][i] = f[i].w;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (m0 + r + i < p.T) store8(p.Y + (int64_t)(m0 + r + i) * p.N + n, v[i]);
      }
    }
    __syncwarp();
    cluster_sync_all();   // the peers have read this CTA's shared memory
  }
  __syncthreads();
  if (warp == 1) {
    fence_after();
    tmem_dealloc(tmem, 512);
  }
}

constexpr int kMaxSplits = 8;   // portable cluster size

template <int BN, bool TR, bool MASK, bool SPLIT>
cudaError_t launch_tile(const TileParams& prm, cudaStream_t st) {
  static std::atomic<uint64_t> set{0};
  const cudaError_t e = once_on_device(set, [] {
    cudaError_t err = cudaFuncSetAttribute(k_block_tile<BN, TR, MASK, SPLIT>,
                                           cudaFuncAttributeMaxDynamicSharedMemorySize, TileCfg<BN>::kSmem);
    // a build that launches with fewer registers would wait for them forever
    cudaFuncAttributes fa;
    if (err == cudaSuccess) err = cudaFuncGetAttributes(&fa, k_block_tile<BN, TR, MASK, SPLIT>);
    if (err == cudaSuccess && fa.numRegs != kLaunchRegs) err = cudaErrorInvalidConfiguration;
    return err;
  });
  if (e != cudaSuccess) return e;
  const int sms = sm_count();
  if constexpr (!SPLIT)
    return launch_kernel(k_block_tile<BN, TR, MASK, SPLIT>, (unsigned)(prm.total < sms ? prm.total : sms),
                         kTileThreads, TileCfg<BN>::kSmem, st, prm);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(prm.total * prm.splits));
  cfg.blockDim = dim3(kTileThreads);
  cfg.dynamicSmemBytes = TileCfg<BN>::kSmem;
  cfg.stream = st;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)prm.splits;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = add_pdl_attr(at, 1);
  return cudaLaunchKernelEx(&cfg, k_block_tile<BN, TR, MASK, SPLIT>, prm);
}

// Clusters of `splits` CTAs (one per SM) that the device holds at once (0: not known).
int resident_clusters(int splits) {
  static DeviceValues<kMaxSplits + 1> known;
  const int found = known.get(current_device(), splits, [&] {
    auto kernel = k_block_tile<128, false, false, true>;
    int n = 0;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)splits);
    cfg.blockDim = dim3(kTileThreads);
    cfg.dynamicSmemBytes = TileCfg<128>::kSmem;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)splits;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, TileCfg<128>::kSmem) != cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) {
      cudaGetLastError();
      return -1;
    }
    return n;
  });
  return found < 0 ? 0 : found;
}

cudaError_t run_tile(const BlockProductArgs& a, cudaStream_t st, int prof_kind) {
  static TileParams prm;   // large: filled per call on the host, copied into the launch
  static std::mutex mu;
  std::lock_guard<std::mutex> lk(mu);
  std::memset(&prm, 0, sizeof(prm));
  const int64_t K = a.transposed ? a.out_dim : a.in_dim, N = a.transposed ? a.in_dim : a.out_dim;
  const int sms = sm_count();
  if (sms <= 0) return cudaErrorInvalidDevice;
  const int64_t mt = (a.T + 127) / 128;
  // rounds of tiles times a K-block's time: 0.48 us for 128 x 256, 0.37 us for 128 x 128 (the
  // smaller tile reads as many bytes of shared memory per output, and hands over twice as often)
  const int64_t t128 = mt * ((N + 127) / 128);
  const int64_t r256 = (mt * ((N + 255) / 256) + sms - 1) / sms;
  const int64_t r128 = (t128 + sms - 1) / sms;
  const int bn = 37 * r128 < 48 * r256 ? 128 : 256;
  // Few tiles: a cluster shares each one's blocks. A round of 128 x 128 tiles takes 0.31 us per block
  // then, S shares cost 1.6 + 0.7 S us for meeting (us with S = 1 / 2 / 3 / 4 / 6 / 8: 300 tokens 14336 ->
  // 512 44.0 / 27.0 / 22.2 / 19.9 / 18.1 / 17.8; 129 tokens 9728 -> 2560 30.9 / 20.8 / 18.8; 129 tokens
  // 2560 -> 2560 11.9 / 11.3 / 10.7; 512 tokens 1024 -> 1024 7.3 / 8.7). Only as long as every cluster
  // is resident at once (300 tokens 2560 -> 1024, 24 clusters: 10.9 with 4, 17.0 with 6). Halves of
  // a 128 x 256 tile never paid: its partial sums are twice as large.
  int splits = 1;
  if (bn == 128 && r128 == 1) {
    const int64_t n = (K + kBlk - 1) / kBlk + (a.p ? (a.rank + 31) / 32 : 0);
    int64_t best = 31 * n;
    for (int s = 2; s <= kMaxSplits && s <= n && t128 * s <= sms; ++s) {
      const int64_t us = 31 * ((n + s - 1) / s) + 160 + 70 * s;
      if (us < best && t128 <= resident_clusters(s)) {
        best = us;
        splits = s;
      }
    }
  }
  const CUtensorMapDataType u8 = CU_TENSOR_MAP_DATA_TYPE_UINT8;
  if (!make_map_2d(&prm.ta, a.codes, u8, 1, K, a.T, K, 128, 128) ||
      !make_map_2d(&prm.tb, a.W8, u8, 1, a.in_dim, a.out_dim, a.in_dim, 128, a.transposed ? 128 : bn) ||
      !make_map_2d(&prm.to, a.Y, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, N, a.T, N, 32, 32))
    return cudaErrorInvalidValue;
  if (a.p) {
    const CUtensorMapDataType f32 = CU_TENSOR_MAP_DATA_TYPE_FLOAT32;
    if (!make_map_2d(&prm.tp, a.p, f32, 4, a.rank, a.T, a.rank, 32, 128) ||
        !make_map_2d(&prm.tq, a.q, f32, 4, a.rank, N, a.rank, 32, bn))
      return cudaErrorInvalidValue;
    prm.n_lora = (a.rank + 31) / 32;
    prm.drop = a.drop;
  }
  const int64_t ib = (a.in_dim + kBlk - 1) / kBlk;
  prm.sx = a.scales; prm.ld_sx = a.ld_scales;
  prm.sw = a.sw;
  prm.sw_n = a.transposed ? 1 : ib;
  prm.sw_k = a.transposed ? ib : 1;
  prm.T = a.T; prm.N = N;
  prm.nk = (int32_t)((K + kBlk - 1) / kBlk);
  prm.n_tiles = (int32_t)((N + bn - 1) / bn);
  prm.m_tiles = (int32_t)mt;
  prm.group_m = prm.n_tiles > 16 ? 32 : 1;
  if ((int64_t)prm.n_tiles * mt > INT32_MAX) return cudaErrorInvalidValue;
  prm.total = (int32_t)(prm.n_tiles * mt);
  prm.splits = splits;
  prm.Y = static_cast<__nv_bfloat16*>(a.Y);
  prm.err = error_word();
  if (!prm.err) return cudaErrorInvalidDevice;
  prm.wait_limit = tc_wait_limit();
  prof_begin(prof_kind, st);
  cudaError_t e;
  const bool mask = prm.n_lora > 0 && prm.drop.enabled;
  if (mask && !a.transposed) return cudaErrorInvalidValue;   // only the input gradient is masked
  if (splits > 1)
    e = mask ? launch_tile<128, true, true, true>(prm, st)
             : a.transposed ? launch_tile<128, true, false, true>(prm, st) : launch_tile<128, false, false, true>(prm, st);
  else if (bn == 256)
    e = mask ? launch_tile<256, true, true, false>(prm, st)
             : a.transposed ? launch_tile<256, true, false, false>(prm, st) : launch_tile<256, false, false, false>(prm, st);
  else
    e = mask ? launch_tile<128, true, true, false>(prm, st)
             : a.transposed ? launch_tile<128, true, false, false>(prm, st) : launch_tile<128, false, false, false>(prm, st);
  if (e != cudaSuccess) return e;
  prof_end(prof_kind, st);
  return cudaGetLastError();
}

// ---- 128 outputs x NT tokens, the contraction split over a cluster -----------------------------
// Warps: 0 .. 3 epilogue (warp w drains TMEM lanes 32 w ..: a thread holds one output row and NT
// accumulators), 4 TMA, 5 TMEM allocation and MMA. Split s of S takes an even share of the
// K-blocks; the S partial tiles meet in distributed shared memory, each CTA adding an S-th of the
// tile in split order, so that reruns are bitwise equal.
//
// The weight's bytes bound it, so it wants every SM to stream all the time: short shares (at least
// two K-blocks) in several small CTAs per SM, all resident at once.
//
// FUSED (a few tokens): the epilogue warps quantise the CTA's share of X themselves while the
// weight is on its way, and the call is one launch.
constexpr int kStreamThreads = 192;
constexpr int kFusedTokens = 8;    // tokens of the fused form
constexpr int kFusedBlocks = 8;    // K-blocks of a CTA's share in it

template <int NT, bool FUSED>
struct StreamCfg {
  static constexpr int kXTile = NT * 128;
  static constexpr int kStageBytes = kTileBytes + (FUSED ? 0 : kXTile);
  static constexpr int kScaleBytes = FUSED ? 0 : NT * 4;
  static constexpr int kXBytes = FUSED ? kFusedBlocks * (kXTile + NT * 4) : 0;   // the share of X
  static constexpr int kTileF32 = 128 * NT * 4;   // the partial tile, over the drained stages
  static constexpr int kPerSm = FUSED ? 3 : NT == 16 ? 4 : NT == 32 ? 3 : 2;
  static constexpr int kStages = NT == 64 ? 4 : 3;
  static constexpr int kSmem = kStages * (kStageBytes + kScaleBytes) + kXBytes + 512 + 1024;
  static constexpr uint32_t kCols = 2 * NT < 32 ? 32 : 2 * NT;
  static_assert(kTileF32 <= kStages * kStageBytes, "partial tile fits the stages");
  static_assert(kPerSm * (kSmem + 1024) <= 228 * 1024 && kPerSm * kCols <= 512, "CTAs per SM");
};

struct StreamParams {
  CUtensorMap tw;     // W8 [out, in], box {128, 128}
  CUtensorMap tx;     // codes [T, K], box {128, NT}
  const __nv_bfloat16* X;   // fused: [T, K]
  const float* sx;
  const float* sw;
  int64_t ld_sx, sw_n, sw_k;
  int64_t T, N, K;
  int32_t nk, splits;
  __nv_bfloat16* Y;
  uint32_t* err;
  unsigned long long wait_limit;
};

template <int NT, bool TR, bool FUSED>
__global__ void __launch_bounds__(kStreamThreads, StreamCfg<NT, FUSED>::kPerSm)
    k_block_stream(const __grid_constant__ StreamParams p) {
  using C = StreamCfg<NT, FUSED>;
  constexpr int kStages = C::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* xtiles = base + kStages * C::kStageBytes;                       // fused: [block][NT][128]
  float* scales = reinterpret_cast<float*>(xtiles + (FUSED ? kFusedBlocks * C::kXTile : 0));
  uint64_t* full_bar = reinterpret_cast<uint64_t*>(scales + (FUSED ? kFusedBlocks : kStages) * NT);
  uint64_t* empty_bar = full_bar + kStages;   // MMA and epilogue have read the stage
  uint64_t* acc_full = empty_bar + kStages;   // [2]
  uint64_t* acc_empty = acc_full + 2;         // [2]
  uint64_t* mma_done = acc_empty + 2;
  uint64_t* x_ready = mma_done + 1;           // fused: the share of X is quantised
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(x_ready + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int split = (int)blockIdx.x % p.splits, nt = (int)blockIdx.x / p.splits;
  const int kb0 = (int)((int64_t)p.nk * split / p.splits);
  const int kb1 = (int)((int64_t)p.nk * (split + 1) / p.splits);
  const int nk = kb1 - kb0;
  const int32_t t0 = (int32_t)blockIdx.y * NT, n0 = nt * 128;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full_bar[s], 1);
      mbar_init(&empty_bar[s], FUSED ? 1 : 1 + 4);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], 4);
    }
    mbar_init(mma_done, 1);
    mbar_init(x_ready, 128);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  if (warp == 5) tmem_alloc(tmem_slot, C::kCols);
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = *tmem_slot;
  if constexpr (FUSED) grid_dep_sync();   // X and the weight may come from the kernel before this one

  uint64_t acc[NT / 2];
  bool lost = false;   // epilogue: a wait has run out
  if (warp == 4) {
    if (lane == 0) {
      // Not fused: the weight does not depend on the kernel before this one (the quantisation of X,
      // which itself waited for everything earlier), so the first stages' weight tiles are on their
      // way before that kernel has finished.
      auto load_w = [&](int i) {
        const int s = i % kStages;
        mbar_expect_tx(&full_bar[s], C::kStageBytes + C::kScaleBytes);
        const int32_t k0 = (kb0 + i) * kBlk;
        tma_load_2d(base + s * C::kStageBytes, &p.tw, &full_bar[s], TR ? n0 : k0, TR ? k0 : n0);
      };
      auto load_x = [&](int i) {
        if constexpr (!FUSED) {
          const int s = i % kStages;
          tma_load_2d(base + s * C::kStageBytes + kTileBytes, &p.tx, &full_bar[s], (kb0 + i) * kBlk, t0);
          asm volatile(
              "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                  smem_u32(scales + s * NT)),
              "l"(p.sx + (int64_t)(kb0 + i) * p.ld_sx + t0), "r"(C::kScaleBytes), "r"(smem_u32(&full_bar[s]))
              : "memory");
        }
      };
      const int ahead = nk < kStages ? nk : kStages;
      for (int i = 0; i < ahead; ++i) load_w(i);
      if constexpr (!FUSED) grid_dep_sync();
      int i = 0;
      for (; i < ahead; ++i) load_x(i);
      for (; i < nk; ++i) {
        if (!mbar_wait_for(&empty_bar[i % kStages], (uint32_t)(i / kStages - 1) & 1u, 1u, p.err, p.wait_limit))
          break;
        load_w(i);
        load_x(i);
      }
      // every issued load has landed before the stages are written over or the CTA exits
      for (int k = (i > kStages ? i - kStages : 0); k < i; ++k)
        if (!mbar_wait(&full_bar[k % kStages], (uint32_t)(k / kStages) & 1u, 1u, p.err)) break;
    }
  } else if (warp == 5) {
    if (lane == 0) {
      constexpr uint32_t id8 = idesc(kFmtE4M3, 128, NT, TR, false);
      bool ok = !FUSED || mbar_wait_for(x_ready, 0u, 2u, p.err, p.wait_limit);
      for (int i = 0; i < nk && ok; ++i) {
        const int b = i & 1, s = i % kStages;
        if (i >= 2 && !mbar_wait_for(&acc_empty[b], (uint32_t)((i >> 1) - 1) & 1u, 2u, p.err, p.wait_limit)) break;
        if (!mbar_wait_for(&full_bar[s], (uint32_t)(i / kStages) & 1u, 2u, p.err, p.wait_limit)) break;
        fence_after();
        const uint32_t sw = smem_u32(base + s * C::kStageBytes);
        const uint64_t da = TR ? smem_desc_sw128_mn(sw, kTileBytes) : smem_desc_sw128(sw);
        const uint64_t db = smem_desc_sw128(FUSED ? smem_u32(xtiles + i * C::kXTile) : sw + kTileBytes);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          umma_f8(tmem + (uint32_t)(b * NT), da + (TR ? 256 : 2) * k, db + 2 * k, id8, k > 0 ? 1u : 0u);
        umma_commit(&empty_bar[s]);
        umma_commit(&acc_full[b]);
      }
      umma_commit(mma_done);
      mbar_wait(mma_done, 0u, 2u, p.err);
    }
  } else {
    if constexpr (FUSED) {
      // Half-warp per (block, token), four in flight; rows past T keep what they hold (their outputs
      // are not stored).
      const int sub = threadIdx.x & 15, T = (int)p.T, units = nk * T;
      for (int u0 = threadIdx.x >> 4; u0 < units; u0 += 32) {
        uint4 v[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int u = u0 + q * 8, i = u / T, t = u - i * T;
          const int64_t col = (int64_t)(kb0 + i) * kBlk + sub * 8;
          v[q] = u < units && col < p.K ? __ldg(reinterpret_cast<const uint4*>(p.X + t * p.K + col))
                                        : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int u = u0 + q * 8, i = u / T, t = u - i * T;
          float m = amax8(v[q]);
#pragma unroll
          for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFu << (threadIdx.x & 16), m, o));
          if (u >= units) break;
          float rcp, sc;
          block_scales(m, rcp, sc);
          if (sub == 0) scales[i * NT + t] = sc;
          *reinterpret_cast<uint2*>(xtiles + i * C::kXTile + t * 128 + (((sub >> 1) ^ (t & 7)) << 4) + (sub & 1) * 8) =
              encode8(v[q], rcp);
        }
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      mbar_arrive(x_ready);
    }
#pragma unroll
    for (int c = 0; c < NT / 2; ++c) acc[c] = 0;
    const float* sw = p.sw + (int64_t)nt * p.sw_n + (int64_t)kb0 * p.sw_k;
    float w_next = nk > 0 ? __ldg(sw) : 0.f;
    constexpr int CH = NT < 32 ? NT : 32;   // columns in flight beside the accumulators
    for (int i = 0; i < nk; ++i) {
      const int b = i & 1, s = i % kStages;
      const float w = w_next;
      if (i + 1 < nk) w_next = __ldg(sw + (int64_t)(i + 1) * p.sw_k);
      // the block's scales (its stage's barrier, or the quantisation) and its sums
      bool ready;
      if constexpr (FUSED) {
        ready = i > 0 || mbar_wait_for(x_ready, 0u, 4u, p.err, p.wait_limit);
      } else {
        ready = mbar_wait_for(&full_bar[s], (uint32_t)(i / kStages) & 1u, 4u, p.err, p.wait_limit);
      }
      ready = ready && mbar_wait_for(&acc_full[b], (uint32_t)(i >> 1) & 1u, 4u, p.err, p.wait_limit);
      if (!__all_sync(0xffffffffu, ready)) {
        lost = true;
        break;
      }
      fence_after();
      const float4* sc = reinterpret_cast<const float4*>(scales + (FUSED ? i : s) * NT);
#pragma unroll
      for (int c = 0; c < NT / CH; ++c) {
        uint32_t r[CH];
        const uint32_t d = tmem + ((uint32_t)(warp * 32) << 16) + (uint32_t)(b * NT + c * CH);
        tmem_ldc(d, r);
        tmem_wait_ld(r);
#pragma unroll
        for (int v = 0; v < CH; v += 4) {
          const float4 f = sc[(c * CH + v) / 4];
          fma2(acc[(c * CH + v) / 2], pack2(f.x * w, f.y * w), r[v], r[v + 1]);
          fma2(acc[(c * CH + v) / 2 + 1], pack2(f.z * w, f.w * w), r[v + 2], r[v + 3]);
        }
      }
      fence_before();
      // the scales' reads come before the copy that overwrites them (another proxy: the arrive alone
      // does not order them, and late reads found the scales of block i + kStages)
      if constexpr (!FUSED) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&acc_empty[b]);
        if constexpr (!FUSED) mbar_arrive(&empty_bar[s]);
      }
    }
  }
  // all loads have landed and all MMAs are done: the stages become the partial tile [NT][128]
  __syncthreads();
  float* part = reinterpret_cast<float*>(base);
  if (warp < 4) {
#pragma unroll
    for (int c = 0; c < NT / 2; ++c) {
      float a, b;
      unpack2(lost ? kNan2 : acc[c], a, b);   // (no sum with a NaN hides it)
      part[2 * c * 128 + warp * 32 + lane] = a;
      part[(2 * c + 1) * 128 + warp * 32 + lane] = b;
    }
  }
  __syncwarp();
  if (p.splits > 1) cluster_sync_all();
  else __syncthreads();
  // vectors of four outputs of one token; this CTA adds an S-th of the tokens' ones
  const int rows = (int)(p.T - t0 < NT ? p.T - t0 : NT), vecs = rows * 32;
  for (int e = split * kStreamThreads + threadIdx.x; e < vecs; e += p.splits * kStreamThreads) {
    const int at = e * 4;
    const int64_t t = t0 + at / 128, n = n0 + at % 128;
    if (n >= p.N) continue;
    float4 v;
    if (p.splits > 1) {
      v = dsmem_ld4(part + at, 0);
      for (int s = 1; s < p.splits; ++s) {
        const float4 o = dsmem_ld4(part + at, (uint32_t)s);
        v.x += o.x; v.y += o.y; v.z += o.z; v.w += o.w;
      }
    } else {
      v = *reinterpret_cast<const float4*>(part + at);
    }
    store4(p.Y + t * p.N + n, &v.x);
  }
  __syncwarp();
  if (p.splits > 1) cluster_sync_all();   // the peers have read this CTA's shared memory
  else __syncthreads();
  if (warp == 5) {
    fence_after();
    tmem_dealloc(tmem, C::kCols);
  }
}

// Shares per output tile: as many as keep all CTAs resident at once, at least two K-blocks each and
// at most ten (us with 2 / 5 / 8 / 10 / 16 shares: 37 tokens 9728 -> 2560 20.5 / 12.6 / 12.7 / 12.2 /
// 17.6; 1 token 2560 -> 1024 7.5 / 5.5 / 5.4 / 4.8 / 4.8; 1 token 4096 -> 14336 14.0 / 13.2 / 16.5 /
// 16.9 / 26.3, where more than five are not resident together).
int stream_splits(int64_t tiles, int64_t nk, int per_sm) {
  int64_t s = (int64_t)per_sm * sm_count() / tiles;
  if (s > nk / 2) s = nk / 2;
  if (s > 10) s = 10;
  return s < 1 ? 1 : (int)s;
}

template <int NT, bool TR, bool FUSED>
cudaError_t launch_stream(const BlockProductArgs& a, StreamParams& prm, cudaStream_t st) {
  using C = StreamCfg<NT, FUSED>;
  static std::atomic<uint64_t> set{0};
  const cudaError_t e = once_on_device(set, [] {
    const cudaError_t err = cudaFuncSetAttribute(k_block_stream<NT, TR, FUSED>,
                                                 cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    return err != cudaSuccess ? err : cudaFuncSetAttribute(k_block_stream<NT, TR, FUSED>,
                                                           cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  });
  if (e != cudaSuccess) return e;
  if (!FUSED && !make_map_2d(&prm.tx, a.codes, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, prm.K, a.T, prm.K, 128, NT))
    return cudaErrorInvalidValue;
  const int64_t nt = (prm.N + 127) / 128, tt = (a.T + NT - 1) / NT;
  prm.splits = stream_splits(nt * tt, prm.nk, C::kPerSm);
  if (FUSED) {   // a share fits its room
    const int least = (prm.nk + kFusedBlocks - 1) / kFusedBlocks;
    if (prm.splits < least) prm.splits = least;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(nt * prm.splits), (unsigned)tt);
  cfg.blockDim = dim3(kStreamThreads);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = st;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)prm.splits;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = add_pdl_attr(at, 1);
  return cudaLaunchKernelEx(&cfg, k_block_stream<NT, TR, FUSED>, prm);
}

template <int NT, bool FUSED>
cudaError_t launch_stream(const BlockProductArgs& a, StreamParams& prm, cudaStream_t st) {
  return a.transposed ? launch_stream<NT, true, FUSED>(a, prm, st) : launch_stream<NT, false, FUSED>(a, prm, st);
}

cudaError_t run_stream(const BlockProductArgs& a, bool fused, cudaStream_t st, int prof_kind) {
  StreamParams prm;
  std::memset(&prm, 0, sizeof(prm));
  if (!make_map_2d(&prm.tw, a.W8, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, a.in_dim, a.out_dim, a.in_dim, 128, 128))
    return cudaErrorInvalidValue;
  const int64_t ib = (a.in_dim + kBlk - 1) / kBlk;
  prm.K = a.transposed ? a.out_dim : a.in_dim;
  prm.X = static_cast<const __nv_bfloat16*>(a.X);
  prm.sx = a.scales; prm.ld_sx = a.ld_scales; prm.sw = a.sw;
  prm.sw_n = a.transposed ? 1 : ib;
  prm.sw_k = a.transposed ? ib : 1;
  prm.T = a.T;
  prm.N = a.transposed ? a.in_dim : a.out_dim;
  prm.nk = (int32_t)((prm.K + kBlk - 1) / kBlk);
  prm.Y = static_cast<__nv_bfloat16*>(a.Y);
  prm.err = error_word();
  if (!prm.err || sm_count() <= 0) return cudaErrorInvalidDevice;
  prm.wait_limit = tc_wait_limit();
  prof_begin(prof_kind, st);
  cudaError_t e;
  if (fused) e = launch_stream<16, true>(a, prm, st);
  else if (a.T <= 16) e = launch_stream<16, false>(a, prm, st);
  else if (a.T <= 32) e = launch_stream<32, false>(a, prm, st);
  else e = launch_stream<64, false>(a, prm, st);   // (two 64-token tiles beat one of 128, whose
                                                   // accumulators do not fit the registers)
  if (e != cudaSuccess) return e;
  prof_end(prof_kind, st);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_block_gemm(const BlockProductArgs& a, cudaStream_t st, int prof_kind) {
  if (a.T <= 128 && !a.p) return run_stream(a, false, st, prof_kind);
  return run_tile(a, st, prof_kind);
}

cudaError_t launch_block_product(const BlockProductArgs& a, cudaStream_t st, int prof_kind) {
  const int64_t K = a.transposed ? a.out_dim : a.in_dim;
  // One launch for a few tokens and a weight that streams in a few microseconds (1 token: 2560 ->
  // 1024 4.0 us against 4.8, 4096 -> 4096 6.5 against 7.8); a larger one gains more from its loads
  // starting ahead of the quantisation (4096 -> 14336 15.5 against 13.2).
  if (a.T <= kFusedTokens && !a.p && K <= 10 * kFusedBlocks * kBlk && a.in_dim * a.out_dim <= (32 << 20))
    return run_stream(a, true, st, prof_kind);
  cudaError_t e = launch_block_quant(a.X, a.T, K, a.codes, a.scales, 1, a.ld_scales, st);
  return e != cudaSuccess ? e : launch_block_gemm(a, st, prof_kind);
}

}  // namespace lora
