// Causal attention over packed sequences: the plan of a batch's tiles and the forward pass.
//
//   S = Q K^T (tcgen05, tiles of 128 x 128),  P = exp2(c S - m),  l = sum P,  O = (P V) / l
//   with c = scale log2(e) and a running reference m for each row
//
// A work item is two tiles of 128 query rows that read the same keys: two heads of a group, or, where a
// group's heads do not pair up, two neighbouring tiles of one head. The tensor cores work on one tile
// while the softmax of the other runs: per 128 keys they take S and P V of both tiles, 4 x 512 cycles at
// head_dim 128, and each tile's 128 threads (one row each) have the other tile's 1024 to turn S into P.
// P goes back to tensor memory over S, so that P V takes it from there.
//
// The reference m follows the running maximum only where that has grown by more than 8 (a factor 256 in P,
// which bf16 and the fp32 sums hold as well): most rows rescale O once or twice, not with every tile.
//
// CTA layout (384 threads): warps 0-3 and 4-7 softmax, rescale and epilogue of tile 0 and 1; warp 8 loads
// (TMA); warp 9 issues the products; warp 10 zeroes rows behind a sequence (11 fills their warpgroup, which hands
// its registers to the softmax).
// Every wait is bounded; a warp whose wait ran out stops, and no later
// warp sees its part arrive, so that outputs are stored from complete products only.
//
// Bound by the tensor cores at the power limit's clock: one sequence of 8192 tokens, 32 / 8 heads of 128, 355-373 us
// (1470 to 1550 TFLOP/s of the 1763 that a library product sustains; 330 us and the tensor cores busy for 74% of
// them where the clock holds), 32768 tokens 5.4 to 5.5 ms (1590 to 1620). 16384 tokens in 28 sequences of 66 to 1008
// take 115 to 117 us, 840 TFLOP/s of useful and 1150 to 1160 of tiles' operations: whole tiles are 1.37 times the
// useful operations, and a query tile has 3.5 key tiles between its first load and its last store, where both tiles of
// a CTA end together and leave the tensor cores the next item's first scores alone. Steps at 8192 tokens: products issued by a
// single lane's branch 481, by a whole warp 380; P in halves and three-operand maxima 369; persistent CTAs 364. Not
// kept: two issuing warps 421, half of P against the reference of the tile before 384.
#include <new>

#include "attn_common.cuh"
#include "api_util.h"

namespace lora {

namespace {

using namespace attn;

// ---- the plan ------------------------------------------------------------------------------
constexpr int kPlanThreads = 1024;

struct PlanK {
  const int32_t* start;
  int32_t n_seq;
  int64_t T;
  AttnPlan p;
};

// Inclusive scan over the block; `sh` holds kPlanThreads values.
template <typename Op>
__device__ int64_t block_scan(int64_t v, int64_t* sh, Op op) {
  const int t = threadIdx.x;
  sh[t] = v;
  __syncthreads();
  for (int o = 1; o < kPlanThreads; o <<= 1) {
    const int64_t u = t >= o ? op(sh[t - o], sh[t]) : sh[t];
    __syncthreads();
    sh[t] = u;
    __syncthreads();
  }
  return sh[t];
}

// One CTA. Sequences (clamped, in order), then for tiles of 128 and of 256 rows: how many sequences have
// an i-th tile, the place of the tiles of each index in falling order (a causal tile's work grows with its
// index), and the tiles in their places. The order among tiles of one index is not fixed; it decides when
// a tile runs, not what it computes. 11 us for up to 8 sequences of 1024 tokens, 12 for 28 of 16380 tokens in all, 12 to
// 14 for one of 8192, 100 to 135 for 3000 of 5 tokens: once for all layers of a batch.
__global__ void __launch_bounds__(kPlanThreads) k_attn_plan(const __grid_constant__ PlanK a) {
  grid_dep_sync();
  __shared__ int64_t sh[kPlanThreads];
  __shared__ int64_t carry;
  const int t = threadIdx.x;
  if (t == 0) {
    carry = 0;
    a.p.count[2] = (int)a.T;
    a.p.count[3] = a.n_seq;
  }
  __syncthreads();
  for (int64_t k0 = 0; k0 < a.n_seq; k0 += kPlanThreads) {
    const int64_t k = k0 + t;
    int64_t lo = 0, hi = 0;
    if (k < a.n_seq) {
      lo = a.start[k];
      hi = a.start[k + 1];
      lo = lo < 0 ? 0 : lo > a.T ? a.T : lo;
      hi = hi < 0 ? 0 : hi > a.T ? a.T : hi;
    }
    const int64_t before = carry;   // the furthest end of the sequences ahead
    block_scan(hi, sh, [](int64_t x, int64_t y) { return x > y ? x : y; });
    const int64_t prev = t ? sh[t - 1] : 0;
    const int64_t last = sh[kPlanThreads - 1];
    __syncthreads();
    const int64_t end = prev > before ? prev : before;
    const int64_t from = lo > end ? lo : end;
    if (k < a.n_seq) a.p.seq[k] = make_int2((int)from, (int)(hi > from ? hi - from : 0));
    if (t == 0) carry = before > last ? before : last;
    __syncthreads();
  }
  for (int w = 0; w < 2; ++w) {
    const int rows = kAttnTile << w;
    const int64_t buckets = (a.T + rows - 1) / rows;
    for (int64_t i = t; i < buckets; i += kPlanThreads) a.p.hist[i] = 0;
    __syncthreads();
    for (int64_t k = t; k < a.n_seq; k += kPlanThreads) {
      const int n = a.p.seq[k].y;
      if (n > 0) atomicAdd(a.p.hist + (n - 1) / rows, 1);
    }
    __syncthreads();
    // from the highest index down: sequences that reach it, and tiles placed ahead of it
    int64_t reach = 0, placed = 0;
    for (int64_t i0 = 0; i0 < buckets; i0 += kPlanThreads) {
      const int64_t i = buckets - 1 - (i0 + t);
      const int64_t here = i >= 0 ? a.p.hist[i] : 0;
      const auto add = [](int64_t x, int64_t y) { return x + y; };
      const int64_t n = reach + block_scan(here, sh, add);     // sequences with a tile i
      const int64_t all = sh[kPlanThreads - 1];
      __syncthreads();
      const int64_t upto = placed + block_scan(i >= 0 ? n : 0, sh, add);
      const int64_t tiles = sh[kPlanThreads - 1];
      __syncthreads();
      if (i >= 0) a.p.hist[i] = (int)(upto - n);
      reach += all;
      placed += tiles;
      __syncthreads();
    }
    if (t == 0) a.p.count[w] = (int)placed;
    __syncthreads();
    // a warp per sequence, a lane per tile
    for (int64_t k = t / 32; k < a.n_seq; k += kPlanThreads / 32) {
      const int2 s = a.p.seq[k];
      const int n = (s.y + rows - 1) / rows;
      for (int i = t % 32; i < n; i += 32) {
        const int64_t at = atomicAdd(a.p.hist + i, 1);
        if (at < a.p.most[w]) a.p.tiles[w][at] = AttnTile{s.x, s.y, i, 0};
      }
    }
    __syncthreads();
  }
}

// ---- forward -------------------------------------------------------------------------------
constexpr float kRescale = 8.f;   // growth of a row's maximum, in powers of two, that rescales O

template <int D>
struct FwdCfg {
  static constexpr int kTile = Tile<D>::kBytes;
  static constexpr int kStages = D == 128 ? 4 : 8;   // K and V tiles in flight or in use
  static constexpr int kStage = 32 * 64 * 2;         // a warp's rows on their way out, 64 columns at a time
  static constexpr int kSmem = (2 + kStages) * kTile + 8 * kStage + 1024 /*barriers*/ + 1024 /*alignment*/;
  static_assert(kSmem <= 227 * 1024, "shared memory per CTA");
  static constexpr uint32_t kIdS = idesc(kFmtBF16, 128, 128);
  static constexpr uint32_t kIdO = idesc(kFmtBF16, 128, D, false, true);
  // tensor memory: S (and P over it) of both tiles, O of both
  static constexpr uint32_t kS = 0, kO = 256;
};

struct FwdK {
  CUtensorMap tq, tk, tv, to;
  PlanRef plan;
  int32_t groups;        // items of a tile of the list
  int32_t by_heads;      // two heads of a 128-row tile, or two 128-row tiles of a head
  int32_t per;           // query heads of a key / value head
  float c;               // scale log2(e)
  int64_t T, ld_o;
  __nv_bfloat16* O;
  float* lse;
  uint32_t* err;
  unsigned long long limit;
};

template <int D>
__global__ void __launch_bounds__(SplitFwd::kThreads, 1) k_attn_fwd(const __grid_constant__ FwdK p) {
  using C = FwdCfg<D>;
  using Tl = Tile<D>;
  constexpr int ST = C::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sq = base;
  uint8_t* ring = base + 2 * C::kTile;
  uint8_t* stages = ring + ST * C::kTile;
  uint64_t* full = reinterpret_cast<uint64_t*>(stages + 8 * C::kStage);
  uint64_t* empty = full + ST;
  uint64_t* q_full = empty + ST;     // [2]
  uint64_t* q_empty = q_full + 2;    // [2] the last S of a tile is complete
  uint64_t* s_full = q_empty + 2;    // [2] S of a tile is complete
  uint64_t* p_full = s_full + 2;     // [2][2] half of a tile's P is in place, O rescaled
  uint64_t* o_full = p_full + 4;     // [2] P V is complete
  uint64_t* landed = o_full + 2;     // [ST] see Partial
  uint64_t* done = landed + ST;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
  uint32_t* ended = tmem_slot + 1;   // see Partial
  const int warp = uniform((int)threadIdx.x >> 5), lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < ST; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
      mbar_init(&landed[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&q_full[s], 1);
      mbar_init(&q_empty[s], 1);
      mbar_init(&s_full[s], 1);
      mbar_init(&p_full[2 * s], 4);
      mbar_init(&p_full[2 * s + 1], 4);
      mbar_init(&o_full[s], 1);
    }
    mbar_init(done, 1);
    *ended = 0u;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    fence_async();
  }
  if (warp == 9) tmem_alloc(tmem_slot, 512);
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = (uint32_t)uniform((int)*tmem_slot);
  grid_dep_sync();   // from here on, the earlier kernels' outputs are visible

  if (warp >= 8) SplitFwd::issue();
  AttnTile t;
  int group;
  Items items(p.plan, p.groups);
  if (warp == 8) {
    // ---- loads: Q of both tiles, then K and V tile by tile ----
    int g = 0, nq0 = 0, nq1 = 0;   // tiles of the ring, of Q
    Partial part;
    bool ok = true;
    while (ok && items.take(t, group)) {
      const Pair pr(t, group, p.by_heads);
      const int kv_col = pr.h0 / p.per * D;
      for (int j = 0; j < 2 * pr.most && ok; ++j, ++g) {
        if (j < 2 && pr.n(j)) {   // Q of tile 0 ahead of the first K, of tile 1 behind it
          const int before = j ? nq1++ : nq0++;
          if (before && !(ok = warp_wait(&q_empty[j], (uint32_t)(before - 1) & 1u, 1u, p.err, p.limit))) {
            (j ? nq1 : nq0) = before;
            break;
          }
          if (lane == 0) {
            mbar_expect_tx(&q_full[j], C::kTile);
            Tl::load(sq + j * C::kTile, &p.tq, &q_full[j], pr.h(j) * D, t.row0 + pr.qi(j) * kRows);
          }
        }
        const int s = g % ST, kt = j >> 1;
        if (g >= ST && !(ok = warp_wait(&empty[s], (uint32_t)(g / ST - 1) & 1u, 1u, p.err, p.limit))) break;
        uint8_t* dst = ring + s * C::kTile;
        const int rows = t.len - kt * kRows;   // of the sequence from here on
        const bool some = (j & 1) && rows < kRows;   // V of the sequence's last rows
        if (lane == 0) {
          uint64_t* bar = some ? &landed[s] : &full[s];
          mbar_expect_tx(bar, C::kTile);
          Tl::load(dst, (j & 1) ? &p.tv : &p.tk, bar, kv_col, t.row0 + kt * kRows);
        }
        if (some) part.next(s);
      }
    }
    // every copy has landed before the CTA ends
    if (lane == 0) {
      *static_cast<volatile uint32_t*>(ended) = 1u + part.n;
      if (nq0) mbar_wait(&q_full[0], (uint32_t)(nq0 - 1) & 1u, 1u, p.err);
      if (nq1) mbar_wait(&q_full[1], (uint32_t)(nq1 - 1) & 1u, 1u, p.err);
      part.drain(landed, ST, p.err);
      for (int k = g > ST ? g - ST : 0; k < g; ++k)
        if (!mbar_wait(&full[k % ST], (uint32_t)(k / ST) & 1u, 1u, p.err)) break;
    }
    __syncwarp();
  } else if (warp == 9) {
    // ---- products ----
    const uint32_t one = elect_one();
    const uint32_t q0 = smem_u32(sq), rg = smem_u32(ring);
    auto wait = [&](uint64_t* b, uint32_t par) {
      const bool r = warp_wait(b, par & 1u, 2u, p.err, p.limit);
      fence_after();
      return r;
    };
    auto stage_full = [&](int g) { return wait(&full[g % ST], (uint32_t)(g / ST)); };
    auto stage_at = [&](int g) { return rg + (uint32_t)(g % ST) * C::kTile; };
    int g = 0;                                // ring tiles before key tile j's
    uint32_t i0 = 0, i1 = 0, c0 = 0, c1 = 0;  // of each tile: items and key tiles so far
    bool ok = true;
    while (ok && items.take(t, group)) {
      const Pair pr(t, group, p.by_heads);
      const int tiles = pr.n1 ? 2 : 1;
      auto score = [&](int s, int at, bool last) {   // S over the P before it
        Tl::mma_nt(tmem + C::kS + 128 * s, q0 + s * C::kTile, stage_at(at), C::kIdS, one);
        commit(&s_full[s], one);
        if (last) commit(&q_empty[s], one);
      };
      ok = stage_full(g);
#pragma unroll 1
      for (int s = 0; s < tiles && ok; ++s) {
        if (!(ok = wait(&q_full[s], s ? i1 : i0))) break;
        score(s, g, pr.n(s) == 1);
      }
      if (ok) commit(&empty[g % ST], one);
#pragma unroll 1
      for (int j = 0; j < pr.most && ok; ++j, g += 2) {
        if (!(ok = stage_full(g + 1))) break;
        bool have_k = false;
#pragma unroll 1
        for (int s = j < pr.n0 ? 0 : 1; s < tiles; ++s) {
          const uint32_t ps = tmem + C::kS + 128 * s, os = tmem + C::kO + 128 * s, c = s ? c1 : c0;
          if (!(ok = wait(&p_full[2 * s], c))) break;
          Tl::template mma_tn<128, 0, 4>(os, ps, stage_at(g + 1), C::kIdO, j > 0, one);
          if (!(ok = wait(&p_full[2 * s + 1], c))) break;
          Tl::template mma_tn<128, 4, 8>(os, ps, stage_at(g + 1), C::kIdO, true, one);
          commit(&o_full[s], one);
          if (s + 1 == tiles) commit(&empty[(g + 1) % ST], one);
          if (s) ++c1; else ++c0;
          if (j + 1 < pr.n(s)) {
            if (!have_k && !(ok = stage_full(g + 2))) break;
            have_k = true;
            score(s, g + 2, j + 2 == pr.n(s));
          }
        }
        if (ok && have_k) commit(&empty[(g + 2) % ST], one);
      }
      ++i0;
      if (pr.n1) ++i1;
    }
    // every product has completed before the tensor memory is freed
    commit(done, one);
    mbar_wait(done, 0u, 2u, p.err);
    __syncwarp();
  } else if (warp == 10) {
    // ---- zeros behind the sequences, in V ----
    Partial part;
    int g = 0;   // tiles of the ring
    while (items.take(t, group)) {
      const Pair pr(t, group, p.by_heads);
      g += 2 * pr.most;
      const int rows = t.len - (pr.most - 1) * kRows, s = (g - 1) % ST;
      if (rows < kRows && !part.pass<D>(ring + s * C::kTile, s, rows, landed, full, lane, p.err, ended, part.n)) break;
    }
  } else if (warp < 8) {
    SplitFwd::compute();
    // ---- softmax and epilogue: thread = row of tile s ----
    const int s = warp >> 2, r = threadIdx.x & 127;
    const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t ts = lanes + C::kS + 128 * s, to = lanes + C::kO + 128 * s;
    uint32_t ns = 0, no = 0;   // S's waited for, P V's before this item
    bool ok = true;
    while (ok && items.take(t, group)) {
      const Pair pr(t, group, p.by_heads);
      const int n = pr.n(s);
      if (!n) continue;
      const bool dead = pr.qi(s) * kRows + (warp & 3) * 32 >= t.len;   // all of the warp's rows lie behind the sequence
      float m = -INFINITY, l = 0.f;
      for (int j = 0; j < n; ++j) {
        if (!(ok = warp_wait(&s_full[s], ns++ & 1u, 4u, p.err, p.limit))) break;
        fence_after();
        if (dead) {   // (whatever stands there as P makes O's rows of these queries alone)
          if (lane < 2) mbar_arrive(&p_full[2 * s + lane]);
          continue;
        }
        uint32_t x[128];
#pragma unroll
        for (int k = 0; k < 4; ++k) tmem_ld32_nw(ts + 32 * k, x + 32 * k);
        tmem_wait_ld_n<128>(x);
        if (j == n - 1) {   // the tile on the diagonal: keys up to the row's own, 32 at a time beside the warp's rows
#pragma unroll
          for (int b = 0; b < 4; ++b) {
            int ahead = b - (warp & 3);   // (hidden from the compiler, which would index x by the warp)
            asm volatile("" : "+r"(ahead));
            if (ahead == 0) {
#pragma unroll
              for (int k = 0; k < 32; ++k)
                if (k > lane) x[32 * b + k] = 0xff800000u;
            } else if (ahead > 0) {
#pragma unroll
              for (int k = 0; k < 32; ++k) x[32 * b + k] = 0xff800000u;
            }
          }
        }
        float mx[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) mx[k] = __uint_as_float(x[k]);
#pragma unroll
        for (int k = 4; k < 124; k += 8)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            mx[i] = max3(mx[i], __uint_as_float(x[k + 2 * i]), __uint_as_float(x[k + 2 * i + 1]));
        const float top = max3(max3(mx[0], mx[1], mx[2]), max3(mx[3], __uint_as_float(x[124]), __uint_as_float(x[125])),
                               fmaxf(__uint_as_float(x[126]), __uint_as_float(x[127]))) * p.c;
        if (j == 0) {
          m = top;
        } else if (__any_sync(0xffffffffu, top > m + kRescale)) {
          const bool grow = top > m + kRescale;
          const float f = grow ? exp2_(m - top) : 1.f;
          if (!(ok = warp_wait(&o_full[s], (no + j - 1) & 1u, 4u, p.err, p.limit))) break;
          fence_after();
#pragma unroll
          for (int k = 0; k < D / 32; ++k) {
            uint32_t o[32];
            tmem_ld32_nw(to + 32 * k, o);
            tmem_wait_ld_n<32>(o);
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
            tmem_st32(to + 32 * k, o);
          }
          if (grow) m = top;
          l *= f;
        }
        // (a row whose scores are all -inf so far has no reference yet: P is 0)
        const float ref = m == -INFINITY ? 0.f : m;
        const f2 c2 = mk2(p.c, p.c), m2 = mk2(-ref, -ref);
        f2 sum0 = mk2(0.f, 0.f), sum1 = sum0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          uint32_t w[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const float2 e = un2(fma2(mk2(__uint_as_float(x[32 * k + 2 * i]), __uint_as_float(x[32 * k + 2 * i + 1])), c2, m2));
            const float a = exp2_(e.x), b = exp2_(e.y);
            if (i & 1) sum1 = add2(sum1, mk2(a, b));
            else sum0 = add2(sum0, mk2(a, b));
            w[i] = pack_bf16(a, b);
          }
          tmem_st16(ts + 16 * k, w);
          if (k & 1) {   // the product of half the keys begins while the other half is turned into P
            tmem_wait_st();
            fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&p_full[2 * s + (k >> 1)]);
          }
        }
        const float2 z = un2(add2(sum0, sum1));
        l += z.x + z.y;
      }
      no += n;
      if (!ok || !(ok = warp_wait(&o_full[s], (no - 1) & 1u, 4u, p.err, p.limit))) break;
      fence_after();
      const int row = pr.qi(s) * kRows + r, row0 = row - lane;
      const int64_t at = (int64_t)t.row0 + row0;
      uint8_t* stage = stages + warp * C::kStage;
#pragma unroll 1
      for (int k = 0; k < (dead ? 0 : D / 64); ++k) {
        uint32_t u[32];
        read_rows<64>(to + 64 * k, 1.f / l, u);
        rows_read(lane);   // (what was sent before)
        stage_rows<64>(stage, u, lane);
        const int col = pr.h(s) * D + 64 * k;
        if (t.len - row0 >= 32)
          send_rows(&p.to, stage, col, at, lane);
        else   // the rows behind belong to others
          write_rows<64>(stage, p.O + at * p.ld_o + col, p.ld_o, t.len - row0, lane);
      }
      if (row < t.len) p.lse[(int64_t)pr.h(s) * p.T + at + lane] = (m + log2f(l)) * kLn2;
      fence_before();   // (O has been read before the next item's first P arrives)
    }
    if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");   // rows sent have been written
    __syncwarp();
    fence_before();
  }
  __syncthreads();
  if (warp == 9) {
    fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int D>
cudaError_t fwd_launch(const AttnArgs& a, cudaStream_t st) {
  static std::atomic<uint64_t> set{0};
  cudaError_t e = once_on_device(set, [] {
    return set_up<SplitFwd>(k_attn_fwd<D>, FwdCfg<D>::kSmem);
  });
  if (e != cudaSuccess) return e;
  FwdK k{};
  if (!attn_map(&k.tq, a.Q, a.q_heads * D, a.T, a.ld_q) || !attn_map(&k.tk, a.K, a.kv_heads * D, a.T, a.ld_k) ||
      !attn_map(&k.tv, a.V, a.kv_heads * D, a.T, a.ld_v) || !attn_map(&k.to, a.O, a.q_heads * D, a.T, a.ld_o, 32))
    return cudaErrorInvalidValue;
  k.per = a.q_heads / a.kv_heads;
  k.by_heads = k.per % 2 == 0;
  const int w = k.by_heads ? 0 : 1;
  k.plan = plan_ref(a, w);
  k.groups = k.by_heads ? a.q_heads / 2 : a.q_heads;
  k.c = a.scale * kLog2e;
  k.T = a.T;
  k.ld_o = a.ld_o;
  k.O = static_cast<__nv_bfloat16*>(a.O);
  k.lse = a.lse;
  k.err = error_word();
  if (!k.err) return cudaErrorInvalidDevice;
  k.limit = tc_wait_limit();
  const int64_t most = a.plan.most[w] * k.groups;
  const int sms = sm_count();
  if (sms <= 0) return cudaErrorInvalidDevice;
  if (most > INT32_MAX) return cudaErrorInvalidValue;
  prof_begin(0, st);
  return launch_kernel(k_attn_fwd<D>, (unsigned)(most < sms ? most : sms), SplitFwd::kThreads, FwdCfg<D>::kSmem, st, k);
}

}  // namespace

bool attn_map(CUtensorMap* map, const void* ptr, int64_t cols, int64_t rows, int64_t ld, int box_rows) {
  return make_map_2d(map, ptr, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, (uint64_t)cols, (uint64_t)rows, (uint64_t)ld, 64,
                     (uint32_t)box_rows);
}

AttnPlan attn_plan(int64_t T, int32_t n_seq, void* buf) {
  AttnPlan p{};
  Carve c(buf);
  const int64_t some = n_seq < T ? n_seq : T;   // sequences that are not empty
  p.count = c.take<int32_t>(4);
  p.n_seq = n_seq;
  for (int w = 0; w < 2; ++w) {
    p.most[w] = T / (kAttnTile << w) + some;
    p.tiles[w] = c.take<AttnTile>((size_t)p.most[w]);
  }
  p.seq = c.take<int2>((size_t)n_seq);
  p.hist = c.take<int32_t>((size_t)((T + kAttnTile - 1) / kAttnTile));
  p.bytes = c.off;
  return p;
}

cudaError_t launch_attn_plan(int64_t T, int32_t n_seq, const int32_t* seq_start, const AttnPlan& plan, cudaStream_t st) {
  PlanK k{seq_start, n_seq, T, plan};
  prof_begin(0, st);
  return launch_kernel(k_attn_plan, 1, kPlanThreads, 0, st, k);
}

cudaError_t launch_attn_forward(const AttnArgs& a, cudaStream_t st) {
  return a.dim == 128 ? fwd_launch<128>(a, st) : fwd_launch<64>(a, st);
}

}  // namespace lora
