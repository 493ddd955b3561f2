// Causal attention over packed sequences, backward: delta = sum do o, then two kernels that recompute the
// scores, one for dV and dK and one for dQ.
//
//   P = exp2(c S - lse log2(e)),  dP = dO V^T,  dS = P (dP - delta)
//   dV = P^T dO,  dK = scale dS^T Q   (key tile fixed, over query tiles and the heads of its group)
//   dQ = scale dS K                   (query tile fixed, over key tiles)
//
// Five products are needed; recomputing S and dP for dQ makes seven. The alternative, dQ added up in
// global memory by the key tiles' CTAs, takes fp32 additions in a fixed order if reruns are to be equal, 64 KB of
// them per five products (25 bytes per cycle and SM into L2, whose rate for additions was not measured), and a pass
// that clears and rounds them. It was not built.
//
// dV and dK (k_attn_dkv): the scores are computed turned, S^T = K Q^T and dP^T = V dO^T, keys along the
// tensor memory's lanes, so that P^T and dS^T, written back over them in bf16, are first operands of
// P^T dO and dS^T Q as they are; a warp has 32 keys and 32 of the tile's queries. The products of one
// query tile run while the other half of its elementwise work does: S^T of the next tile under dS^T of
// this one, dP^T of the next under P^T of the next. At head_dim 128 a pair of tiles takes four products of
// 512 cycles.
//
// dQ (k_attn_dq): two query tiles over shared keys, as in the forward pass; S = Q K^T and dP = dO V^T with queries
// along the lanes. A tile's S, dP and dS share one place in tensor memory: dP goes over S once that is in registers,
// dS, in bf16, over dP, as the first operand of dS K, and the next S over dS behind that product. The elementwise work
// of one tile runs beside the products of the other.
//
// CTA layout, k_attn_dkv (640 threads): warps 0-15 elementwise (four warpgroups, 32 columns each) and epilogue, warp 16
// loads, warp 17 issues the products, warp 18 brings the queries' statistics, warp 19 zeroes rows behind a sequence.
// k_attn_dq (384 threads): as in the forward pass. Waits are bounded as there. The cluster form of k_attn_dkv reloads
// 108 (head_dim 128) and 136 bytes of spilled registers a thread, k_attn_dq at head_dim 128 20, the others none.
//
// One sequence of 8192 tokens, 32 / 8 heads of 128: 1166 to 1194 us by the clock that the power limit leaves (seven
// products: 1610 to 1650 TFLOP/s; a library product sustains 1763); alone delta takes 24 us, dV and dK 589 (1870
// TFLOP/s, tensor cores 90% busy), dQ 473 (1745, 77%). 16384 tokens in sequences of 64 to 1024: 393 to 406 us; one by
// one delta takes 40, dV and dK 183, dQ 156. The tiles' seven products are 470 GFLOP there (tiles are 1.37 times the
// useful operations), 267 us at the sustained rate.
#include "attn_common.cuh"

namespace lora {

namespace {

using namespace attn;

using Sp = SplitBwd;
constexpr int kGroups = (Sp::kThreads - 128) / 128;   // warpgroups that share a tile's columns
constexpr int kCols = 128 / kGroups;                  // columns of a thread
constexpr int kComputeWarps = 4 * kGroups, kLoadWarp = kComputeWarps, kIssueWarp = kLoadWarp + 1, kStatWarp = kLoadWarp + 2, kZeroWarp = kLoadWarp + 3;

// ---- delta ---------------------------------------------------------------------------------
// delta[h, t] = sum do o, D / 8 lanes per head of a token. Bound by memory.
template <int D>
__global__ void __launch_bounds__(256) k_attn_delta(const __nv_bfloat16* __restrict__ O,
                                                    const __nv_bfloat16* __restrict__ dO, int64_t ld, int heads,
                                                    int64_t T, float* __restrict__ delta, int32_t* ready) {
  grid_dep_sync();
  if (blockIdx.x == 0 && threadIdx.x == 0) *ready = 0;   // (the last call's readers are done)
  constexpr int G = D / 8;
  const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) / G;   // token, then head
  const int l = threadIdx.x % G;
  const int64_t t = i / heads;
  const int h = (int)(i - t * heads);
  float a[8], b[8], s = 0.f;
  if (t < T) {
    load16(O + t * ld + (int64_t)h * D + l * 8, a);
    load16(dO + t * ld + (int64_t)h * D + l * 8, b);
#pragma unroll
    for (int k = 0; k < 8; ++k) s = fmaf(a[k], b[k], s);
  }
#pragma unroll
  for (int o = G / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (t < T && l == 0) delta[(int64_t)h * T + t] = s;
}

struct BwdK {
  CUtensorMap tq, tk, tv, tdo, tdq;
  PlanRef plan;
  int32_t heads;         // dK, dV: work items of a tile
  int32_t split;         // dK, dV: CTAs of a cluster, which share a group's query heads
  int32_t groups;        // dQ: work items of a tile of the list
  int32_t by_heads;      // dQ: two heads of a 128-row tile, or two 128-row tiles of a head
  int32_t per;
  float c, scale;
  int64_t T, ld_q, ld_k, ld_v;
  const float *lse, *delta;
  int32_t* ready;        // set by k_attn_dkv once it may read delta, for k_attn_dq
  __nv_bfloat16 *dQ, *dK, *dV;
  uint32_t* err;
  unsigned long long limit;
};

// ---- dV and dK -----------------------------------------------------------------------------
template <int D>
struct DkvCfg {
  static constexpr int kTile = Tile<D>::kBytes;
  static constexpr int kQ = 3, kDo = 2;   // tiles of Q and dO in flight or in use: dO's are free earlier
  static constexpr int kBarriers = 512;
  static constexpr int kSmem = (2 + kQ + kDo) * kTile + 2 * kRows * 4 + kBarriers + 1024 /*alignment*/;
  static_assert(kSmem <= 227 * 1024, "shared memory per CTA");
  static_assert((kQ + kDo) * kTile >= 2 * kRows * D * 4, "both sums fit where Q and dO were");
  static constexpr uint32_t kIdS = idesc(kFmtBF16, 128, 128);
  static constexpr uint32_t kIdD = idesc(kFmtBF16, 128, D, false, true);
  static constexpr uint32_t kS = 0, kDp = 128, kDv = 256, kDk = 384;   // tensor memory
};

// Element (row, 4 c ..) of a [128, D] fp32 tile in shared memory, in 16-byte pieces, turned within each row so that
// 32 rows' pieces lie in different banks.
template <int D>
__device__ __forceinline__ float* sum_at(float* tile, int row, int c) {
  return tile + row * D + ((c ^ (row & (D / 4 - 1))) << 2);
}

// k_attn_dkv's wait for the kernels ahead of it. Behind it their outputs are visible, and the first CTA passes that on to
// k_attn_dq before it lets that begin (a CTA's first thread to issue the instruction counts).
__device__ __forceinline__ void dkv_dep_sync(int32_t* ready) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (threadIdx.x == 0) {
    if (blockIdx.x == 0) flag_set(ready);
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  }
}

// CL: the query heads of a group are dealt out to the `split` CTAs of a cluster, one item each, and their sums added
// up over the cluster; otherwise the CTAs are persistent over the items and take all heads of a group.
template <int D, bool CL>
__global__ void __launch_bounds__(Sp::kThreads, 1) k_attn_dkv(const __grid_constant__ BwdK p) {
  using C = DkvCfg<D>;
  using Tl = Tile<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sk = base;
  uint8_t* sv = sk + C::kTile;
  uint8_t* sq = sv + C::kTile;
  uint8_t* sdo = sq + C::kQ * C::kTile;
  float* s_lse = reinterpret_cast<float*>(sdo + C::kDo * C::kTile);   // of the query tile: -lse log2(e), -delta
  float* s_delta = s_lse + kRows;
  uint64_t* q_full = reinterpret_cast<uint64_t*>(s_delta + kRows);
  uint64_t* q_empty = q_full + C::kQ;
  uint64_t* do_full = q_empty + C::kQ;
  uint64_t* do_empty = do_full + C::kDo;
  uint64_t* k_full = do_empty + C::kDo;
  uint64_t* k_empty = k_full + 1;    // the item's last S is complete
  uint64_t* v_full = k_empty + 1;
  uint64_t* v_empty = v_full + 1;    // the item's sums have left through V's place
  uint64_t* s_full = v_empty + 1;
  uint64_t* p_full = s_full + 1;     // P^T is in place
  uint64_t* dp_full = p_full + 1;
  uint64_t* ds_full = dp_full + 1;   // dS^T is in place
  uint64_t* lse_full = ds_full + 1;
  uint64_t* lse_empty = lse_full + 1;
  uint64_t* delta_full = lse_empty + 1;
  uint64_t* delta_empty = delta_full + 1;
  uint64_t* landed_q = delta_empty + 1;       // [kQ], [kDo] see Partial
  uint64_t* landed_do = landed_q + C::kQ;
  uint64_t* all = landed_do + C::kDo;        // both sums of an item are complete
  uint64_t* done = all + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
  uint32_t* complete = tmem_slot + 1;   // CL: this CTA's sums are in shared memory
  uint32_t* ended = tmem_slot + 2;      // see Partial
  static_assert((3 * (C::kQ + C::kDo) + 14) * 8 + 12 <= C::kBarriers, "barriers");
  const int warp = uniform((int)threadIdx.x >> 5), lane = threadIdx.x & 31;
  const int rank = CL ? (int)cluster_ctarank() : 0;
  if constexpr (CL) {   // clusters behind the last item leave before they take tensor memory
    dkv_dep_sync(p.ready);
    if ((int)blockIdx.x / p.split >= p.plan.items(p.heads)) return;
  }

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kQ; ++s) {
      mbar_init(&q_full[s], 1);
      mbar_init(&q_empty[s], 1);
      mbar_init(&landed_q[s], 1);
    }
    for (int s = 0; s < C::kDo; ++s) {
      mbar_init(&do_full[s], 1);
      mbar_init(&do_empty[s], 1);
      mbar_init(&landed_do[s], 1);
    }
    mbar_init(k_full, 1);
    mbar_init(k_empty, 1);
    mbar_init(v_full, 1);
    mbar_init(v_empty, kComputeWarps);
    mbar_init(s_full, 1);
    mbar_init(p_full, kComputeWarps);
    mbar_init(dp_full, 1);
    mbar_init(ds_full, kComputeWarps);
    mbar_init(lse_full, 1);
    mbar_init(lse_empty, kComputeWarps);
    mbar_init(delta_full, 1);
    mbar_init(delta_empty, kComputeWarps);
    mbar_init(all, 1);
    mbar_init(done, 1);
    *complete = 1u;
    *ended = 0u;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    fence_async();
  }
  if (warp == kIssueWarp) tmem_alloc(tmem_slot, 512);
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = (uint32_t)uniform((int)*tmem_slot);
  if constexpr (!CL) dkv_dep_sync(p.ready);   // from here on, the earlier kernels' outputs are visible

  if (warp >= kComputeWarps) Sp::issue();
  AttnTile t{};
  int hk = 0;
  Items items(p.plan, p.heads, CL ? p.split : 1);
  const int mine = p.per / (CL ? p.split : 1);   // query heads of an item in this CTA
  // An item: key tile j of nb, its query tiles j .. nb - 1 under each of its query heads, head by head.
  struct Span {
    int nb, j, nq, n, h0;
    __device__ Span(const AttnTile& t, int hk, int per, int mine, int rank)
        : nb((t.len + kRows - 1) / kRows), j(nb - 1 - t.index), nq(t.index + 1), n(nq * mine), h0(hk * per + rank * mine) {}
  };
  if (warp == kLoadWarp) {
    // ---- loads ----
    int nk = 0, nv = 0, nqs = 0, ndo = 0;   // tiles asked for
    Partial part_q, part_do;
    bool ok = true;
    auto fetch = [&](uint8_t* tiles, int s, const CUtensorMap* map, uint64_t* full, uint64_t* landed, Partial& part, int col, int qi) {
      const bool some = t.len - qi * kRows < kRows;   // the sequence's last rows
      if (lane == 0) {
        uint64_t* bar = some ? &landed[s] : &full[s];
        mbar_expect_tx(bar, C::kTile);
        Tl::load(tiles + s * C::kTile, map, bar, col, t.row0 + qi * kRows);
      }
      if (some) part.next(s);
    };
    auto keys = [&](uint8_t* dst, const CUtensorMap* map, uint64_t* full, uint64_t* empty, int& n, int j) {
      if (n && !warp_wait(empty, (uint32_t)(n - 1) & 1u, 1u, p.err, p.limit)) return false;
      ++n;
      if (lane == 0) {
        mbar_expect_tx(full, C::kTile);
        Tl::load(dst, map, full, hk * D, t.row0 + j * kRows);
      }
      return true;
    };
    while (ok && items.take(t, hk)) {
      const Span sp(t, hk, p.per, mine, rank);
      if (!(ok = keys(sk, &p.tk, k_full, k_empty, nk, sp.j))) break;
      int qi = sp.j, h = sp.h0;
      for (int it = 0; it < sp.n; ++it) {
        const int a = nqs % C::kQ, b = ndo % C::kDo, col = h * D;
        if (nqs >= C::kQ && !(ok = warp_wait(&q_empty[a], (uint32_t)(nqs / C::kQ - 1) & 1u, 1u, p.err, p.limit))) break;
        ++nqs;
        fetch(sq, a, &p.tq, q_full, landed_q, part_q, col, qi);
        if (it == 0 && !(ok = keys(sv, &p.tv, v_full, v_empty, nv, sp.j))) break;
        if (ndo >= C::kDo && !(ok = warp_wait(&do_empty[b], (uint32_t)(ndo / C::kDo - 1) & 1u, 1u, p.err, p.limit))) break;
        ++ndo;
        fetch(sdo, b, &p.tdo, do_full, landed_do, part_do, col, qi);
        if (++qi == sp.nb) {
          qi = sp.j;
          ++h;
        }
      }
    }
    if (lane == 0) {   // every copy has landed before the CTA ends
      *static_cast<volatile uint32_t*>(ended) = 1u + part_q.n + part_do.n;
      if (nk) mbar_wait(k_full, (uint32_t)(nk - 1) & 1u, 1u, p.err);
      if (nv) mbar_wait(v_full, (uint32_t)(nv - 1) & 1u, 1u, p.err);
      part_q.drain(landed_q, C::kQ, p.err);
      part_do.drain(landed_do, C::kDo, p.err);
      for (int k = nqs > C::kQ ? nqs - C::kQ : 0; k < nqs; ++k)
        if (!mbar_wait(&q_full[k % C::kQ], (uint32_t)(k / C::kQ) & 1u, 1u, p.err)) break;
      for (int k = ndo > C::kDo ? ndo - C::kDo : 0; k < ndo; ++k)
        if (!mbar_wait(&do_full[k % C::kDo], (uint32_t)(k / C::kDo) & 1u, 1u, p.err)) break;
    }
    __syncwarp();
  } else if (warp == kIssueWarp) {
    // ---- products ----
    const uint32_t one = elect_one();
    const uint32_t ak = smem_u32(sk), av = smem_u32(sv), aq = smem_u32(sq), ado = smem_u32(sdo);
    auto wait = [&](uint64_t* b, uint32_t par) {
      const bool r = warp_wait(b, par & 1u, 2u, p.err, p.limit);
      fence_after();
      return r;
    };
    auto q_in = [&](int g) { return wait(&q_full[g % C::kQ], (uint32_t)(g / C::kQ)); };
    auto do_in = [&](int g) { return wait(&do_full[g % C::kDo], (uint32_t)(g / C::kDo)); };
    auto q_at = [&](int g) { return aq + (uint32_t)(g % C::kQ) * C::kTile; };
    auto do_at = [&](int g) { return ado + (uint32_t)(g % C::kDo) * C::kTile; };
    const uint32_t ts = tmem + C::kS, tp = tmem + C::kDp;
    int g = 0;          // query tiles so far
    uint32_t i = 0;     // items so far
    bool ok = true;
    while (ok && items.take(t, hk)) {
      const Span sp(t, hk, p.per, mine, rank);
      if (!(ok = wait(k_full, i))) break;
      // S and dP of tile it over the P and dS of the one before, whose products come first
#pragma unroll 1
      for (int it = 0; it <= sp.n; ++it, ++g) {
        if (it > 0) {
          if (!(ok = wait(p_full, (uint32_t)(g - 1)))) break;
          Tl::template mma_tn<kCols>(tmem + C::kDv, ts, do_at(g - 1), C::kIdD, it > 1, one);
          commit(&do_empty[(g - 1) % C::kDo], one);
        }
        if (it < sp.n) {
          if (!(ok = q_in(g))) break;
          Tl::mma_nt(ts, ak, q_at(g), C::kIdS, one);
          commit(s_full, one);
          if (it + 1 == sp.n) commit(k_empty, one);
        }
        if (it > 0) {
          if (!(ok = wait(ds_full, (uint32_t)(g - 1)))) break;
          Tl::template mma_tn<kCols>(tmem + C::kDk, tp, q_at(g - 1), C::kIdD, it > 1, one);
          commit(&q_empty[(g - 1) % C::kQ], one);
        }
        if (it < sp.n) {
          if (!(ok = (it > 0 || wait(v_full, i)) && do_in(g))) break;
          Tl::mma_nt(tp, av, do_at(g), C::kIdS, one);
          commit(dp_full, one);
        }
      }
      --g;   // (n + 1 rounds)
      ++i;
      if (ok) commit(all, one);
    }
    commit(done, one);   // every product has completed before the tensor memory is freed
    mbar_wait(done, 0u, 2u, p.err);
    __syncwarp();
  } else if (warp == kStatWarp) {
    // ---- statistics of the query tile, four queries per lane, read one tile ahead ----
    uint32_t g = 0;
    bool ok = true;
    while (ok && items.take(t, hk)) {
      const Span sp(t, hk, p.per, mine, rank);
      float vl[4], vd[4];
      int qi = sp.j, h = sp.h0;
      auto read = [&](bool more) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int r = qi * kRows + lane + 32 * k;
          const bool in = more && r < t.len;
          const int64_t at = (int64_t)h * p.T + t.row0 + r;
          vl[k] = in ? -p.lse[at] * kLog2e : -INFINITY;   // a query behind the sequence: P = 0
          vd[k] = in ? -p.delta[at] : 0.f;
        }
      };
      read(true);
      for (int it = 0; it < sp.n; ++it, ++g) {
        if (g && !(ok = warp_wait(lse_empty, (g - 1) & 1u, 1u, p.err, p.limit))) break;
#pragma unroll
        for (int k = 0; k < 4; ++k) s_lse[lane + 32 * k] = vl[k];
        __syncwarp();
        if (lane == 0) mbar_arrive(lse_full);
        if (g && !(ok = warp_wait(delta_empty, (g - 1) & 1u, 1u, p.err, p.limit))) break;
#pragma unroll
        for (int k = 0; k < 4; ++k) s_delta[lane + 32 * k] = vd[k];
        __syncwarp();
        if (lane == 0) mbar_arrive(delta_full);
        if (++qi == sp.nb) {
          qi = sp.j;
          ++h;
        }
        read(it + 1 < sp.n);
      }
    }
  } else if (warp == kZeroWarp) {
    // ---- zeros behind the sequences, in Q and dO ----
    Partial part_q, part_do;
    int g = 0;   // query tiles so far
    bool ok = true;
    while (ok && items.take(t, hk)) {
      const Span sp(t, hk, p.per, mine, rank);
      const int rows = t.len - (sp.nb - 1) * kRows;
      if (rows < kRows)
        for (int it = sp.nq - 1; it < sp.n && ok; it += sp.nq) {   // the last query tile of each head
          const int a = (g + it) % C::kQ, b = (g + it) % C::kDo;
          ok = part_q.pass<D>(sq + a * C::kTile, a, rows, landed_q, q_full, lane, p.err, ended, part_q.n + part_do.n) &&
               part_do.pass<D>(sdo + b * C::kTile, b, rows, landed_do, do_full, lane, p.err, ended, part_q.n + part_do.n);
        }
      g += sp.n;
    }
  } else if (warp < kComputeWarps) {
    Sp::compute();
    // ---- elementwise: warpgroup w has queries 32 w .. 32 w + 31. A thread has four keys and eight queries of
    // each warp's 32 x 32: a whole key's 32 queries would want all their statistics, 16 reads of shared memory
    // per tile, which the products keep as busy as themselves.
    const int w = warp >> 2, r = threadIdx.x & 127, q = lane & 3;
    const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t ts = lanes + C::kS + kCols * w, tp = lanes + C::kDp + kCols * w;
    const f2 c2 = mk2(p.c, p.c);
    const uint64_t* z_lse = reinterpret_cast<const uint64_t*>(s_lse + kCols * w + 2 * q);
    const uint64_t* z_delta = reinterpret_cast<const uint64_t*>(s_delta + kCols * w + 2 * q);
    uint32_t g = 0, item = 0;
    bool ok = true;
    while (ok && items.take(t, hk)) {
      const Span sp(t, hk, p.per, mine, rank);
      int qi = sp.j;
      for (int it = 0; it < sp.n; ++it, ++g) {
        const uint32_t par = g & 1u;
        if (!(ok = warp_wait(lse_full, par, 4u, p.err, p.limit) && warp_wait(s_full, par, 4u, p.err, p.limit))) break;
        fence_after();
        uint32_t x[kCols], u[kCols / 2];   // x: keys +0 and +8, then +16 and +24
        tmem_ld16x32_nw(ts, x);
        tmem_ld16x32_nw(ts + (16u << 16), x + 16);
        f2 z[4];
#pragma unroll
        for (int b = 0; b < 4; ++b) z[b] = z_lse[4 * b];
        tmem_wait_ld_n<kCols>(x);
#pragma unroll
        for (int k = 0; k < kCols / 2; ++k) {
          const float2 a = un2(fma2(mk2(__uint_as_float(x[2 * k]), __uint_as_float(x[2 * k + 1])), c2, z[k / 2 % 4]));
          x[2 * k] = __float_as_uint(exp2_(a.x));
          x[2 * k + 1] = __float_as_uint(exp2_(a.y));
        }
        if (qi == sp.j && w <= (warp & 3)) {   // the tile on the diagonal: queries from the key's own on
          const int key = w == (warp & 3) ? lane >> 2 : 32;   // (none beside keys behind all of the warpgroup's queries)
#pragma unroll
          for (int k = 0; k < kCols; ++k)
            if (8 * (k / 4 % 4) + 2 * q + (k & 1) < key + 8 * (k / 2 % 2) + 16 * (k / 16)) x[k] = 0u;
        }
#pragma unroll
        for (int k = 0; k < kCols / 2; ++k) u[k] = pack_bf16(__uint_as_float(x[2 * k]), __uint_as_float(x[2 * k + 1]));
        tmem_st16x16(ts, u);
        tmem_st16x16(ts + (16u << 16), u + 8);
        tmem_wait_st();
        fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(p_full);
          mbar_arrive(lse_empty);
        }
        if (!(ok = warp_wait(delta_full, par, 4u, p.err, p.limit) && warp_wait(dp_full, par, 4u, p.err, p.limit))) break;
        fence_after();
        uint32_t y[kCols];
        tmem_ld16x32_nw(tp, y);
        tmem_ld16x32_nw(tp + (16u << 16), y + 16);
#pragma unroll
        for (int b = 0; b < 4; ++b) z[b] = z_delta[4 * b];
        tmem_wait_ld_n<kCols>(y);
#pragma unroll
        for (int k = 0; k < kCols / 2; ++k) {
          const float2 a = un2(mul2(mk2(__uint_as_float(x[2 * k]), __uint_as_float(x[2 * k + 1])),
                                    add2(mk2(__uint_as_float(y[2 * k]), __uint_as_float(y[2 * k + 1])), z[k / 2 % 4])));
          u[k] = pack_bf16(a.x, a.y);
        }
        tmem_st16x16(tp, u);
        tmem_st16x16(tp + (16u << 16), u + 8);
        tmem_wait_st();
        fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(ds_full);
          mbar_arrive(delta_empty);
        }
        if (++qi == sp.nb) qi = sp.j;
      }
      if (!ok || !(ok = warp_wait(all, item++ & 1u, 4u, p.err, p.limit))) break;
      fence_after();
      const int row = sp.j * kRows + r, half = w & 1, c0 = half * (D / 2);
      if constexpr (CL) {
        // the item's only one: no copy is under way into Q's and dO's places, and every product has read them
        float* tile = reinterpret_cast<float*>(sq) + (w >> 1) * kRows * D;
        const uint32_t col = lanes + (w < 2 ? C::kDv : C::kDk) + c0;
#pragma unroll
        for (int k = 0; k < D / 64; ++k) {
          float v[32];
          tmem_ld32(col + 32 * k, v);
#pragma unroll
          for (int c = 0; c < 8; ++c)
            *reinterpret_cast<float4*>(sum_at<D>(tile, r, c0 / 4 + 8 * k + c)) = make_float4(v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]);
        }
      } else {
        // through V's place, whose products are complete
        const int row0 = row - lane;
        const int64_t at = (int64_t)t.row0 + row0, ld = w < 2 ? p.ld_v : p.ld_k;
        __nv_bfloat16* out = (w < 2 ? p.dV : p.dK) + at * ld + (int64_t)hk * D + c0;
        const uint32_t col = lanes + (w < 2 ? C::kDv : C::kDk) + c0;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          uint8_t* stage = sv + warp * (C::kTile / kComputeWarps);
          uint32_t u[D / 8];
          read_rows<D / 4>(col + k * (D / 4), w < 2 ? 1.f : p.scale, u);
          stage_rows<D / 4>(stage, u, lane);
          write_rows<D / 4>(stage, out + k * (D / 4), ld, t.len - row0, lane);
        }
        fence_async();   // (the reads come before the next copy, which is of another proxy)
        __syncwarp();
        if (lane == 0) mbar_arrive(v_empty);
      }
      fence_before();   // (the sums have been read before the next item's first P arrives)
    }
    if (CL && !ok) *complete = 0u;
    fence_before();
  }
  if constexpr (CL) {
    cluster_sync_all();
    Items again(p.plan, p.heads, p.split);
    // (the compute warps alone: the others have few registers left)
    if (warp < kComputeWarps && again.take(t, hk)) {   // the same for every CTA of the cluster
      const int split = p.split, j = (t.len + kRows - 1) / kRows - 1 - t.index;
      bool whole = true;   // sums that lack a CTA's part are not stored
      for (int k = 0; k < split; ++k) {
        uint32_t at, v;
        asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(complete)), "r"(k));
        asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
        whole = whole && v != 0u;
      }
      // this CTA's share of the rows, the CTAs' parts added in order
      const int rows = kRows / split, total = 2 * rows * (D / 4);
      for (int e = threadIdx.x; whole && e < total; e += 32 * kComputeWarps) {
        const int c = e % (D / 4), rr = e / (D / 4), which = rr / rows, r = rank * rows + rr % rows;
        const int64_t row = (int64_t)j * kRows + r;
        if (row >= t.len) continue;
        const float* src = sum_at<D>(reinterpret_cast<float*>(sq) + which * kRows * D, r, c);
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int k = 0; k < split; ++k) {
          const float4 u = dsmem_ld4(src, k);
          v.x += u.x; v.y += u.y; v.z += u.z; v.w += u.w;
        }
        const float f = which ? p.scale : 1.f;
        const float out[4] = {v.x * f, v.y * f, v.z * f, v.w * f};
        store4((which ? p.dK + (t.row0 + row) * p.ld_k : p.dV + (t.row0 + row) * p.ld_v) + (int64_t)hk * D + 4 * c, out);
      }
    }
    cluster_sync_all();   // the peers have read this CTA's shared memory
  }
  __syncthreads();
  if (warp == kIssueWarp) {
    fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ---- dQ ------------------------------------------------------------------------------------
template <int D>
struct DqCfg {
  static constexpr int kTile = Tile<D>::kBytes;
  static constexpr int kK = D == 128 ? 2 : 4, kV = D == 128 ? 1 : 3;   // tiles of K and V in flight or in use
  static constexpr int kBarriers = 512;
  static constexpr int kSmem = (4 + kK + kV) * kTile + kBarriers + 1024 /*alignment*/;
  static_assert(kSmem <= 227 * 1024, "shared memory per CTA");
  static constexpr uint32_t kIdS = idesc(kFmtBF16, 128, 128);
  static constexpr uint32_t kIdD = idesc(kFmtBF16, 128, D, false, true);
  static constexpr uint32_t kX = 0, kDq = 256;   // tensor memory: S, then dP, then dS of both tiles; dQ of both
};

template <int D>
__global__ void __launch_bounds__(SplitFwd::kThreads, 1) k_attn_dq(const __grid_constant__ BwdK p) {
  using C = DqCfg<D>;
  using Tl = Tile<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sq = base;
  uint8_t* sdo = sq + 2 * C::kTile;
  uint8_t* sk = sdo + 2 * C::kTile;
  uint8_t* sv = sk + C::kK * C::kTile;
  uint64_t* k_full = reinterpret_cast<uint64_t*>(sv + C::kV * C::kTile);
  uint64_t* k_empty = k_full + C::kK;
  uint64_t* v_full = k_empty + C::kK;
  uint64_t* v_empty = v_full + C::kV;
  uint64_t* q_full = v_empty + C::kV;   // [2]
  uint64_t* q_empty = q_full + 2;       // [2] the last S of a tile is complete
  uint64_t* do_full = q_empty + 2;      // [2]
  uint64_t* do_empty = do_full + 2;     // [2] dQ of a tile has left through dO's place
  uint64_t* s_full = do_empty + 2;      // [2]
  uint64_t* s_read = s_full + 2;        // [2] S is in registers
  uint64_t* dp_full = s_read + 2;       // [2]
  uint64_t* ds_full = dp_full + 2;      // [2][2] half of a tile's dS is in place
  uint64_t* dq_full = ds_full + 4;      // [2]
  uint64_t* landed = dq_full + 2;       // [kK] see Partial
  uint64_t* done = landed + C::kK;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
  uint32_t* ended = tmem_slot + 1;      // see Partial
  float* s_c = reinterpret_cast<float*>(tmem_slot + 2);
  uint32_t* go = tmem_slot + 3;         // the inputs are there
  static_assert((3 * C::kK + 2 * C::kV + 21) * 8 + 16 <= C::kBarriers, "barriers");
  const int warp = uniform((int)threadIdx.x >> 5), lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kK; ++s) {
      mbar_init(&k_full[s], 1);
      mbar_init(&k_empty[s], 1);
      mbar_init(&landed[s], 1);
    }
    for (int s = 0; s < C::kV; ++s) {
      mbar_init(&v_full[s], 1);
      mbar_init(&v_empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&q_full[s], 1);
      mbar_init(&q_empty[s], 1);
      mbar_init(&do_full[s], 1);
      mbar_init(&do_empty[s], 4);
      mbar_init(&s_full[s], 1);
      mbar_init(&s_read[s], 4);
      mbar_init(&dp_full[s], 1);
      mbar_init(&ds_full[2 * s], 4);
      mbar_init(&ds_full[2 * s + 1], 4);
      mbar_init(&dq_full[s], 1);
    }
    mbar_init(done, 1);
    *s_c = p.c;
    *ended = 0u;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    fence_async();
  }
  if (warp == 9) tmem_alloc(tmem_slot, 512);
  // The kernel ahead, k_attn_dkv, reads what this one reads and writes none of it: a CTA begins where that leaves an SM,
  // and waits for it at its end only, so that whatever follows finds both complete. That it was let in says nothing of
  // what it can see. The outputs of delta's and all earlier kernels are seen through `ready`, which k_attn_dkv
  // releases behind its own wait for them, and before it lets this kernel in, so that the flag is there at the first
  // look; the barrier hands it to all threads, the fence to the bulk copies. (Packed batch, when the early start came in:
  // 411 -> 404 us.)
  if (warp == 11 && lane == 0) *go = flag_wait(p.ready, 1u, p.err, p.limit) ? 1u : 0u;
  fence_before();
  __syncthreads();
  fence_after();
  asm volatile("fence.proxy.async;" ::: "memory");
  const uint32_t tmem = (uint32_t)uniform((int)*tmem_slot);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  if (warp >= 8) SplitFwd::issue();
  AttnTile t;
  int group;
  Items items(p.plan, p.groups);
  if (!uniform((int)*go)) items.n = 0;
  if (warp == 8) {
    // ---- loads, in the order in which the products free their places ----
    int gk = 0, gv = 0, nq0 = 0, nq1 = 0, nd0 = 0, nd1 = 0;   // tiles asked for
    Partial part;
    bool ok = true;
    auto own = [&](uint8_t* dst, const CUtensorMap* map, uint64_t* full, uint64_t* empty, int& n, int col, int row) {
      if (n && !warp_wait(empty, (uint32_t)(n - 1) & 1u, 1u, p.err, p.limit)) return false;
      ++n;
      if (lane == 0) {
        mbar_expect_tx(full, C::kTile);
        Tl::load(dst, map, full, col, row);
      }
      return true;
    };
    while (ok && items.take(t, group)) {
      const Pair pr(t, group, p.by_heads);
      const int col = pr.h0 / p.per * D;
      ok = own(sq, &p.tq, &q_full[0], &q_empty[0], nq0, pr.h0 * D, t.row0 + pr.q0 * kRows);
      for (int j = 0; j < pr.most && ok; ++j) {
        const int a = gk % C::kK, b = gv % C::kV, rows = t.len - j * kRows;
        if (gk >= C::kK && !(ok = warp_wait(&k_empty[a], (uint32_t)(gk / C::kK - 1) & 1u, 1u, p.err, p.limit))) break;
        const bool some = rows < kRows;   // the sequence's last rows
        if (lane == 0) {
          uint64_t* bar = some ? &landed[a] : &k_full[a];
          mbar_expect_tx(bar, C::kTile);
          Tl::load(sk + a * C::kTile, &p.tk, bar, col, t.row0 + j * kRows);
        }
        if (some) part.next(a);
        ++gk;
        if (j == 0) {
          if (pr.n1 && !(ok = own(sq + C::kTile, &p.tq, &q_full[1], &q_empty[1], nq1, pr.h1 * D, t.row0 + pr.q1 * kRows))) break;
          if (!(ok = own(sdo, &p.tdo, &do_full[0], &do_empty[0], nd0, pr.h0 * D, t.row0 + pr.q0 * kRows))) break;
        }
        if (gv >= C::kV && !(ok = warp_wait(&v_empty[b], (uint32_t)(gv / C::kV - 1) & 1u, 1u, p.err, p.limit))) break;
        if (lane == 0) {
          mbar_expect_tx(&v_full[b], C::kTile);
          Tl::load(sv + b * C::kTile, &p.tv, &v_full[b], col, t.row0 + j * kRows);
        }
        ++gv;
        if (j == 0 && pr.n1)
          ok = own(sdo + C::kTile, &p.tdo, &do_full[1], &do_empty[1], nd1, pr.h1 * D, t.row0 + pr.q1 * kRows);
      }
    }
    if (lane == 0) {   // every copy has landed before the CTA ends
      *static_cast<volatile uint32_t*>(ended) = 1u + part.n;
      if (nq0) mbar_wait(&q_full[0], (uint32_t)(nq0 - 1) & 1u, 1u, p.err);
      if (nq1) mbar_wait(&q_full[1], (uint32_t)(nq1 - 1) & 1u, 1u, p.err);
      if (nd0) mbar_wait(&do_full[0], (uint32_t)(nd0 - 1) & 1u, 1u, p.err);
      if (nd1) mbar_wait(&do_full[1], (uint32_t)(nd1 - 1) & 1u, 1u, p.err);
      part.drain(landed, C::kK, p.err);
      for (int k = gk > C::kK ? gk - C::kK : 0; k < gk; ++k)
        if (!mbar_wait(&k_full[k % C::kK], (uint32_t)(k / C::kK) & 1u, 1u, p.err)) break;
      for (int k = gv > C::kV ? gv - C::kV : 0; k < gv; ++k)
        if (!mbar_wait(&v_full[k % C::kV], (uint32_t)(k / C::kV) & 1u, 1u, p.err)) break;
    }
    __syncwarp();
  } else if (warp == 9) {
    // ---- products ----
    const uint32_t one = elect_one();
    const uint32_t aq = smem_u32(sq), ado = smem_u32(sdo), ak = smem_u32(sk), av = smem_u32(sv);
    auto wait = [&](uint64_t* b, uint32_t n) {
      const bool r = warp_wait(b, n & 1u, 2u, p.err, p.limit);
      fence_after();
      return r;
    };
    auto k_in = [&](int g) { return wait(&k_full[g % C::kK], (uint32_t)(g / C::kK)); };
    auto v_in = [&](int g) { return wait(&v_full[g % C::kV], (uint32_t)(g / C::kV)); };
    int g = 0;                                // key tiles so far
    uint32_t i0 = 0, i1 = 0, c0 = 0, c1 = 0;  // of each tile: items and key tiles so far
    bool ok = true;
    while (ok && items.take(t, group)) {
      const Pair pr(t, group, p.by_heads);
      const int tiles = pr.n1 ? 2 : 1;
      auto score = [&](int s, int at, bool last) {   // S over the dS before it
        Tl::mma_nt(tmem + C::kX + 128 * s, aq + s * C::kTile, ak + (uint32_t)(at % C::kK) * C::kTile, C::kIdS, one);
        commit(&s_full[s], one);
        if (last) commit(&q_empty[s], one);
      };
      ok = k_in(g);
#pragma unroll 1
      for (int s = 0; s < tiles && ok; ++s) {
        if (!(ok = wait(&q_full[s], s ? i1 : i0))) break;
        score(s, g, pr.n(s) == 1);
      }
#pragma unroll 1
      for (int j = 0; j < pr.most && ok; ++j, ++g) {
        if (!(ok = v_in(g))) break;
#pragma unroll 1
        for (int s = j < pr.n0 ? 0 : 1; s < tiles; ++s) {
          if (j == 0 && !(ok = wait(&do_full[s], s ? i1 : i0))) break;
          if (!(ok = wait(&s_read[s], s ? c1 : c0))) break;
          Tl::mma_nt(tmem + C::kX + 128 * s, ado + s * C::kTile, av + (uint32_t)(g % C::kV) * C::kTile, C::kIdS, one);
          commit(&dp_full[s], one);
        }
        if (!ok) break;
        commit(&v_empty[g % C::kV], one);
        const uint32_t kt = ak + (uint32_t)(g % C::kK) * C::kTile;
        bool have_k = false;
#pragma unroll 1
        for (int s = j < pr.n0 ? 0 : 1; s < tiles; ++s) {
          const uint32_t td = tmem + C::kX + 128 * s, tq = tmem + C::kDq + 128 * s, c = s ? c1 : c0;
          if (!(ok = wait(&ds_full[2 * s], c))) break;
          Tl::template mma_tn<128, 0, 4>(tq, td, kt, C::kIdD, j > 0, one);
          if (!(ok = wait(&ds_full[2 * s + 1], c))) break;
          Tl::template mma_tn<128, 4, 8>(tq, td, kt, C::kIdD, true, one);
          if (s + 1 == tiles) commit(&k_empty[g % C::kK], one);
          if (s) ++c1; else ++c0;
          if (j + 1 < pr.n(s)) {
            if (!have_k && !(ok = k_in(g + 1))) break;
            have_k = true;
            score(s, g + 1, j + 2 == pr.n(s));
          } else {
            commit(&dq_full[s], one);
          }
        }
      }
      ++i0;
      if (pr.n1) ++i1;
    }
    commit(done, one);   // every product has completed before the tensor memory is freed
    mbar_wait(done, 0u, 2u, p.err);
    __syncwarp();
  } else if (warp == 10) {
    // ---- zeros behind the sequences, in K ----
    Partial part;
    int g = 0;   // key tiles so far
    while (items.take(t, group)) {
      const Pair pr(t, group, p.by_heads);
      g += pr.most;
      const int rows = t.len - (pr.most - 1) * kRows, a = (g - 1) % C::kK;
      if (rows < kRows && !part.pass<D>(sk + a * C::kTile, a, rows, landed, k_full, lane, p.err, ended, part.n)) break;
    }
  } else if (warp < 8) {
    SplitFwd::compute();
    // ---- elementwise and epilogue: thread = query r of tile s ----
    const int s = warp >> 2, r = threadIdx.x & 127;
    const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t tx = lanes + C::kX + 128 * s, tq = lanes + C::kDq + 128 * s;
    uint32_t c = 0, i = 0;   // key tiles and items so far
    bool ok = true;
    while (ok && items.take(t, group)) {
      const Pair pr(t, group, p.by_heads);
      const int n = pr.n(s);
      if (!n) continue;
      const int row = pr.qi(s) * kRows + r, h = pr.h(s);
      const int64_t at = (int64_t)t.row0 + row;
      const bool live = row < t.len;
      const float lse = live ? p.lse[(int64_t)h * p.T + at] * kLog2e : 0.f;
      const float delta = live ? p.delta[(int64_t)h * p.T + at] : 0.f;
      for (int j = 0; j < n; ++j, ++c) {
        if (!(ok = warp_wait(&s_full[s], c & 1u, 4u, p.err, p.limit))) break;
        fence_after();
        uint32_t x[128];
#pragma unroll
        for (int k = 0; k < 4; ++k) tmem_ld32_nw(tx + 32 * k, x + 32 * k);
        tmem_wait_ld_n<128>(x);
        fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s_read[s]);   // dP may go over it, while P is computed
        const float c1 = read_here(s_c);
        const f2 c2 = mk2(c1, c1), l2 = mk2(-lse, -lse), d2 = mk2(-delta, -delta);
#pragma unroll
        for (int k = 0; k < 64; ++k) {
          const float2 a = un2(fma2(mk2(__uint_as_float(x[2 * k]), __uint_as_float(x[2 * k + 1])), c2, l2));
          x[2 * k] = __float_as_uint(exp2_(a.x));
          x[2 * k + 1] = __float_as_uint(exp2_(a.y));
        }
        if (!(ok = warp_wait(&dp_full[s], c & 1u, 4u, p.err, p.limit))) break;
        fence_after();
        uint32_t y[2][32];   // dP, 32 columns worked on and 32 on their way
        tmem_ld32_nw(tx, y[0]);
        tmem_ld32_nw(tx + 32, y[1]);
        tmem_wait_ld_n<32>(y[0]);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          uint32_t* yk = y[k & 1];
          uint32_t u[16];
          if (k) tmem_wait_ld_n<32>(yk);
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const int at2 = 32 * k + 2 * e;
            const float2 a = un2(mul2(mk2(__uint_as_float(x[at2]), __uint_as_float(x[at2 + 1])),
                                      add2(mk2(__uint_as_float(yk[2 * e]), __uint_as_float(yk[2 * e + 1])), d2)));
            u[e] = pack_bf16(a.x, a.y);
          }
          if (j == n - 1) {   // the tile on the diagonal: keys up to the query's own, 32 at a time beside the warp's rows
            if (k == (warp & 3)) {
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                if (2 * e > lane) u[e] = 0u;
                else if (2 * e + 1 > lane) u[e] &= 0xffffu;
              }
            } else if (k > (warp & 3)) {
#pragma unroll
              for (int e = 0; e < 16; ++e) u[e] = 0u;
            }
          }
          tmem_st16(tx + 16 * k, u);
          if (k & 1) {   // the product of half the keys begins while the other half is turned into dS
            tmem_wait_st();
            fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&ds_full[2 * s + (k >> 1)]);
          }
          if (k < 2) tmem_ld32_nw(tx + 32 * (k + 2), yk);
        }
      }
      if (!ok || !(ok = warp_wait(&dq_full[s], i++ & 1u, 4u, p.err, p.limit))) break;
      fence_after();
      // through dO's place, whose products are complete
      const int row0 = row - lane;
      const bool whole = t.len - row0 >= 32;
#pragma unroll 1
      for (int k = 0; k < D / 64; ++k) {
        uint8_t* stage = sdo + s * C::kTile + ((warp & 3) * (D / 64) + k) * 4096;
        uint32_t u[32];
        read_rows<64>(tq + 64 * k, p.scale, u);
        stage_rows<64>(stage, u, lane);
        if (whole)
          send_rows(&p.tdq, stage, h * D + 64 * k, at - lane, lane);
        else   // the rows behind belong to others
          write_rows<64>(stage, p.dQ + (at - lane) * p.ld_q + (int64_t)h * D + 64 * k, p.ld_q, t.len - row0, lane);
      }
      rows_read(lane);
      fence_async();   // (the reads come before the next copy, which is of another proxy)
      __syncwarp();
      if (lane == 0) mbar_arrive(&do_empty[s]);
      fence_before();   // (dQ has been read before the next item's first dS arrives)
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
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// CTAs that share a key tile's query heads: as many as the SMs hold at once, so that few key heads over few tokens
// still use them. 8 sequences of 128 tokens, 32 / 4 heads of 64: 32 items, a cluster of 4 each; all of the backward
// pass 18.6 us, 20.5 with one CTA for each. Where items fill the SMs, persistent CTAs overlap them. The host knows the
// tokens and the number of sequences, and takes them to be equally long (a short one has a key tile of its own, too):
// 1024 tokens in 128 sequences 106 us, 177 in clusters by the tokens alone; in 32, 43 and 66 (32 / 8 heads of 128).
// Empty sequences count: one of 1024 tokens and 63 empty ones take 72 us, without those 30.
int dkv_split(const AttnArgs& a, int sms) {
  const int64_t seqs = a.plan.n_seq < a.T ? a.plan.n_seq : a.T;
  const int64_t items = seqs * ((a.T + seqs * kRows - 1) / (seqs * kRows)) * a.kv_heads;
  int n = 1;
  while (n < 8 && a.q_heads / a.kv_heads % (2 * n) == 0 && items * 2 * n <= sms) n *= 2;
  return n;
}

cudaError_t launch_clusters(void (*kernel)(const BwdK), unsigned grid, unsigned threads, size_t smem, cudaStream_t st,
                            const BwdK& k, int cluster) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)cluster;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = add_pdl_attr(at, 1);
  return cudaLaunchKernelEx(&cfg, kernel, k);
}

template <int D>
cudaError_t bwd_launch(const AttnArgs& a, cudaStream_t st) {
  static std::atomic<uint64_t> set{0};
  cudaError_t e = once_on_device(set, [] {
    cudaError_t r = set_up<Sp>(k_attn_dkv<D, false>, DkvCfg<D>::kSmem);
    if (r == cudaSuccess) r = set_up<Sp>(k_attn_dkv<D, true>, DkvCfg<D>::kSmem);
    return r != cudaSuccess ? r : set_up<SplitFwd>(k_attn_dq<D>, DqCfg<D>::kSmem);
  });
  if (e != cudaSuccess) return e;
  BwdK k{};
  if (!attn_map(&k.tq, a.Q, a.q_heads * D, a.T, a.ld_q) || !attn_map(&k.tk, a.K, a.kv_heads * D, a.T, a.ld_k) ||
      !attn_map(&k.tv, a.V, a.kv_heads * D, a.T, a.ld_v) || !attn_map(&k.tdo, a.dO, a.q_heads * D, a.T, a.ld_o) ||
      !attn_map(&k.tdq, a.dQ, a.q_heads * D, a.T, a.ld_q, 32))
    return cudaErrorInvalidValue;
  k.per = a.q_heads / a.kv_heads;
  k.c = a.scale * kLog2e;
  k.scale = a.scale;
  k.T = a.T; k.ld_q = a.ld_q; k.ld_k = a.ld_k; k.ld_v = a.ld_v;
  k.lse = a.lse; k.delta = a.delta; k.ready = a.ready;
  k.dQ = static_cast<__nv_bfloat16*>(a.dQ);
  k.dK = static_cast<__nv_bfloat16*>(a.dK);
  k.dV = static_cast<__nv_bfloat16*>(a.dV);
  k.err = error_word();
  if (!k.err) return cudaErrorInvalidDevice;
  k.limit = tc_wait_limit();
  const int sms = sm_count();
  if (sms <= 0) return cudaErrorInvalidDevice;
  k.by_heads = k.per % 2 == 0;
  const int w = k.by_heads ? 0 : 1;
  k.groups = k.by_heads ? a.q_heads / 2 : a.q_heads;
  const int64_t pre = (a.T * a.q_heads * (D / 8) + 255) / 256, most = a.plan.most[w] * k.groups;
  const int64_t grid = a.plan.most[0] * a.kv_heads;
  if (pre > INT32_MAX || most > INT32_MAX || grid > INT32_MAX) return cudaErrorInvalidValue;
  prof_begin(0, st);
  e = launch_kernel(k_attn_delta<D>, (unsigned)pre, 256, 0, st, static_cast<const __nv_bfloat16*>(a.O),
                    static_cast<const __nv_bfloat16*>(a.dO), a.ld_o, (int)a.q_heads, a.T, a.delta, a.ready);
  if (e != cudaSuccess) return e;
  k.plan = plan_ref(a, 0);
  k.heads = a.kv_heads;
  k.split = dkv_split(a, sms);
  if (grid * k.split > INT32_MAX) return cudaErrorInvalidValue;
  prof_begin(0, st);
  e = k.split > 1 ? launch_clusters(k_attn_dkv<D, true>, (unsigned)(grid * k.split), Sp::kThreads, DkvCfg<D>::kSmem, st, k, k.split)
                  : launch_kernel(k_attn_dkv<D, false>, (unsigned)(grid < sms ? grid : sms), Sp::kThreads, DkvCfg<D>::kSmem, st, k);
  if (e != cudaSuccess) return e;
  k.plan = plan_ref(a, w);
  prof_begin(0, st);
  return launch_kernel(k_attn_dq<D>, (unsigned)(most < sms ? most : sms), SplitFwd::kThreads, DqCfg<D>::kSmem, st, k);
}

}  // namespace

cudaError_t launch_attn_backward(const AttnArgs& a, cudaStream_t st) {
  return a.dim == 128 ? bwd_launch<128>(a, st) : bwd_launch<64>(a, st);
}

}  // namespace lora
