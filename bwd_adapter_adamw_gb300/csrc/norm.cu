// Layer norm and root-mean-square norm in front of an adapted linear: forward, and the backward
// pass with the token sums of the weight's and the shift's gradients.
//
//   forward   xhat = (x - mean) rstd,  Y = gamma xhat + beta
//   backward  g = gamma dY,  dX = rstd (g - sum g / dim - xhat (sum g xhat) / dim)   (RMS: without
//             the sum of g),  dgamma += sum_t dY xhat,  dbeta += sum_t dY
//
// Both passes are bound by memory: a row is read once, held in registers between its sums and its
// outputs, and written once.
#include "tc_ptx.cuh"

namespace lora {

namespace {

constexpr int kNormThreads = 256;

// Two floats in a 64-bit register pair, one instruction for both: in bf16 both passes are as much
// issue-bound as memory-bound.
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
__device__ __forceinline__ float sum2(f2 v) {
  const float2 f = un2(v);
  return f.x + f.y;
}

// A 16-byte vector of N elements as N / 2 pairs.
template <typename E> struct Pack;
template <> struct Pack<float> {
  static constexpr int N = 4;
  __device__ static void get(const uint4& v, f2* f) {
    f[0] = mk2(__uint_as_float(v.x), __uint_as_float(v.y));
    f[1] = mk2(__uint_as_float(v.z), __uint_as_float(v.w));
  }
  __device__ static uint4 put(const f2* f) {
    const float2 a = un2(f[0]), b = un2(f[1]);
    return make_uint4(__float_as_uint(a.x), __float_as_uint(a.y), __float_as_uint(b.x),
                      __float_as_uint(b.y));
  }
};
template <> struct Pack<__nv_bfloat16> {
  static constexpr int N = 8;
  __device__ static void get(const uint4& v, f2* f) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j)
      f[j] = mk2(__uint_as_float(w[j] << 16), __uint_as_float(w[j] & 0xFFFF0000u));
  }
  __device__ static uint4 put(const f2* f) {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 a = un2(f[j]);
      const __nv_bfloat162 h = __floats2bfloat162_rn(a.x, a.y);
      w[j] = *reinterpret_cast<const uint32_t*>(&h);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};

// N floats of a weight vector as pairs
template <int N>
__device__ __forceinline__ void load_pairs(const float* p, f2* f) {
#pragma unroll
  for (int j = 0; j < N; j += 4) {
    float t[4];
    load16(p + j, t);
    f[j / 2] = mk2(t[0], t[1]);
    f[j / 2 + 1] = mk2(t[2], t[3]);
  }
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Sums over the WPR warps of a row for R rows, the same in every lane. `sh` holds R floats per warp;
// the caller alternates two buffers so that one barrier per sum suffices.
template <int WPR, int R>
__device__ __forceinline__ void row_sums(float (&v)[R], float (*sh)[kNormThreads / 32]) {
#pragma unroll
  for (int r = 0; r < R; ++r) v[r] = warp_sum(v[r]);
  if constexpr (WPR > 1) {
    const int warp = threadIdx.x >> 5;
    if ((threadIdx.x & 31) == 0) {
#pragma unroll
      for (int r = 0; r < R; ++r) sh[r][warp] = v[r];
    }
    __syncthreads();
    const int w0 = warp / WPR * WPR;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      v[r] = 0.f;
#pragma unroll
      for (int w = 0; w < WPR; ++w) v[r] += sh[r][w0 + w];
    }
  }
}

// WPR warps per row, NV 16-byte vectors per lane and row, R rows per warp, 8 R / WPR rows per CTA.
template <typename E, int WPR, int NV, int R>
__global__ void __launch_bounds__(kNormThreads) k_norm_fwd(const E* __restrict__ X,
                                                           const float* __restrict__ gamma,
                                                           const float* __restrict__ beta,
                                                           E* __restrict__ Y,
                                                           float2* __restrict__ stats, int64_t T,
                                                           int dim, float inv_dim, float eps,
                                                           int rms) {
  grid_dep_sync();
  constexpr int N = Pack<E>::N;
  __shared__ float sh[2][R][kNormThreads / 32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t t0 = ((int64_t)blockIdx.x * (kNormThreads / 32 / WPR) + warp / WPR) * R;
  const int nvec = dim / N;
  const int first = (warp % WPR) * 32 + lane;
  uint4 v[R][NV];
  float s[R], mean[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const uint4* src = reinterpret_cast<const uint4*>(X + (t0 + r) * dim);
#pragma unroll
    for (int u = 0; u < NV; ++u) {
      const int i = first + u * 32 * WPR;
      v[r][u] = t0 + r < T && i < nvec ? __ldg(src + i) : make_uint4(0, 0, 0, 0);
    }
    mean[r] = 0.f;
  }
  if (!rms) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      f2 a = mk2(0.f, 0.f);
#pragma unroll
      for (int u = 0; u < NV; ++u) {
        f2 f[N / 2];
        Pack<E>::get(v[r][u], f);
#pragma unroll
        for (int j = 0; j < N / 2; ++j) a = add2(a, f[j]);
      }
      s[r] = sum2(a);
    }
    row_sums<WPR, R>(s, sh[0]);
#pragma unroll
    for (int r = 0; r < R; ++r) mean[r] = s[r] * inv_dim;
  }
#pragma unroll
  for (int r = 0; r < R; ++r) {
    f2 a = mk2(0.f, 0.f);
    const f2 m = mk2(-mean[r], -mean[r]);
#pragma unroll
    for (int u = 0; u < NV; ++u) {
      const int i = first + u * 32 * WPR;
      if (i < nvec) {
        f2 f[N / 2];
        Pack<E>::get(v[r][u], f);
#pragma unroll
        for (int j = 0; j < N / 2; ++j) {
          const f2 d = add2(f[j], m);
          a = fma2(d, d, a);
        }
      }
    }
    s[r] = sum2(a);
  }
  row_sums<WPR, R>(s, sh[1]);
#pragma unroll
  for (int r = 0; r < R; ++r) {
    s[r] = 1.f / sqrtf(s[r] * inv_dim + eps);
    if (first == 0 && t0 + r < T) stats[t0 + r] = make_float2(mean[r], s[r]);
  }
#pragma unroll
  for (int u = 0; u < NV; ++u) {
    const int i = first + u * 32 * WPR;
    if (i >= nvec) continue;
    f2 ga[N / 2], be[N / 2];
    load_pairs<N>(gamma + i * N, ga);
    if (beta) load_pairs<N>(beta + i * N, be);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (t0 + r >= T) break;
      f2 f[N / 2];
      Pack<E>::get(v[r][u], f);
      const f2 m = mk2(-mean[r], -mean[r]), q = mk2(s[r], s[r]);
#pragma unroll
      for (int j = 0; j < N / 2; ++j) {
        const f2 h = mul2(add2(f[j], m), q);
        f[j] = beta ? fma2(h, ga[j], be[j]) : mul2(h, ga[j]);
      }
      reinterpret_cast<uint4*>(Y + (t0 + r) * dim)[i] = Pack<E>::put(f);
    }
  }
}

// dst = sum of n tensors in fp32, one 16-byte vector per thread, four sources' loads in flight; rounded
// once, where adding into a bf16 tensor would round with every source. Memory-bound: three sources of
// 8192 x 4096 bf16 45.7 us, 5.9 TB/s.
template <typename E>
__global__ void __launch_bounds__(kNormThreads) k_sum(const __grid_constant__ SumArgs a) {
  grid_dep_sync();
  constexpr int P = Pack<E>::N / 2;
  const int64_t i = (int64_t)blockIdx.x * kNormThreads + threadIdx.x;
  if (i >= a.count / Pack<E>::N) return;
  f2 s[P];
#pragma unroll
  for (int j = 0; j < P; ++j) s[j] = mk2(0.f, 0.f);
  for (int k0 = 0; k0 < a.n; k0 += 4) {
    uint4 v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)   // (plain loads: dst may be a source)
      v[k] = k0 + k < a.n ? static_cast<const uint4*>(a.src[k0 + k])[i] : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      f2 f[P];
      Pack<E>::get(v[k], f);
#pragma unroll
      for (int j = 0; j < P; ++j) s[j] = add2(s[j], f[j]);
    }
  }
  static_cast<uint4*>(a.dst)[i] = Pack<E>::put(s);
}

constexpr int kBwdRing = 8;   // most groups of rows in flight

// Groups of rows in flight per CTA: two CTAs of 256 threads per SM, or one of 512.
int bwd_ring(int64_t group_bytes, int threads) {
  const int64_t room = (threads == 256 ? 96 : 200) * 1024;
  const int64_t n = room / (2 * group_bytes);
  return (int)(n < 1 ? 1 : n > kBwdRing ? kBwdRing : n);
}

// TPR threads per row, NV vectors per thread, R rows per thread, R TH / TPR rows at a time; persistent over
// the rows, so that a thread keeps its columns and sums their gradients in registers. Groups of
// rows of X and dY arrive in a ring of shared-memory buffers by bulk copies issued `ring` groups
// ahead: loading the next group into registers instead kept 32 KB in flight per SM and ran at
// 2.8 TB/s (8192 x 4096 bf16, 72 us). The barrier of a row's sums also frees its buffer. Partials
// go to part[CTA][2][dim], added up in order by k_norm_reduce.
//
// A thread takes 16 columns where the row allows: a row's fixed cost (the wait, the sums' shuffles
// and barrier) was as large as its arithmetic with 8 (8192 x 4096 bf16: 51 us with 512 threads per
// row, 41 with 256; 35 in packed pairs and with two rows at a time).
template <typename E, int TH, int TPR, int NV, int R>
__global__ void __launch_bounds__(TH, TH == 256 ? 2 : 1)
    k_norm_bwd(const E* __restrict__ X, const float* __restrict__ gamma, const E* __restrict__ dY,
               const float2* __restrict__ stats, const E* dX_add, E* dX, float* __restrict__ part,
               int64_t T, int dim, float inv_dim, int rms, int want, int ring, uint32_t* err,
               unsigned long long wait_limit) {
  grid_dep_sync();
  constexpr int N = Pack<E>::N;
  constexpr int RPB = TH / TPR * R;   // rows of a group; a thread's R rows are row, row + TH / TPR, ..
  constexpr int WPR = TPR / 32;
  extern __shared__ __align__(16) uint8_t bufs[];   // [ring][X | dY][RPB][dim]; then the column sums
  __shared__ float2 sh[2][R][TH / 32];
  __shared__ uint64_t full[kBwdRing];
  __shared__ uint32_t mark;              // a wait of this CTA has run out
  volatile uint32_t* failed = &mark;
  const int row = threadIdx.x / TPR, col = threadIdx.x % TPR;
  const int warp = threadIdx.x >> 5;
  const int nvec = dim / N;
  const int group = RPB * dim * (int)sizeof(E);
  const int64_t step = (int64_t)gridDim.x * RPB;
  const int64_t t_first = (int64_t)blockIdx.x * RPB;
  int filled = 0, waited = 0;            // thread 0: groups asked for, groups that have arrived
  auto fill = [&](int s, int64_t t0) {   // thread 0: rows t0 .. of the group, as far as they exist
    if (t0 >= T) return;
    ++filled;
    const int64_t rows = T - t0 < RPB ? T - t0 : RPB;
    const uint32_t bytes = (uint32_t)(rows * dim * (int64_t)sizeof(E));
    tc::mbar_expect_tx(&full[s], 2 * bytes);
    for (int k = 0; k < 2; ++k)
      asm volatile(
          "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
              tc::smem_u32(bufs + (size_t)(2 * s + k) * group)),
          "l"((k ? dY : X) + t0 * dim), "r"(bytes), "r"(tc::smem_u32(&full[s]))
          : "memory");
  };
  if (threadIdx.x == 0) {
    *failed = 0u;
    for (int s = 0; s < ring; ++s) tc::mbar_init(&full[s], 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    for (int s = 0; s < ring; ++s) fill(s, t_first + s * step);
  }
  // with few columns per thread the weights, and a row's g and xhat, stay in registers
  constexpr bool kKeep = NV * N <= 16, kHold = NV * N * R <= 16;
  constexpr int P = N / 2;   // pairs of a vector
  f2 dg[NV * P], db[NV * P], gw[kKeep ? NV * P : 1];
#pragma unroll
  for (int j = 0; j < NV * P; ++j) dg[j] = db[j] = mk2(0.f, 0.f);
  if constexpr (kKeep) {
#pragma unroll
    for (int u = 0; u < NV; ++u) {
      const int i = col + u * TPR;
      if (i < nvec) load_pairs<N>(gamma + i * N, gw + u * P);
    }
  }
  auto weights = [&](int u, int i, f2 (&ga)[P]) {
    if constexpr (kKeep) {
#pragma unroll
      for (int j = 0; j < P; ++j) ga[j] = gw[u * P + j];
    } else {
      load_pairs<N>(gamma + i * N, ga);
    }
  };
  __syncthreads();   // the barriers are set up
  int buf = 0, s = 0;
  uint32_t phase = 0;
  bool ok = true;   // from the barrier of a group on, the same in every thread: no wait has run out
  for (int64_t t0 = t_first; t0 < T; t0 += step, buf ^= 1) {
    float2 sc[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int64_t t = t0 + row + r * (TH / TPR);
      sc[r] = t < T ? __ldg(stats + t) : make_float2(0.f, 0.f);
    }
    if (ok && !tc::mbar_wait_strict(&full[s], phase, 1u, err, wait_limit)) {
      *failed = 1u;
      ok = false;
    }
    waited += ok;
    uint4 xc[R][NV], yc[R][NV];
    f2 hk[R][kHold ? NV * P : 1], gk[R][kHold ? NV * P : 1];
    float s1[R], s2[R];   // sum g, sum g xhat
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int at = row + r * (TH / TPR);
      const uint4* px = reinterpret_cast<const uint4*>(bufs + (size_t)(2 * s) * group) + at * nvec;
      const uint4* py = reinterpret_cast<const uint4*>(bufs + (size_t)(2 * s + 1) * group) + at * nvec;
      f2 a1 = mk2(0.f, 0.f), a2 = a1;
      const f2 m = mk2(-sc[r].x, -sc[r].x), q = mk2(sc[r].y, sc[r].y);
#pragma unroll
      for (int u = 0; u < NV; ++u) {
        const int i = col + u * TPR;
        const bool in = t0 + at < T && i < nvec;
        xc[r][u] = in ? px[i] : make_uint4(0, 0, 0, 0);
        yc[r][u] = in ? py[i] : make_uint4(0, 0, 0, 0);
        if (i >= nvec) continue;
        f2 x[P], y[P], ga[P];
        Pack<E>::get(xc[r][u], x);
        Pack<E>::get(yc[r][u], y);
        weights(u, i, ga);
#pragma unroll
        for (int j = 0; j < P; ++j) {
          const f2 h = mul2(add2(x[j], m), q), g = mul2(y[j], ga[j]);
          a1 = add2(a1, g);
          a2 = fma2(g, h, a2);
          dg[u * P + j] = fma2(y[j], h, dg[u * P + j]);
          db[u * P + j] = add2(db[u * P + j], y[j]);
          if constexpr (kHold) {
            hk[r][u * P + j] = h;
            gk[r][u * P + j] = g;
          }
        }
      }
      s1[r] = sum2(a1);
      s2[r] = sum2(a2);
    }
    if (want & 1) {
#pragma unroll
      for (int r = 0; r < R; ++r) {
        s1[r] = warp_sum(s1[r]);
        s2[r] = warp_sum(s2[r]);
        if ((threadIdx.x & 31) == 0) sh[buf][r][warp] = make_float2(s1[r], s2[r]);
      }
    }
    // the sums are in place, and every thread has read the buffer (its reads come before the next
    // copy, which is of another proxy)
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncthreads();
    ok = *failed == 0u;
    if (threadIdx.x == 0 && ok) fill(s, t0 + ring * step);
    if (++s == ring) {
      s = 0;
      phase ^= 1u;
    }
    if (!(want & 1)) continue;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if constexpr (WPR > 1) {   // lane w adds warp w's share, the lanes in a fixed tree
        const float2 v = sh[buf][r][warp / WPR * WPR + (threadIdx.x & (WPR - 1))];
        s1[r] = v.x;
        s2[r] = v.y;
#pragma unroll
        for (int o = WPR / 2; o > 0; o >>= 1) {
          s1[r] += __shfl_xor_sync(0xffffffffu, s1[r], o);
          s2[r] += __shfl_xor_sync(0xffffffffu, s2[r], o);
        }
      }
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int64_t t = t0 + row + r * (TH / TPR);
      if (t >= T || !ok) continue;
      const float c1 = rms ? 0.f : s1[r] * inv_dim * sc[r].y, c2 = s2[r] * inv_dim * sc[r].y;
      const f2 m = mk2(-sc[r].x, -sc[r].x), q = mk2(sc[r].y, sc[r].y);
      const f2 n1 = mk2(-c1, -c1), n2 = mk2(-c2, -c2);
#pragma unroll
      for (int u = 0; u < NV; ++u) {
        const int i = col + u * TPR;
        if (i >= nvec) continue;
        f2 x[P], y[P], ga[P], add[P];
        if constexpr (!kHold) {
          Pack<E>::get(xc[r][u], x);
          Pack<E>::get(yc[r][u], y);
          weights(u, i, ga);
        }
        if (dX_add) Pack<E>::get(*(reinterpret_cast<const uint4*>(dX_add + t * dim) + i), add);
#pragma unroll
        for (int j = 0; j < P; ++j) {
          f2 h, g;
          if constexpr (kHold) {
            h = hk[r][u * P + j];
            g = gk[r][u * P + j];
          } else {
            h = mul2(add2(x[j], m), q);
            g = mul2(y[j], ga[j]);
          }
          const f2 d = fma2(h, n2, fma2(g, q, n1));
          x[j] = dX_add ? add2(d, add[j]) : d;
        }
        __stcs(reinterpret_cast<uint4*>(dX + t * dim) + i, Pack<E>::put(x));
      }
    }
  }
  // after a wait that ran out: the copies still under way land before the CTA exits
  if (threadIdx.x == 0)
    for (; waited < filled; ++waited)
      if (!tc::mbar_wait(&full[waited % ring], (uint32_t)(waited / ring) & 1u, 1u, err)) break;
  if (!(want & 6)) return;
  // sums that lack rows are not passed on: a NaN, which the gradients' preparation rejects
  if (!ok) {
#pragma unroll
    for (int j = 0; j < NV * P; ++j) dg[j] = db[j] = mk2(__int_as_float(0x7fffffff), __int_as_float(0x7fffffff));
  }
  float* out = part + (int64_t)blockIdx.x * 2 * dim;
  float* comb = reinterpret_cast<float*>(bufs);   // every copy has landed and been read
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    if (!(want & (2 << k))) continue;
    if constexpr (TH > TPR) {
      __syncthreads();
#pragma unroll
      for (int j = 0; j < NV * P; ++j)
        *reinterpret_cast<float2*>(comb + row * (TPR * NV * N) + (col + j / P * TPR) * N + j % P * 2) =
            un2(k ? db[j] : dg[j]);
      __syncthreads();
      for (int c = threadIdx.x; c < dim; c += TH) {
        float v = 0.f;
#pragma unroll 4
        for (int r = 0; r < TH / TPR; ++r) v += comb[r * (TPR * NV * N) + c];
        out[k * dim + c] = v;
      }
    } else {
#pragma unroll
      for (int u = 0; u < NV; ++u) {
        const int i = col + u * TPR;
        if (i >= nvec) continue;
#pragma unroll
        for (int j = 0; j < P; j += 2) {
          const float2 a = un2((k ? db : dg)[u * P + j]), b = un2((k ? db : dg)[u * P + j + 1]);
          *reinterpret_cast<float4*>(out + k * dim + i * N + 2 * j) = make_float4(a.x, a.y, b.x, b.y);
        }
      }
    }
  }
}

// dst[c] += sum over the CTAs of part[CTA][k][c]: interleaved runs in CTA order, then the runs in a
// fixed tree. A thread's whole run, at most ten partials, is in flight at once; few partials take few
// runs (256 x 4096 bf16, dX and both sums: 9.9 us with 32 runs, 7.6 with 8).
constexpr int kRedRun = 10;
constexpr int kRedMost = 2 * 152;   // most CTAs of k_norm_bwd
template <int RUNS>
__global__ void __launch_bounds__(32 * RUNS) k_norm_reduce(const float* __restrict__ part, int n, int dim,
                                                           float* dgamma, float* dbeta) {
  static_assert(RUNS == 8 || RUNS == 32, "a warp adds the runs of 32 / RUNS columns");
  grid_dep_sync();
  __shared__ float sh[RUNS][33];
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + tx;
  float* dst = blockIdx.y ? dbeta : dgamma;
  if (!dst) return;
  const float* p = part + (int64_t)blockIdx.y * dim + c;
  float v[kRedRun];
#pragma unroll
  for (int k = 0; k < kRedRun; ++k) {
    const int i = ty + k * RUNS;
    v[k] = c < dim && i < n ? __ldcg(p + (int64_t)i * 2 * dim) : 0.f;
  }
  float s = 0.f;
#pragma unroll
  for (int k = 0; k < kRedRun; ++k) s += v[k];
  sh[ty][tx] = s;
  __syncthreads();
  // warp ty: columns ty 32 / RUNS .., RUNS lanes each
  const int col = ty * (32 / RUNS) + tx / RUNS, cc = blockIdx.x * 32 + col;
  s = sh[tx % RUNS][col];
#pragma unroll
  for (int o = RUNS / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (tx % RUNS == 0 && cc < dim) dst[cc] += s;
}
static_assert(32 * kRedRun >= kRedMost, "the partials fit the runs");

template <typename E, int WPR, int NV, int R = 1>
cudaError_t fwd_launch(const NormArgs& a, cudaStream_t st) {
  constexpr int rows = kNormThreads / 32 / WPR * R;
  prof_begin(0, st);
  return launch_kernel(k_norm_fwd<E, WPR, NV, R>, (unsigned)((a.T + rows - 1) / rows), kNormThreads,
                       0, st, static_cast<const E*>(a.X), a.gamma, a.beta, static_cast<E*>(a.Y),
                       reinterpret_cast<float2*>(a.stats), a.T, (int)a.dim, 1.f / (float)a.dim,
                       a.eps, a.rms);
}

template <typename E>
cudaError_t fwd_type(const NormArgs& a, cudaStream_t st) {
  const int64_t nvec = a.dim / Pack<E>::N;
  if (nvec <= 32) return fwd_launch<E, 1, 1>(a, st);
  if (nvec <= 64) return fwd_launch<E, 1, 2>(a, st);
  if (a.T > 2048) {
    // Enough rows to fill the SMs: few warps per row. In bf16 two rows share the fp32 weight and
    // shift, which otherwise are four times a row's own bytes through L1 (8192 x 4096: 24.1 us with
    // two rows, 29.0 with one, 28.3 with four, whose registers cost residency; 4096 x 2560: 11.2
    // against 13.1; fp32 8192 x 2048: 22.1 against 21.3).
    constexpr int R = sizeof(E) == 2 ? 2 : 1;
    if (nvec <= 128) return fwd_launch<E, 1, 4, R>(a, st);
    if (nvec <= 256) return fwd_launch<E, 2, 4, R>(a, st);
    if (nvec <= 384) return fwd_launch<E, 4, 3, R>(a, st);
    if (nvec <= 512) return fwd_launch<E, 4, 4, R>(a, st);
  }
  if (nvec <= 256) return fwd_launch<E, 8, 1>(a, st);
  if (nvec <= 512) return fwd_launch<E, 8, 2>(a, st);
  if (nvec <= 1024) return fwd_launch<E, 8, 4>(a, st);
  if (nvec <= 2048) return fwd_launch<E, 8, 8>(a, st);
  if constexpr (sizeof(E) == 4) return fwd_launch<E, 8, 16>(a, st);
  return cudaErrorInvalidValue;   // past LORA_NORM_MAX_DIM
}

template <typename E, int TH, int TPR, int NV, int R>
cudaError_t bwd_launch(const NormArgs& a, int grid, cudaStream_t st) {
  constexpr int RPB = TH / TPR * R;
  static std::atomic<uint64_t> set{0};
  cudaError_t e = once_on_device(set, [] {
    return cudaFuncSetAttribute(k_norm_bwd<E, TH, TPR, NV, R>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                200 * 1024);
  });
  if (e != cudaSuccess) return e;
  const int64_t group = RPB * a.dim * (int64_t)sizeof(E);
  const int ring = bwd_ring(group, TH);
  int64_t smem = 2 * ring * group;
  const int64_t comb = TH > TPR ? (int64_t)TH * NV * Pack<E>::N * 4 : 0;
  if (smem < comb) smem = comb;
  uint32_t* err = tc::error_word();
  if (!err) return cudaErrorInvalidDevice;
  prof_begin(0, st);
  const int want = (a.dX ? 1 : 0) | (a.dgamma ? 2 : 0) | (a.dbeta ? 4 : 0);
  e = launch_kernel(
      k_norm_bwd<E, TH, TPR, NV, R>, (unsigned)grid, TH, (size_t)smem, st, static_cast<const E*>(a.X),
      a.gamma, static_cast<const E*>(a.dY), reinterpret_cast<const float2*>(a.stats),
      static_cast<const E*>(a.dX_add), static_cast<E*>(a.dX), a.part, a.T, (int)a.dim,
      1.f / (float)a.dim, a.rms, want, ring, err, tc_wait_limit());
  if (e != cudaSuccess || !(want & 6)) return e;
  prof_begin(0, st);
  const dim3 blocks((unsigned)((a.dim + 31) / 32), 2);
  return grid <= 8 * kRedRun
             ? launch_kernel(k_norm_reduce<8>, blocks, 256, 0, st, a.part, grid, (int)a.dim, a.dgamma, a.dbeta)
             : launch_kernel(k_norm_reduce<32>, blocks, 1024, 0, st, a.part, grid, (int)a.dim, a.dgamma, a.dbeta);
}

// Threads of a CTA and of a row of a backward pass.
void norm_bwd_shape(int64_t dim, int dtype, int64_t& th, int64_t& tpr) {
  const int64_t nvec = dim / (dtype == LORA_BF16 ? 8 : 4);
  th = nvec <= 512 ? 256 : 512;
  tpr = 32;
  while (2 * tpr < nvec && tpr < th) tpr *= 2;
}

// Rows per thread of a backward pass: two where a CTA has many groups of them, so that a wait and a
// barrier serve both (8192 x 4096 bf16 38.9 -> 35.3 us, 8192 x 2048 fp32 37.9 -> 31.8, 2048 x 4096
// 17.9 -> 17.3; 1023 x 4096 11.8 -> 14.2, 2048 x 1024 7.5 -> 9.3).
int norm_bwd_rows(int64_t dim, int dtype, int64_t T) {
  const int64_t nvec = dim / (dtype == LORA_BF16 ? 8 : 4);
  int64_t th, tpr;
  norm_bwd_shape(dim, dtype, th, tpr);
  return nvec > 32 && nvec <= 512 && T * tpr / th >= 6 * kRedMost ? 2 : 1;
}

template <typename E>
cudaError_t bwd_type(const NormArgs& a, cudaStream_t st) {
  const int64_t nvec = a.dim / Pack<E>::N;
  const int grid = norm_bwd_parts(a.dim, a.dtype, a.T);
  const bool two = norm_bwd_rows(a.dim, a.dtype, a.T) == 2;
  if (nvec <= 32) return bwd_launch<E, 256, 32, 1, 1>(a, grid, st);
  if (nvec <= 64) return two ? bwd_launch<E, 256, 32, 2, 2>(a, grid, st) : bwd_launch<E, 256, 32, 2, 1>(a, grid, st);
  if (nvec <= 128) return two ? bwd_launch<E, 256, 64, 2, 2>(a, grid, st) : bwd_launch<E, 256, 64, 2, 1>(a, grid, st);
  if (nvec <= 256) return two ? bwd_launch<E, 256, 128, 2, 2>(a, grid, st) : bwd_launch<E, 256, 128, 2, 1>(a, grid, st);
  if (nvec <= 512) return two ? bwd_launch<E, 256, 256, 2, 2>(a, grid, st) : bwd_launch<E, 256, 256, 2, 1>(a, grid, st);
  if (nvec <= 1024) return bwd_launch<E, 512, 512, 2, 1>(a, grid, st);
  if (nvec <= 2048) return bwd_launch<E, 512, 512, 4, 1>(a, grid, st);
  if constexpr (sizeof(E) == 4) return bwd_launch<E, 512, 512, 8, 1>(a, grid, st);
  return cudaErrorInvalidValue;   // past LORA_NORM_MAX_DIM
}

}  // namespace

// CTAs (and partials) of a backward pass: two per SM, one where a row takes 512
// threads, and few enough that a CTA has four groups of rows (the partials are 8 bytes per column
// and CTA, a row 6 or 12).
int norm_bwd_parts(int64_t dim, int dtype, int64_t T) {
  int64_t th, tpr;
  norm_bwd_shape(dim, dtype, th, tpr);
  const int64_t per = th / tpr * norm_bwd_rows(dim, dtype, T);
  const int64_t groups = (T + per - 1) / per;
  const int64_t most = th == 256 ? kRedMost : kRedMost / 2;
  const int64_t want = (groups + 3) / 4;
  return (int)(want < most ? want : most);
}

cudaError_t launch_norm_forward(const NormArgs& a, cudaStream_t st) {
  return a.dtype == LORA_BF16 ? fwd_type<__nv_bfloat16>(a, st) : fwd_type<float>(a, st);
}

cudaError_t launch_sum(const SumArgs& a, cudaStream_t st) {
  const int64_t vecs = a.count / (a.dtype == LORA_BF16 ? 8 : 4);
  const unsigned grid = (unsigned)((vecs + kNormThreads - 1) / kNormThreads);
  prof_begin(0, st);
  return a.dtype == LORA_BF16 ? launch_kernel(k_sum<__nv_bfloat16>, grid, kNormThreads, 0, st, a)
                              : launch_kernel(k_sum<float>, grid, kNormThreads, 0, st, a);
}

cudaError_t launch_norm_backward(const NormArgs& a, cudaStream_t st) {
  return a.dtype == LORA_BF16 ? bwd_type<__nv_bfloat16>(a, st) : bwd_type<float>(a, st);
}

}  // namespace lora
