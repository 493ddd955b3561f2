// Layer norm and root-mean-square norm in front of an adapted linear: forward, and the backward
// pass with the token sums of the weight's and the shift's gradients.
//
//   forward   xhat = (x - mean) rstd,  Y = gamma xhat + beta
//   backward  g = gamma dY,  dX = rstd (g - sum g / dim - xhat (sum g xhat) / dim)   (RMS: without
//             the sum of g),  dgamma += sum_t dY xhat,  dbeta += sum_t dY
//
// Both passes are bound by memory: a row is read once, held in registers between its sums and its
// outputs, and written once.
#include "lora_kernels.h"

namespace lora {

namespace {

constexpr int kNormThreads = 256;

template <typename E> struct Pack;
template <> struct Pack<float> {
  static constexpr int N = 4;
  __device__ static void get(const uint4& v, float* f) {
    f[0] = __uint_as_float(v.x); f[1] = __uint_as_float(v.y);
    f[2] = __uint_as_float(v.z); f[3] = __uint_as_float(v.w);
  }
  __device__ static uint4 put(const float* f) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                      __float_as_uint(f[3]));
  }
};
template <> struct Pack<__nv_bfloat16> {
  static constexpr int N = 8;
  __device__ static void get(const uint4& v, float* f) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      f[2 * j] = __uint_as_float(w[j] << 16);
      f[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
    }
  }
  __device__ static uint4 put(const float* f) {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * j], f[2 * j + 1]);
      w[j] = *reinterpret_cast<const uint32_t*>(&h);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Sum over the WPR warps of a row, the same in every lane. `sh` holds one float per warp; the
// caller alternates two buffers so that one barrier per sum suffices.
template <int WPR>
__device__ __forceinline__ float row_sum(float v, float* sh) {
  v = warp_sum(v);
  if constexpr (WPR > 1) {
    const int warp = threadIdx.x >> 5;
    if ((threadIdx.x & 31) == 0) sh[warp] = v;
    __syncthreads();
    const int w0 = warp / WPR * WPR;
    v = 0.f;
#pragma unroll
    for (int w = 0; w < WPR; ++w) v += sh[w0 + w];
  }
  return v;
}

// WPR warps per row, NV 16-byte vectors per lane, 8 / WPR rows per CTA.
template <typename E, int WPR, int NV>
__global__ void __launch_bounds__(kNormThreads) k_norm_fwd(const E* __restrict__ X,
                                                           const float* __restrict__ gamma,
                                                           const float* __restrict__ beta,
                                                           E* __restrict__ Y,
                                                           float2* __restrict__ stats, int64_t T,
                                                           int dim, float inv_dim, float eps,
                                                           int rms) {
  grid_dep_sync();
  constexpr int N = Pack<E>::N;
  __shared__ float sh[2][kNormThreads / 32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t t = (int64_t)blockIdx.x * (kNormThreads / 32 / WPR) + warp / WPR;
  const bool live = t < T;
  const int nvec = dim / N;
  const int first = (warp % WPR) * 32 + lane;
  const uint4* src = reinterpret_cast<const uint4*>(X + t * dim);
  uint4 v[NV];
  float s = 0.f;
#pragma unroll
  for (int u = 0; u < NV; ++u) {
    const int i = first + u * 32 * WPR;
    v[u] = live && i < nvec ? __ldg(src + i) : make_uint4(0, 0, 0, 0);
  }
  float mean = 0.f;
  if (!rms) {
#pragma unroll
    for (int u = 0; u < NV; ++u) {
      float f[N];
      Pack<E>::get(v[u], f);
#pragma unroll
      for (int j = 0; j < N; ++j) s += f[j];
    }
    mean = row_sum<WPR>(s, sh[0]) * inv_dim;
  }
  s = 0.f;
#pragma unroll
  for (int u = 0; u < NV; ++u) {
    const int i = first + u * 32 * WPR;
    if (i < nvec) {
      float f[N];
      Pack<E>::get(v[u], f);
#pragma unroll
      for (int j = 0; j < N; ++j) s = fmaf(f[j] - mean, f[j] - mean, s);
    }
  }
  const float var = row_sum<WPR>(s, sh[1]) * inv_dim;
  const float rstd = 1.f / sqrtf(var + eps);
  if (!live) return;
  if (first == 0) stats[t] = make_float2(mean, rstd);
  uint4* dst = reinterpret_cast<uint4*>(Y + t * dim);
#pragma unroll
  for (int u = 0; u < NV; ++u) {
    const int i = first + u * 32 * WPR;
    if (i >= nvec) continue;
    float f[N], ga[N], be[N];
    Pack<E>::get(v[u], f);
#pragma unroll
    for (int j = 0; j < N; j += 4) {
      load16(gamma + i * N + j, ga + j);
      if (beta) load16(beta + i * N + j, be + j);
    }
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const float h = (f[j] - mean) * rstd;
      f[j] = beta ? fmaf(h, ga[j], be[j]) : h * ga[j];
    }
    dst[i] = Pack<E>::put(f);
  }
}

constexpr int kBwdThreads = 512;

// TPR threads per row, NV vectors per thread, kBwdThreads / TPR rows at a time; persistent over
// the rows, so that a thread keeps its columns and sums their gradients in registers. The next
// rows are loaded ahead of the current rows' sums. Partials go to part[CTA][2][dim], added up in
// order by k_norm_reduce.
template <typename E, int TPR, int NV>
__global__ void __launch_bounds__(kBwdThreads, NV == 1 ? 2 : 1)
    k_norm_bwd(const E* __restrict__ X, const float* __restrict__ gamma, const E* __restrict__ dY,
               const float2* __restrict__ stats, const E* dX_add, E* dX, float* __restrict__ part,
               int64_t T, int dim, float inv_dim, int rms, int want) {
  grid_dep_sync();
  constexpr int N = Pack<E>::N;
  constexpr int RPB = kBwdThreads / TPR;
  constexpr int WPR = TPR / 32;
  __shared__ float2 sh[2][kBwdThreads / 32];
  __shared__ float comb[RPB > 1 ? kBwdThreads * NV * N : 1];
  const int row = threadIdx.x / TPR, col = threadIdx.x % TPR;
  const int warp = threadIdx.x >> 5;
  const int nvec = dim / N;
  float dg[NV * N], db[NV * N];
#pragma unroll
  for (int j = 0; j < NV * N; ++j) dg[j] = db[j] = 0.f;
  uint4 xv[NV], yv[NV];
  float2 st = make_float2(0.f, 0.f);
  const int64_t step = (int64_t)gridDim.x * RPB;
  const int64_t t_first = (int64_t)blockIdx.x * RPB;
  auto load = [&](int64_t t) {
#pragma unroll
    for (int u = 0; u < NV; ++u) {
      const int i = col + u * TPR;
      const bool in = t < T && i < nvec;
      xv[u] = in ? __ldcs(reinterpret_cast<const uint4*>(X + t * dim) + i) : make_uint4(0, 0, 0, 0);
      yv[u] = in ? __ldcs(reinterpret_cast<const uint4*>(dY + t * dim) + i) : make_uint4(0, 0, 0, 0);
    }
    st = t < T ? __ldg(stats + t) : make_float2(0.f, 0.f);
  };
  load(t_first + row);
  int buf = 0;
  for (int64_t t0 = t_first; t0 < T; t0 += step, buf ^= 1) {
    const int64_t t = t0 + row;
    uint4 xc[NV], yc[NV];
    const float2 sc = st;
#pragma unroll
    for (int u = 0; u < NV; ++u) { xc[u] = xv[u]; yc[u] = yv[u]; }
    if (t0 + step < T) load(t + step);
    float s1 = 0.f, s2 = 0.f;   // sum g, sum g xhat
#pragma unroll
    for (int u = 0; u < NV; ++u) {
      const int i = col + u * TPR;
      if (i >= nvec) continue;
      float x[N], y[N], ga[N];
      Pack<E>::get(xc[u], x);
      Pack<E>::get(yc[u], y);
#pragma unroll
      for (int j = 0; j < N; j += 4) load16(gamma + i * N + j, ga + j);
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const float h = (x[j] - sc.x) * sc.y;
        const float g = y[j] * ga[j];
        s1 += g;
        s2 = fmaf(g, h, s2);
        dg[u * N + j] = fmaf(y[j], h, dg[u * N + j]);
        db[u * N + j] += y[j];
      }
    }
    if (!(want & 1)) continue;   // no dX: the rows' sums are not needed
    s1 = warp_sum(s1);
    s2 = warp_sum(s2);
    if constexpr (WPR > 1) {
      if ((threadIdx.x & 31) == 0) sh[buf][warp] = make_float2(s1, s2);
      __syncthreads();
      const int w0 = warp / WPR * WPR;
      s1 = s2 = 0.f;
#pragma unroll
      for (int w = 0; w < WPR; ++w) {
        s1 += sh[buf][w0 + w].x;
        s2 += sh[buf][w0 + w].y;
      }
    }
    if (t >= T) continue;
    s1 = rms ? 0.f : s1 * inv_dim;
    s2 *= inv_dim;
#pragma unroll
    for (int u = 0; u < NV; ++u) {
      const int i = col + u * TPR;
      if (i >= nvec) continue;
      float x[N], y[N], ga[N], add[N];
      Pack<E>::get(xc[u], x);
      Pack<E>::get(yc[u], y);
#pragma unroll
      for (int j = 0; j < N; j += 4) load16(gamma + i * N + j, ga + j);
      if (dX_add) Pack<E>::get(*(reinterpret_cast<const uint4*>(dX_add + t * dim) + i), add);
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const float h = (x[j] - sc.x) * sc.y;
        const float d = (y[j] * ga[j] - s1 - h * s2) * sc.y;
        x[j] = dX_add ? d + add[j] : d;
      }
      *(reinterpret_cast<uint4*>(dX + t * dim) + i) = Pack<E>::put(x);
    }
  }
  if (!(want & 6)) return;
  float* out = part + (int64_t)blockIdx.x * 2 * dim;
  for (int k = 0; k < 2; ++k) {
    if (!(want & (2 << k))) continue;
    const float* acc = k ? db : dg;
    if constexpr (RPB > 1) {
      __syncthreads();
#pragma unroll
      for (int j = 0; j < NV * N; ++j)
        comb[row * (TPR * NV * N) + (col + j / N * TPR) * N + j % N] = k ? db[j] : dg[j];
      __syncthreads();
      for (int c = threadIdx.x; c < dim; c += kBwdThreads) {
        float s = 0.f;
#pragma unroll 4
        for (int r = 0; r < RPB; ++r) s += comb[r * (TPR * NV * N) + c];
        out[k * dim + c] = s;
      }
    } else {
      (void)acc;
#pragma unroll
      for (int u = 0; u < NV; ++u) {
        const int i = col + u * TPR;
        if (i >= nvec) continue;
#pragma unroll
        for (int j = 0; j < N; j += 4)
          store4(out + k * dim + i * N + j, (k ? db : dg) + u * N + j);
      }
    }
  }
}

// dst[c] += sum over the CTAs of part[CTA][k][c], in CTA order within each of 8 interleaved runs,
// then the runs in order.
__global__ void __launch_bounds__(256) k_norm_reduce(const float* __restrict__ part, int n, int dim,
                                                     float* dgamma, float* dbeta) {
  grid_dep_sync();
  __shared__ float sh[8][33];
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + tx;
  float* dst = blockIdx.y ? dbeta : dgamma;
  if (!dst) return;
  float s = 0.f;
  if (c < dim) {
    const float* p = part + (int64_t)blockIdx.y * dim + c;
#pragma unroll 4
    for (int i = ty; i < n; i += 8) s += __ldcg(p + (int64_t)i * 2 * dim);
  }
  sh[ty][tx] = s;
  __syncthreads();
  if (ty == 0 && c < dim) {
    s = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) s += sh[k][tx];
    dst[c] += s;
  }
}

template <typename E, int WPR, int NV>
cudaError_t fwd_launch(const NormArgs& a, cudaStream_t st) {
  constexpr int rows = kNormThreads / 32 / WPR;
  prof_begin(0, st);
  return launch_kernel(k_norm_fwd<E, WPR, NV>, (unsigned)((a.T + rows - 1) / rows), kNormThreads,
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
    if (nvec <= 128) return fwd_launch<E, 1, 4>(a, st);
    if (nvec <= 256) return fwd_launch<E, 2, 4>(a, st);
    if (nvec <= 512) return fwd_launch<E, 4, 4>(a, st);
  }
  if (nvec <= 256) return fwd_launch<E, 8, 1>(a, st);
  if (nvec <= 512) return fwd_launch<E, 8, 2>(a, st);
  if (nvec <= 1024) return fwd_launch<E, 8, 4>(a, st);
  if (nvec <= 2048) return fwd_launch<E, 8, 8>(a, st);
  return fwd_launch<E, 8, 16>(a, st);
}

template <typename E, int TPR, int NV>
cudaError_t bwd_launch(const NormArgs& a, int grid, cudaStream_t st) {
  prof_begin(0, st);
  const int want = (a.dX ? 1 : 0) | (a.dgamma ? 2 : 0) | (a.dbeta ? 4 : 0);
  cudaError_t e = launch_kernel(
      k_norm_bwd<E, TPR, NV>, (unsigned)grid, kBwdThreads, 0, st, static_cast<const E*>(a.X),
      a.gamma, static_cast<const E*>(a.dY), reinterpret_cast<const float2*>(a.stats),
      static_cast<const E*>(a.dX_add), static_cast<E*>(a.dX), a.part, a.T, (int)a.dim,
      1.f / (float)a.dim, a.rms, want);
  if (e != cudaSuccess || !(want & 6)) return e;
  prof_begin(0, st);
  return launch_kernel(k_norm_reduce, dim3((unsigned)((a.dim + 31) / 32), 2), 256, 0, st, a.part,
                       grid, (int)a.dim, a.dgamma, a.dbeta);
}

template <typename E>
cudaError_t bwd_type(const NormArgs& a, cudaStream_t st) {
  const int64_t nvec = a.dim / Pack<E>::N;
  const int grid = norm_bwd_parts(a.dim, a.dtype, a.T);
  if (nvec <= 32) return bwd_launch<E, 32, 1>(a, grid, st);
  if (nvec <= 64) return bwd_launch<E, 64, 1>(a, grid, st);
  if (nvec <= 128) return bwd_launch<E, 128, 1>(a, grid, st);
  if (nvec <= 256) return bwd_launch<E, 256, 1>(a, grid, st);
  if (nvec <= 512) return bwd_launch<E, 512, 1>(a, grid, st);
  if (nvec <= 1024) return bwd_launch<E, 512, 2>(a, grid, st);
  if (nvec <= 2048) return bwd_launch<E, 512, 4>(a, grid, st);
  return bwd_launch<E, 512, 8>(a, grid, st);
}

}  // namespace

int norm_bwd_parts(int64_t dim, int dtype, int64_t T) {
  const int64_t nvec = dim / (dtype == LORA_BF16 ? 8 : 4);
  int64_t tpr = 32;
  while (tpr < nvec && tpr < kBwdThreads) tpr *= 2;
  const int64_t groups = (T * tpr + kBwdThreads - 1) / kBwdThreads;
  const int64_t most = nvec <= kBwdThreads ? 2 * 152 : 152;
  return (int)(groups < most ? groups : most);
}

cudaError_t launch_norm_forward(const NormArgs& a, cudaStream_t st) {
  return a.dtype == LORA_BF16 ? fwd_type<__nv_bfloat16>(a, st) : fwd_type<float>(a, st);
}

cudaError_t launch_norm_backward(const NormArgs& a, cudaStream_t st) {
  return a.dtype == LORA_BF16 ? bwd_type<__nv_bfloat16>(a, st) : bwd_type<float>(a, st);
}

}  // namespace lora
