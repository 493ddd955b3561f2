// Norm of each query and key head and rotation by position, forward and backward, and the table of
// cosines and sines.
//
//   forward   r = rsqrt(mean x^2 + eps), h = gamma x r;  (u, v) = (a c - b s, a s + b c) for each pair (a, b) of h
//   backward  h' = the pairs of dy turned back;  dgamma += sum h' x r;  g = gamma h';
//             dx = r (g - x r mean(g x r))
//
// Bound by memory: a head's vector is read once, held in registers by a group of lanes between its sum
// and its outputs, and written once. The statistics are recomputed in the backward pass, which reads x
// anyway, so that the forward pass writes no more than y.
#include "tc_ptx.cuh"

namespace lora {

namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeWarps = kRopeThreads / 32;

struct RopeK {
  const void* x[2];        // q, k
  void* y[2];              // outputs
  const void* dy[2];
  const float* gamma[2];
  int64_t ld_x[2], ld_y[2];
  int heads[2];
  const int32_t* pos;
  const float2* table;
  int64_t T, n_pos;
  int parts;               // warps that share a token's heads
  float eps;
  float* part;             // backward: [CTA][q | k][head_dim] sums of the weights' gradients
};

// A lane's 2 V elements of a head: V from `lane V` of each half.
template <typename E> struct Half;
template <> struct Half<float> {
  static constexpr int V = 4;
  __device__ static void get(const uint4& v, float* f) {
    f[0] = __uint_as_float(v.x); f[1] = __uint_as_float(v.y);
    f[2] = __uint_as_float(v.z); f[3] = __uint_as_float(v.w);
  }
  __device__ static uint4 put(const float* f) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
  }
};
template <> struct Half<__nv_bfloat16> {
  static constexpr int V = 8;
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

template <typename E, int D>
struct RopeShape {
  static constexpr int V = Half<E>::V;
  static constexpr int LPH = D / 2 / V;        // lanes of a head
  static constexpr int HPW = 32 / LPH;         // heads of a warp at a time
  static_assert(LPH >= 1 && LPH <= 32, "a head within a warp");
};

template <int LPH>
__device__ __forceinline__ float head_sum(float v) {
#pragma unroll
  for (int o = LPH / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Cosines and sines of a lane's pairs: HALVES, pair i is element i of both vectors; PAIRS, pair i <
// V / 2 is elements 2 i, 2 i + 1 of the first vector, the others of the second. A position outside the
// table gives NaN.
template <typename E, int D, bool PAIRS>
__device__ __forceinline__ void load_turn(const RopeK& p, int64_t n, int l, float2 (&cs)[Half<E>::V]) {
  constexpr int V = Half<E>::V;
  if (n >= p.n_pos) {
#pragma unroll
    for (int i = 0; i < V; ++i) cs[i] = make_float2(__int_as_float(0x7fffffff), __int_as_float(0x7fffffff));
    return;
  }
  const float2* row = p.table + n * (D / 2);
#pragma unroll
  for (int i = 0; i < V; i += 2) {
    const int at = PAIRS ? (i < V / 2 ? l * (V / 2) + i : D / 4 + l * (V / 2) + i - V / 2) : l * V + i;
    const float4 t = __ldg(reinterpret_cast<const float4*>(row + at));
    cs[i] = make_float2(t.x, t.y);
    cs[i + 1] = make_float2(t.z, t.w);
  }
}

// The pairs of (a | b) turned by the angle (SIGN 1) or back (SIGN -1).
template <int V, bool PAIRS, int SIGN>
__device__ __forceinline__ void turn(float (&f)[2 * V], const float2 (&cs)[V]) {
#pragma unroll
  for (int i = 0; i < V; ++i) {
    float& a = f[PAIRS ? 2 * i : i];
    float& b = f[PAIRS ? 2 * i + 1 : V + i];
    const float c = cs[i].x, s = SIGN * cs[i].y, u = a;
    a = u * c - b * s;
    b = u * s + b * c;
  }
}

template <int V>
__device__ __forceinline__ void load_gamma(const float* g, int l, int half, float (&w)[2 * V]) {
#pragma unroll
  for (int k = 0; k < 2; ++k)
#pragma unroll
    for (int i = 0; i < V; i += 4) load16(g + k * half + l * V + i, w + k * V + i);
}

// A warp takes a share of one token's heads, HPW at a time and R such steps in flight: the token's
// angles and the weights stay in registers over them (they are as many bytes as a head's).
template <typename E, int D, bool PAIRS, bool NORM, int R>
__global__ void __launch_bounds__(kRopeThreads) k_rope_fwd(const __grid_constant__ RopeK p) {
  grid_dep_sync();
  using S = RopeShape<E, D>;
  constexpr int V = S::V;
  const int lane = threadIdx.x & 31, l = lane % S::LPH, sub = lane / S::LPH;
  const int64_t item = (int64_t)blockIdx.x * kRopeWarps + (threadIdx.x >> 5);
  const int64_t t = item / p.parts;
  if (t >= p.T) return;
  const int part = (int)(item - t * p.parts);
  const int64_t n = __ldg(p.pos + t);
  if (n < 0) return;
  float2 cs[V];
  load_turn<E, D, PAIRS>(p, n, l, cs);
#pragma unroll 1
  for (int s = 0; s < 2; ++s) {
    const int steps = (p.heads[s] + S::HPW - 1) / S::HPW;
    float w[2 * V];
    if (NORM && part < steps) load_gamma<V>(p.gamma[s], l, D / 2, w);
    const E* x = static_cast<const E*>(p.x[s]) + t * p.ld_x[s] + l * V;
    E* y = static_cast<E*>(p.y[s]) + t * p.ld_y[s] + l * V;
#pragma unroll 1
    for (int k = part; k < steps; k += R * p.parts) {
      uint4 v[R][2];
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const int h = (k + r * p.parts) * S::HPW + sub;
#pragma unroll
        for (int j = 0; j < 2; ++j)
          v[r][j] = h < p.heads[s] ? *reinterpret_cast<const uint4*>(x + h * D + j * (D / 2)) : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const int h = (k + r * p.parts) * S::HPW + sub;
        float f[2 * V];
        Half<E>::get(v[r][0], f);
        Half<E>::get(v[r][1], f + V);
        if constexpr (NORM) {
          float q = 0.f;
#pragma unroll
          for (int i = 0; i < 2 * V; ++i) q = fmaf(f[i], f[i], q);
          const float rstd = 1.f / sqrtf(head_sum<S::LPH>(q) * (1.f / D) + p.eps);
#pragma unroll
          for (int i = 0; i < 2 * V; ++i) f[i] = f[i] * rstd * w[i];
        }
        turn<V, PAIRS, 1>(f, cs);
        if (h < p.heads[s]) {
          *reinterpret_cast<uint4*>(y + h * D) = Half<E>::put(f);
          *reinterpret_cast<uint4*>(y + h * D + D / 2) = Half<E>::put(f + V);
        }
      }
    }
  }
}

// Persistent over tokens, the query heads of all of them before the key heads, so that a lane keeps one
// weight vector and one vector of its gradient's sums. The CTA's sums go to part[CTA][q | k], added up in
// order by k_rope_reduce.
template <typename E, int D, bool PAIRS, bool NORM, int R>
__global__ void __launch_bounds__(kRopeThreads, 2) k_rope_bwd(const __grid_constant__ RopeK p) {
  grid_dep_sync();
  using S = RopeShape<E, D>;
  constexpr int V = S::V;
  __shared__ float sums[NORM ? kRopeWarps * S::HPW : 1][D];
  const int lane = threadIdx.x & 31, l = lane % S::LPH, sub = lane / S::LPH, warp = threadIdx.x >> 5;
  const int64_t items = p.T * p.parts, step = (int64_t)gridDim.x * kRopeWarps;
#pragma unroll 1
  for (int s = 0; s < 2; ++s) {
    const int steps = (p.heads[s] + S::HPW - 1) / S::HPW;
    float w[2 * V], dg[2 * V];
#pragma unroll
    for (int i = 0; i < 2 * V; ++i) dg[i] = 0.f;
    if (NORM && steps > 0) load_gamma<V>(p.gamma[s], l, D / 2, w);
#pragma unroll 1
    for (int64_t item = (int64_t)blockIdx.x * kRopeWarps + warp; item < items; item += step) {
      const int64_t t = item / p.parts;
      const int part = (int)(item - t * p.parts);
      const int64_t n = __ldg(p.pos + t);
      if (n < 0 || part >= steps) continue;
      float2 cs[V];
      load_turn<E, D, PAIRS>(p, n, l, cs);
      const E* x = static_cast<const E*>(p.x[s]) + t * p.ld_x[s] + l * V;
      E* dx = static_cast<E*>(p.y[s]) + t * p.ld_x[s] + l * V;
      const E* dy = static_cast<const E*>(p.dy[s]) + t * p.ld_y[s] + l * V;
#pragma unroll 1
      for (int k = part; k < steps; k += R * p.parts) {
        uint4 a[R][2], b[R][2];
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const int h = (k + r * p.parts) * S::HPW + sub;
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const bool in = h < p.heads[s];
            b[r][j] = in ? *reinterpret_cast<const uint4*>(dy + h * D + j * (D / 2)) : make_uint4(0, 0, 0, 0);
            if (NORM) a[r][j] = in ? *reinterpret_cast<const uint4*>(x + h * D + j * (D / 2)) : make_uint4(0, 0, 0, 0);
          }
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const int h = (k + r * p.parts) * S::HPW + sub;
          float g[2 * V];
          Half<E>::get(b[r][0], g);
          Half<E>::get(b[r][1], g + V);
          turn<V, PAIRS, -1>(g, cs);
          if constexpr (NORM) {
            float f[2 * V];
            Half<E>::get(a[r][0], f);
            Half<E>::get(a[r][1], f + V);
            float q = 0.f, z = 0.f;
#pragma unroll
            for (int i = 0; i < 2 * V; ++i) q = fmaf(f[i], f[i], q);
            const float rstd = 1.f / sqrtf(head_sum<S::LPH>(q) * (1.f / D) + p.eps);
            const bool in = h < p.heads[s];   // (a NaN angle times a missing head's zeros is none of a sum's)
#pragma unroll
            for (int i = 0; i < 2 * V; ++i) {
              f[i] *= rstd;
              if (in) dg[i] = fmaf(g[i], f[i], dg[i]);
              g[i] *= w[i];
              z = fmaf(g[i], f[i], z);
            }
            z = head_sum<S::LPH>(z) * (1.f / D);
#pragma unroll
            for (int i = 0; i < 2 * V; ++i) g[i] = (g[i] - f[i] * z) * rstd;
          }
          if (h < p.heads[s]) {
            *reinterpret_cast<uint4*>(dx + h * D) = Half<E>::put(g);
            *reinterpret_cast<uint4*>(dx + h * D + D / 2) = Half<E>::put(g + V);
          }
        }
      }
    }
    if constexpr (NORM) {
      __syncthreads();   // the sums of the query heads have been read
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int i = 0; i < V; ++i) sums[warp * S::HPW + sub][k * (D / 2) + l * V + i] = dg[k * V + i];
      __syncthreads();
      for (int c = threadIdx.x; c < D; c += kRopeThreads) {
        float v = 0.f;
#pragma unroll 8
        for (int r = 0; r < kRopeWarps * S::HPW; ++r) v += sums[r][c];
        p.part[((int64_t)blockIdx.x * 2 + s) * D + c] = v;
      }
    }
  }
}

// dgamma[c] += sum over the CTAs, interleaved runs of CTAs in order, then the runs in a fixed tree.
constexpr int kRopeRuns = 32;
__global__ void __launch_bounds__(32 * kRopeRuns) k_rope_reduce(const float* __restrict__ part, int n, int D,
                                                                float* dgq, float* dgk) {
  grid_dep_sync();
  __shared__ float sh[kRopeRuns][33];
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  float* dst = blockIdx.y ? dgk : dgq;
  if (!dst) return;
  const float* src = part + (int64_t)blockIdx.y * D + blockIdx.x * 32;
  float v = 0.f;
#pragma unroll 4
  for (int i = ty; i < n; i += kRopeRuns) v += __ldcg(src + (int64_t)i * 2 * D + tx);
  sh[ty][tx] = v;
  __syncthreads();
  v = sh[tx][ty];   // warp ty: the runs of column ty
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (tx == 0) dst[blockIdx.x * 32 + ty] += v;
}

__global__ void k_rope_table(int64_t n_pos, int half, const double* __restrict__ inv_freq, float2* __restrict__ table) {
  grid_dep_sync();
  const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= n_pos * half) return;
  const int64_t n = i / half;
  double s, c;
  sincos((double)n * inv_freq[i - n * half], &s, &c);
  table[i] = make_float2((float)c, (float)s);
}

// Warps that share a token: one per token where the tokens fill the SMs with warps, as many as the
// token has steps where there are few (one decoded token is bound by latency).
int rope_parts(const RopeArgs& a, int hpw, int sms) {
  const int64_t want = (int64_t)sms * 16;
  int64_t n = a.T >= want ? 1 : (want + a.T - 1) / a.T;
  const int most = (a.heads[0] > a.heads[1] ? a.heads[0] : a.heads[1]) + hpw - 1;
  if (n > most / hpw) n = most / hpw;
  return (int)(n < 1 ? 1 : n);
}

RopeK rope_args(const RopeArgs& a, int parts) {
  RopeK k{};
  for (int s = 0; s < 2; ++s) {
    k.x[s] = a.x[s]; k.y[s] = a.y[s]; k.dy[s] = a.dy[s]; k.gamma[s] = a.gamma[s];
    k.ld_x[s] = a.ld_x[s]; k.ld_y[s] = a.ld_y[s]; k.heads[s] = a.heads[s];
  }
  k.pos = a.pos; k.table = reinterpret_cast<const float2*>(a.table);
  k.T = a.T; k.n_pos = a.n_pos; k.eps = a.eps; k.part = a.part; k.parts = parts;
  return k;
}

template <typename E, int D, bool PAIRS, bool NORM>
cudaError_t rope_launch(const RopeArgs& a, bool bwd, cudaStream_t st) {
  using S = RopeShape<E, D>;
  const int sms = tc::sm_count();
  if (sms <= 0) return cudaErrorInvalidDevice;
  const RopeK k = rope_args(a, rope_parts(a, S::HPW, sms));
  const int64_t blocks = (a.T * k.parts + kRopeWarps - 1) / kRopeWarps;
  prof_begin(0, st);
  if (!bwd) return launch_kernel(k_rope_fwd<E, D, PAIRS, NORM, 2>, (unsigned)blocks, kRopeThreads, 0, st, k);
  const unsigned grid = (unsigned)(blocks < kRopeMostCtas ? blocks : kRopeMostCtas);
  cudaError_t e = launch_kernel(k_rope_bwd<E, D, PAIRS, NORM, 2>, grid, kRopeThreads, 0, st, k);
  if (e != cudaSuccess || !NORM || (!a.dgamma[0] && !a.dgamma[1])) return e;
  prof_begin(0, st);
  return launch_kernel(k_rope_reduce, dim3(D / 32, 2), 32 * kRopeRuns, 0, st, (const float*)a.part, (int)grid, D,
                       a.dgamma[0], a.heads[1] ? a.dgamma[1] : (float*)nullptr);
}

template <typename E, int D>
cudaError_t rope_dim(const RopeArgs& a, bool bwd, cudaStream_t st) {
  if (a.gamma[0]) return a.pairs ? rope_launch<E, D, true, true>(a, bwd, st) : rope_launch<E, D, false, true>(a, bwd, st);
  return a.pairs ? rope_launch<E, D, true, false>(a, bwd, st) : rope_launch<E, D, false, false>(a, bwd, st);
}

template <typename E>
cudaError_t rope_type(const RopeArgs& a, bool bwd, cudaStream_t st) {
  if (a.dim == 64) return rope_dim<E, 64>(a, bwd, st);
  if (a.dim == 128) return rope_dim<E, 128>(a, bwd, st);
  return rope_dim<E, 256>(a, bwd, st);
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& a, bool bwd, cudaStream_t st) {
  return a.dtype == LORA_BF16 ? rope_type<__nv_bfloat16>(a, bwd, st) : rope_type<float>(a, bwd, st);
}

cudaError_t launch_rope_table(int64_t n_pos, int dim, const double* inv_freq, float* table, cudaStream_t st) {
  const int64_t n = n_pos * (dim / 2);
  prof_begin(0, st);
  return launch_kernel(k_rope_table, (unsigned)((n + 255) / 256), 256, 0, st, n_pos, dim / 2, inv_freq,
                       reinterpret_cast<float2*>(table));
}

}  // namespace lora
