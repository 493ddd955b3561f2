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
#include "attn_common.cuh"

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

using attn::f2;
using attn::add2;
using attn::fma2;
using attn::mk2;
using attn::mul2;
using attn::un2;

// A lane's 2 V elements of a head: V = 4 from `lane V` of each half, as packed pairs of neighbours (one instruction
// for two elements). In bf16 that is 8 bytes of each half. With 16 the same bytes in flight (two steps of a warp for
// four) do not fit the registers that the CTAs per SM leave, 64 forward and 128 backward: a lane's vectors, angles,
// weights and sums spill 148 and 216 bytes. 8192 tokens of 40 heads of 128: 39.9 and 63.0 us against 29.6 and 49.9; with
// one step in flight 35.2 and 57.9.
template <typename E> struct Half;
template <> struct Half<float> {
  static constexpr int V = 4;
  using raw = uint4;
  __device__ static raw none() { return make_uint4(0, 0, 0, 0); }
  __device__ static void get(const raw& v, f2* f) {
    f[0] = mk2(__uint_as_float(v.x), __uint_as_float(v.y));
    f[1] = mk2(__uint_as_float(v.z), __uint_as_float(v.w));
  }
  __device__ static raw put(const f2* f) {
    const float2 a = un2(f[0]), b = un2(f[1]);
    return make_uint4(__float_as_uint(a.x), __float_as_uint(a.y), __float_as_uint(b.x), __float_as_uint(b.y));
  }
};
template <> struct Half<__nv_bfloat16> {
  static constexpr int V = 4;
  using raw = uint2;
  __device__ static raw none() { return make_uint2(0, 0); }
  __device__ static void get(const raw& v, f2* f) {
    f[0] = mk2(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xFFFF0000u));
    f[1] = mk2(__uint_as_float(v.y << 16), __uint_as_float(v.y & 0xFFFF0000u));
  }
  __device__ static raw put(const f2* f) {
    const float2 a = un2(f[0]), b = un2(f[1]);
    return make_uint2(attn::pack_bf16(a.x, a.y), attn::pack_bf16(b.x, b.y));
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
__device__ __forceinline__ float sum2(f2 v) {
  const float2 a = un2(v);
  return a.x + a.y;
}

// Cosines and sines of a lane's pairs. HALVES: pair i is element i of both vectors; c and s hold the cosines and
// the sines of two neighbouring pairs. PAIRS: pair i < V / 2 is elements 2 i, 2 i + 1 of the
// first vector, the others of the second; c holds a pair's cosine and sine. A position outside the table gives NaN.
template <typename E, int D, bool PAIRS>
struct Turn {
  static constexpr int V = Half<E>::V;
  f2 c[PAIRS ? V : V / 2], s[PAIRS ? 1 : V / 2];
  __device__ void load(const RopeK& p, int64_t pos, int l) {
    const float2* row = p.table + pos * (D / 2);
    const bool in = pos < p.n_pos;
    const float nan = __int_as_float(0x7fffffff);
#pragma unroll
    for (int i = 0; i < V; i += 2) {
      const int at = PAIRS ? (i < V / 2 ? l * (V / 2) + i : D / 4 + l * (V / 2) + i - V / 2) : l * V + i;
      const float4 t = in ? __ldg(reinterpret_cast<const float4*>(row + at)) : make_float4(nan, nan, nan, nan);
      if constexpr (PAIRS) {
        c[i] = mk2(t.x, t.y);
        c[i + 1] = mk2(t.z, t.w);
      } else {
        c[i / 2] = mk2(t.x, t.z);
        s[i / 2] = mk2(t.y, t.w);
      }
    }
  }
  // the pairs of f turned by the angle (BACK: by its negative)
  template <bool BACK>
  __device__ void apply(f2 (&f)[V]) const {
    if constexpr (PAIRS) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float2 x = un2(f[i]), t = un2(c[i]);
        const float z = BACK ? -t.y : t.y;
        f[i] = mk2(x.x * t.x - x.y * z, x.x * z + x.y * t.x);
      }
    } else {
#pragma unroll
      for (int i = 0; i < V / 2; ++i) {
        const f2 a = f[i], b = f[V / 2 + i], n = s[i] ^ 0x8000000080000000ull;   // - the sines
        f[i] = fma2(b, BACK ? s[i] : n, mul2(a, c[i]));
        f[V / 2 + i] = fma2(a, BACK ? n : s[i], mul2(b, c[i]));
      }
    }
  }
};

template <int V>
__device__ __forceinline__ void load_gamma(const float* g, int l, int half, f2 (&w)[V]) {
#pragma unroll
  for (int k = 0; k < 2; ++k)
#pragma unroll
    for (int i = 0; i < V; i += 4) {
      const float4 t = __ldg(reinterpret_cast<const float4*>(g + k * half + l * V + i));
      w[(k * V + i) / 2] = mk2(t.x, t.y);
      w[(k * V + i) / 2 + 1] = mk2(t.z, t.w);
    }
}

// A warp takes a share of one token's heads, HPW at a time and R such steps in flight: the token's
// angles and the weights stay in registers over them (they are as many bytes as a head's). 8192 tokens of 40 heads of
// 128: 29.6 us in bf16, 5.8 TB/s (20 bytes are reloaded at 64 registers), 53.4 in fp32, 6.4 TB/s; bf16 with two steps
// in flight and three CTAs per SM, so measured earlier, 39.8.
template <typename E, int D, bool PAIRS, bool NORM, int R>
__global__ void __launch_bounds__(kRopeThreads, 4) k_rope_fwd(const __grid_constant__ RopeK p) {
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
  Turn<E, D, PAIRS> turn;
  turn.load(p, n, l);
#pragma unroll 1
  for (int s = 0; s < 2; ++s) {
    const int steps = (p.heads[s] + S::HPW - 1) / S::HPW;
    f2 w[V];
    if (NORM && part < steps) load_gamma<V>(p.gamma[s], l, D / 2, w);
    const E* x = static_cast<const E*>(p.x[s]) + t * p.ld_x[s] + l * V;
    E* y = static_cast<E*>(p.y[s]) + t * p.ld_y[s] + l * V;
#pragma unroll 1
    for (int k = part; k < steps; k += R * p.parts) {
      typename Half<E>::raw v[R][2];
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const int h = (k + r * p.parts) * S::HPW + sub;
#pragma unroll
        for (int j = 0; j < 2; ++j)
          v[r][j] = h < p.heads[s] ? *reinterpret_cast<const typename Half<E>::raw*>(x + h * D + j * (D / 2)) : Half<E>::none();
      }
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const int h = (k + r * p.parts) * S::HPW + sub;
        f2 f[V];
        Half<E>::get(v[r][0], f);
        Half<E>::get(v[r][1], f + V / 2);
        if constexpr (NORM) {
          f2 q = mul2(f[0], f[0]);
#pragma unroll
          for (int i = 1; i < V; ++i) q = fma2(f[i], f[i], q);
          const float rstd = rsqrtf(head_sum<S::LPH>(sum2(q)) * (1.f / D) + p.eps);
          const f2 r2 = mk2(rstd, rstd);
#pragma unroll
          for (int i = 0; i < V; ++i) f[i] = mul2(mul2(f[i], r2), w[i]);
        }
        turn.template apply<false>(f);
        if (h < p.heads[s]) {
          *reinterpret_cast<typename Half<E>::raw*>(y + h * D) = Half<E>::put(f);
          *reinterpret_cast<typename Half<E>::raw*>(y + h * D + D / 2) = Half<E>::put(f + V / 2);
        }
      }
    }
  }
}

// Persistent over tokens, the query heads of all of them before the key heads, so that a lane keeps one weight
// vector and one vector of its gradient's sums. Both sums of a head, x^2 and (gamma h') x, are taken before rstd is
// known, so that their shuffles run together. The CTA's sums go to part[CTA][q | k], added up in order by
// k_rope_reduce.
//
// 8192 tokens of 40 heads of 128: 49.9 us in bf16, 5.1 TB/s, 80.3 in fp32, 6.4 TB/s; 51.0 and 82.9 with the reduction. In
// bf16 two CTAs of 256 threads per SM (128 registers) wait for their loads and compute in turn: issue slots are 44% busy,
// and long_scoreboard is the largest stall. 59.5 for a call with two copies of the weights' gradients ahead of it; so
// measured, two steps in flight instead of four take 68 us, three CTAs per SM 75, rows brought by bulk copies to per-warp
// rings in shared memory 72. 1023 tokens of 36 heads of 64 in fp32: 7.7 us and 2.2 for the reduction, the latency of two
// launches with one round of warps.
template <typename E, int D, bool PAIRS, bool NORM, int R>
__global__ void __launch_bounds__(kRopeThreads, 2) k_rope_bwd(const __grid_constant__ RopeK p) {
  grid_dep_sync();
  using S = RopeShape<E, D>;
  using raw = typename Half<E>::raw;
  constexpr int V = S::V;
  __shared__ float sums[NORM ? kRopeWarps * S::HPW : 1][D];
  const int lane = threadIdx.x & 31, l = lane % S::LPH, sub = lane / S::LPH, warp = threadIdx.x >> 5;
  const int64_t items = p.T * p.parts, step = (int64_t)gridDim.x * kRopeWarps;
#pragma unroll 1
  for (int s = 0; s < 2; ++s) {
    const int steps = (p.heads[s] + S::HPW - 1) / S::HPW;
    f2 w[V], dg[V];
#pragma unroll
    for (int i = 0; i < V; ++i) dg[i] = mk2(0.f, 0.f);
    if (NORM && steps > 0) load_gamma<V>(p.gamma[s], l, D / 2, w);
#pragma unroll 1
    for (int64_t item = (int64_t)blockIdx.x * kRopeWarps + warp; item < items; item += step) {
      const int64_t t = item / p.parts;
      const int part = (int)(item - t * p.parts);
      const int64_t n = __ldg(p.pos + t);
      if (n < 0 || part >= steps) continue;
      Turn<E, D, PAIRS> turn;
      turn.load(p, n, l);
      const E* x = static_cast<const E*>(p.x[s]) + t * p.ld_x[s] + l * V;
      E* dx = static_cast<E*>(p.y[s]) + t * p.ld_x[s] + l * V;
      const E* dy = static_cast<const E*>(p.dy[s]) + t * p.ld_y[s] + l * V;
#pragma unroll 1
      for (int k = part; k < steps; k += R * p.parts) {
        raw a[R][2], b[R][2];
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const int h = (k + r * p.parts) * S::HPW + sub;
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const bool in = h < p.heads[s];
            b[r][j] = in ? *reinterpret_cast<const raw*>(dy + h * D + j * (D / 2)) : Half<E>::none();
            if (NORM) a[r][j] = in ? *reinterpret_cast<const raw*>(x + h * D + j * (D / 2)) : Half<E>::none();
          }
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const int h = (k + r * p.parts) * S::HPW + sub;
          const bool in = h < p.heads[s];
          f2 g[V];
          Half<E>::get(b[r][0], g);
          Half<E>::get(b[r][1], g + V / 2);
          turn.template apply<true>(g);
          if constexpr (NORM) {
            f2 f[V];
            Half<E>::get(a[r][0], f);
            Half<E>::get(a[r][1], f + V / 2);
            f2 q = mul2(f[0], f[0]), z = mul2(mul2(g[0], w[0]), f[0]);
#pragma unroll
            for (int i = 1; i < V; ++i) {
              q = fma2(f[i], f[i], q);
              z = fma2(mul2(g[i], w[i]), f[i], z);
            }
            const float qs = head_sum<S::LPH>(sum2(q)), zs = head_sum<S::LPH>(sum2(z));
            const float rstd = rsqrtf(qs * (1.f / D) + p.eps);
            const float m = -rstd * zs * (1.f / D);   // - (sum gamma h' xhat) / dim
            const f2 r2 = mk2(rstd, rstd), m2 = mk2(m, m);
#pragma unroll
            for (int i = 0; i < V; ++i) {
              f[i] = mul2(f[i], r2);
              if (in) dg[i] = fma2(g[i], f[i], dg[i]);   // (a NaN angle times a missing head's zeros is none of a sum's)
              g[i] = mul2(fma2(f[i], m2, mul2(g[i], w[i])), r2);
            }
          }
          if (in) {
            *reinterpret_cast<raw*>(dx + h * D) = Half<E>::put(g);
            *reinterpret_cast<raw*>(dx + h * D + D / 2) = Half<E>::put(g + V / 2);
          }
        }
      }
    }
    if constexpr (NORM) {
      __syncthreads();   // the sums of the query heads have been read
#pragma unroll
      for (int i = 0; i < V; ++i)
        *reinterpret_cast<float2*>(&sums[warp * S::HPW + sub][2 * i / V * (D / 2) + l * V + 2 * i % V]) = un2(dg[i]);
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

// dgamma[c] += sum over the CTAs: interleaved runs of CTAs in order, a run's partials all under way at once, then
// the runs in a fixed tree. A CTA takes 32 columns of one weight, or, where both weights' gradients are one array, of
// both, one after the other.
constexpr int kRopeRuns = 32;
__global__ void __launch_bounds__(32 * kRopeRuns) k_rope_reduce(const float* __restrict__ part, int n, int D,
                                                                float* dgq, float* dgk) {
  grid_dep_sync();
  constexpr int kRun = (kRopeMostCtas + kRopeRuns - 1) / kRopeRuns;
  __shared__ float sh[kRopeRuns][33];
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
#pragma unroll 1
  for (int s = blockIdx.y; s < 2; s += gridDim.y) {
    float* dst = s ? dgk : dgq;
    if (!dst) return;   // (one array is given for both or for none)
    const float* src = part + (int64_t)s * D + blockIdx.x * 32;
    float a[kRun], v = 0.f;
#pragma unroll
    for (int k = 0; k < kRun; ++k) {
      const int i = ty + k * kRopeRuns;
      a[k] = i < n ? __ldcg(src + (int64_t)i * 2 * D + tx) : 0.f;
    }
#pragma unroll
    for (int k = 0; k < kRun; ++k) v += a[k];
    if (s != (int)blockIdx.y) __syncthreads();   // the runs before have been read
    sh[ty][tx] = v;
    __syncthreads();
    v = sh[tx][ty];   // warp ty: the runs of column ty
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (tx == 0) dst[blockIdx.x * 32 + ty] += v;
  }
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

// Steps of a warp in flight: 64 bytes of each tensor a lane.
template <typename E>
constexpr int kFlight = sizeof(E) == 2 ? 4 : 2;

// Warps that share a token: one per token where the tokens fill the SMs with warps, as many as the
// token has steps where there are few (one decoded token is bound by latency).
int rope_parts(const RopeArgs& a, int hpw, int sms) {
  const int64_t want = (int64_t)sms * 16;
  int64_t n = want / (a.T < want ? a.T : want);   // (one round of them)
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
  if (!bwd) return launch_kernel(k_rope_fwd<E, D, PAIRS, NORM, kFlight<E>>, (unsigned)blocks, kRopeThreads, 0, st, k);
  const unsigned grid = (unsigned)(blocks < kRopeMostCtas ? blocks : kRopeMostCtas);
  cudaError_t e = launch_kernel(k_rope_bwd<E, D, PAIRS, NORM, kFlight<E>>, grid, kRopeThreads, 0, st, k);
  if (e != cudaSuccess || !NORM || (!a.dgamma[0] && !a.dgamma[1])) return e;
  prof_begin(0, st);
  float* dgk = a.heads[1] ? a.dgamma[1] : nullptr;
  return launch_kernel(k_rope_reduce, dim3(D / 32, dgk && dgk == a.dgamma[0] ? 1 : 2), 32 * kRopeRuns, 0, st,
                       (const float*)a.part, (int)grid, D, a.dgamma[0], dgk);
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
