// Orthogonalised update of the adapter matrices: momentum, then a Newton-Schulz sequence
// X <- (a I + b G + c G^2) X, G = X X^T over the smaller side (at most 64), from X = u / ||u||_F.
//
// The smaller side is the adapter's rank, so the sequence acts on the small Gram matrix G alone:
// with P = a I + b G + c G^2 (a polynomial in G, so they commute) one step maps G to P G P and
// multiplies X by P. Several steps then cost one Gram matrix, small products and one product
// Q X = P_m .. P_1 X on the long axis. A rounding of G, relative to its largest eigenvalue, is
// amplified by about a^2 per step at the smallest ones, so after at most kStageSteps steps the
// Gram matrix is formed again from Q X.
#include "lora_kernels.h"

namespace lora {

namespace {

constexpr int kMuonThreads = 256;
constexpr int kS = LORA_MAX_RANK;   // largest smaller side
constexpr int kLd = kS + 1;         // row stride of the small matrices
constexpr int kTile = 32;           // long-axis elements per tile
constexpr int kStageSteps = 3;
constexpr int kMuonSmem = (5 * kS * kLd + 2 * kTile * kLd) * 4;

__device__ __forceinline__ float block_max(float v, float* sh) {
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = v;
  __syncthreads();
  v = sh[0];
  for (int w = 1; w < kMuonThreads / 32; ++w) v = fmaxf(v, sh[w]);
  return v;
}

// C = alpha I + beta A + gamma A B for s x s matrices (B and A commute; C distinct from both)
__device__ void small_mm(float* C, const float* A, const float* B, int s, float alpha, float beta,
                         float gamma) {
  for (int e = threadIdx.x; e < s * s; e += kMuonThreads) {
    const int i = e / s, j = e % s;
    float d = 0.f;
    for (int k = 0; k < s; ++k) d = fmaf(A[i * kLd + k], B[k * kLd + j], d);
    C[i * kLd + j] = gamma * d + beta * A[i * kLd + j] + (i == j ? alpha : 0.f);
  }
  __syncthreads();
}

// One matrix per CTA.
__global__ void __launch_bounds__(kMuonThreads) k_muon(float* __restrict__ P, float* __restrict__ G,
                                                       float* __restrict__ M, const MuonTab tab,
                                                       const MuonK hp,
                                                       const double* __restrict__ scale_norm,
                                                       const int32_t* __restrict__ status,
                                                       int zero_grads) {
  grid_dep_sync();
  extern __shared__ float sm[];
  float* g0 = sm;                    // Gram matrix
  float* q = g0 + kS * kLd;          // product of the steps so far
  float* t1 = q + kS * kLd;
  float* t2 = t1 + kS * kLd;
  float* t3 = t2 + kS * kLd;
  float* u = t3 + kS * kLd;          // [kTile][kLd]
  float* x = u + kTile * kLd;        // [kTile][kLd]
  __shared__ float sh[kMuonThreads / 32];
  const MuonMat mt = tab.m[blockIdx.x];
  if (status[mt.group] != LORA_OK) return;
  const float c = (float)scale_norm[2 * mt.group];
  const int s = mt.s;
  const int64_t n = mt.n;
  const int64_t sj = mt.tall ? s : 1, si = mt.tall ? 1 : n;   // element (i, j): i * si + j * sj
  float* p = P + mt.offset;
  float* g = G + mt.offset;
  float* m = M + mt.offset;
  const float mu = hp.mu;
  // momentum and the largest |u|
  float mx = 0.f;
  for (int64_t e = threadIdx.x; e < n * s; e += kMuonThreads) {
    const float gh = c * g[e];
    const float mn = fmaf(mu, m[e], gh);
    m[e] = mn;
    mx = fmaxf(mx, fabsf(hp.nesterov ? fmaf(mu, mn, gh) : mn));
  }
  mx = block_max(mx, sh);
  // u scaled by a power of two to about one, so that its squares stay in range
  const float pre = mx > 0.f && isfinite(mx) ? exp2f((float)-min(max(ilogbf(mx), -120), 120)) : 1.f;
  for (int e = threadIdx.x; e < s * s; e += kMuonThreads) q[e / s * kLd + e % s] = e / s == e % s;
  __syncthreads();
  auto load_tile = [&](int64_t j0) {   // u of long-axis elements j0 .. j0 + kTile, zeros past n
    for (int e = threadIdx.x; e < kTile * s; e += kMuonThreads) {
      const int jj = mt.tall ? e / s : e % kTile, i = mt.tall ? e % s : e / kTile;
      float v = 0.f;
      if (j0 + jj < n) {
        const int64_t at = i * si + (j0 + jj) * sj;
        v = hp.nesterov ? fmaf(mu, m[at], c * g[at]) : m[at];
      }
      u[jj * kLd + i] = v * pre;
    }
    __syncthreads();
    for (int e = threadIdx.x; e < kTile * s; e += kMuonThreads) {
      const int jj = e / s, i = e % s;
      float d = 0.f;
      for (int k = 0; k < s; ++k) d = fmaf(q[i * kLd + k], u[jj * kLd + k], d);
      x[jj * kLd + i] = d;
    }
    __syncthreads();
  };
  for (int done = 0; done < hp.steps;) {
    const int left = hp.steps - done;
    const int now = left % kStageSteps ? left % kStageSteps : kStageSteps;
    float acc[kS * kS / kMuonThreads] = {};
    for (int64_t j0 = 0; j0 < n; j0 += kTile) {
      load_tile(j0);
#pragma unroll
      for (int v = 0; v < kS * kS / kMuonThreads; ++v) {
        const int e = threadIdx.x + v * kMuonThreads;
        if (e >= s * s) break;
        const int i = e / s, k = e % s;
        for (int jj = 0; jj < kTile; ++jj) acc[v] = fmaf(x[jj * kLd + i], x[jj * kLd + k], acc[v]);
      }
      __syncthreads();
    }
    for (int v = 0, e = threadIdx.x; e < s * s; ++v, e += kMuonThreads) {
#pragma unroll
      for (int w = 0; w < kS * kS / kMuonThreads; ++w)
        if (w == v) g0[e / s * kLd + e % s] = acc[w];
    }
    __syncthreads();
    if (done == 0) {   // X = u / ||u||, ||u||^2 = trace G
      float tr = 0.f;
      for (int i = 0; i < s; ++i) tr += g0[i * kLd + i];
      __syncthreads();
      const float inv = tr > 0.f ? 1.f / sqrtf(tr) : 0.f;
      for (int e = threadIdx.x; e < s * s; e += kMuonThreads) {
        g0[e / s * kLd + e % s] *= inv * inv;
        q[e / s * kLd + e % s] *= inv;
      }
      __syncthreads();
    }
    for (int k = 0; k < now; ++k) {
      small_mm(t1, g0, g0, s, 0.f, 0.f, 1.f);                 // G^2
      for (int e = threadIdx.x; e < s * s; e += kMuonThreads) {   // P
        const int i = e / s, j = e % s;
        t1[i * kLd + j] = hp.c * t1[i * kLd + j] + hp.b * g0[i * kLd + j] + (i == j ? hp.a : 0.f);
      }
      __syncthreads();
      small_mm(t2, t1, q, s, 0.f, 0.f, 1.f);                  // Q <- P Q
      for (int e = threadIdx.x; e < s * s; e += kMuonThreads) q[e / s * kLd + e % s] = t2[e / s * kLd + e % s];
      __syncthreads();
      if (k + 1 < now) {                                      // G <- P (G P)
        small_mm(t2, g0, t1, s, 0.f, 0.f, 1.f);
        small_mm(t3, t1, t2, s, 0.f, 0.f, 1.f);
        for (int e = threadIdx.x; e < s * s; e += kMuonThreads) g0[e / s * kLd + e % s] = t3[e / s * kLd + e % s];
        __syncthreads();
      }
    }
    done += now;
  }
  const float lr = mt.lr, step = mt.step, wd = mt.decay;
  for (int64_t j0 = 0; j0 < n; j0 += kTile) {
    load_tile(j0);
    for (int e = threadIdx.x; e < kTile * s; e += kMuonThreads) {
      const int jj = mt.tall ? e / s : e % kTile, i = mt.tall ? e % s : e / kTile;
      if (j0 + jj >= n) continue;
      const int64_t at = i * si + (j0 + jj) * sj;
      p[at] = p[at] - step * x[jj * kLd + i] - lr * wd * p[at];
      if (zero_grads) g[at] = 0.f;
    }
    __syncthreads();
  }
}

}  // namespace

cudaError_t launch_muon(float* p, float* g, float* m, const MuonTab& tab, const MuonK& hp,
                        const double* scale_norm, const int32_t* status, int zero_grads,
                        cudaStream_t st) {
  static bool attr = false;
  if (!attr) {
    cudaError_t e = cudaFuncSetAttribute(k_muon, cudaFuncAttributeMaxDynamicSharedMemorySize, kMuonSmem);
    if (e != cudaSuccess) return e;
    attr = true;
  }
  prof_begin(0, st);
  return launch_kernel(k_muon, (unsigned)tab.n, kMuonThreads, kMuonSmem, st, p, g, m, tab, hp,
                       scale_norm, status, zero_grads);
}

}  // namespace lora
