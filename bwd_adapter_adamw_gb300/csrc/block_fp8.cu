// E4M3 operands with one scale per block of 128: quantisation of activations (1 x 128 blocks) and
// of a frozen weight (128 x 128 blocks), and the frozen product over them.
#include "block_e4m3.cuh"

namespace lora {

namespace {

constexpr int kBlk = LORA_SCALE_BLOCK;

// One 1 x 128 block per 16 lanes: a 16-byte load, the maximum over the lanes, an 8-byte store.
// A thread takes kQuantBatch blocks whose loads are in flight together. A CTA's blocks lie in a
// slab of kQuantRows rows, so that a block's row comes from a 32-bit division (with 64-bit ones
// the kernel was bound by its index arithmetic: 45 us for 4096 x 4096).
constexpr int kQuantBatch = 4;
constexpr int kQuantRows = 1024;
__global__ void __launch_bounds__(256) k_block_quant(const __nv_bfloat16* __restrict__ src,
                                                     int64_t rows, int64_t K, uint32_t nkb,
                                                     uint8_t* __restrict__ codes,
                                                     float* __restrict__ scales, int64_t ld_row,
                                                     int64_t ld_kb) {
  grid_dep_sync();
  const int sub = threadIdx.x & 15;
  const int64_t row0 = (int64_t)blockIdx.y * kQuantRows;
  const uint32_t blocks = (uint32_t)(rows - row0 < kQuantRows ? rows - row0 : kQuantRows) * nkb;
  const uint32_t first = blockIdx.x * (16 * kQuantBatch) + (threadIdx.x >> 4);
  uint4 v[kQuantBatch];
  int64_t row[kQuantBatch];
  uint32_t kb[kQuantBatch];
#pragma unroll
  for (int u = 0; u < kQuantBatch; ++u) {
    const uint32_t b = first + u * 16;
    const uint32_t r = b / nkb;
    row[u] = row0 + r;
    kb[u] = b - r * nkb;
    const int64_t col = (int64_t)kb[u] * kBlk + sub * 8;
    v[u] = b < blocks && col < K ? __ldg(reinterpret_cast<const uint4*>(src + row[u] * K + col))
                                 : make_uint4(0, 0, 0, 0);
  }
#pragma unroll
  for (int u = 0; u < kQuantBatch; ++u) {
    float m = amax8(v[u]);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (first + u * 16 >= blocks) continue;
    float rcp, sc;
    block_scales(m, rcp, sc);
    const int64_t col = (int64_t)kb[u] * kBlk + sub * 8;
    if (sub == 0) scales[row[u] * ld_row + kb[u] * ld_kb] = sc;
    if (col < K) *reinterpret_cast<uint2*>(codes + row[u] * K + col) = encode8(v[u], rcp);
  }
}

// One 128 x 128 block of W per CTA.
__global__ void __launch_bounds__(256) k_block_quant_weight(const __nv_bfloat16* __restrict__ W,
                                                            int64_t rows, int64_t cols,
                                                            uint8_t* __restrict__ codes,
                                                            float* __restrict__ scales) {
  grid_dep_sync();
  __shared__ float sh[8];
  const int64_t r0 = (int64_t)blockIdx.y * kBlk, c = (int64_t)blockIdx.x * kBlk + (threadIdx.x & 15) * 8;
  uint4 v[8];
  float m = 0.f;
#pragma unroll
  for (int u = 0; u < 8; ++u) {
    const int64_t r = r0 + (threadIdx.x >> 4) + u * 16;
    v[u] = r < rows && c < cols ? __ldg(reinterpret_cast<const uint4*>(W + r * cols + c))
                                : make_uint4(0, 0, 0, 0);
    m = fmaxf(m, amax8(v[u]));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = m;
  __syncthreads();
  m = sh[0];
#pragma unroll
  for (int w = 1; w < 8; ++w) m = fmaxf(m, sh[w]);
  float rcp, sc;
  block_scales(m, rcp, sc);
  if (threadIdx.x == 0) scales[(int64_t)blockIdx.y * gridDim.x + blockIdx.x] = sc;
#pragma unroll
  for (int u = 0; u < 8; ++u) {
    const int64_t r = r0 + (threadIdx.x >> 4) + u * 16;
    if (r < rows && c < cols) *reinterpret_cast<uint2*>(codes + r * cols + c) = encode8(v[u], rcp);
  }
}

}  // namespace

cudaError_t launch_block_quant(const void* src, int64_t rows, int64_t K, uint8_t* codes,
                               float* scales, int64_t ld_row, int64_t ld_kb, cudaStream_t st) {
  if (rows <= 0) return cudaSuccess;
  const int64_t nkb = (K + kBlk - 1) / kBlk;
  const __nv_bfloat16* x = static_cast<const __nv_bfloat16*>(src);
  // 32768 slabs (2^25 rows) per launch
  constexpr int64_t kMost = (int64_t)32768 * kQuantRows;
  for (int64_t at = 0; at < rows; at += kMost) {
    const int64_t n = rows - at < kMost ? rows - at : kMost;
    const int64_t slab = n < kQuantRows ? n : kQuantRows;
    prof_begin(0, st);
    cudaError_t e = launch_kernel(
        k_block_quant,
        dim3((unsigned)((slab * nkb + 16 * kQuantBatch - 1) / (16 * kQuantBatch)),
             (unsigned)((n + kQuantRows - 1) / kQuantRows)),
        256, 0, st, x + at * K, n, K, (uint32_t)nkb, codes + at * K, scales + at * ld_row, ld_row,
        ld_kb);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

cudaError_t launch_block_quant_weight(const void* W, int64_t rows, int64_t cols, uint8_t* codes,
                                      float* scales, cudaStream_t st) {
  prof_begin(0, st);
  return launch_kernel(k_block_quant_weight,
                       dim3((unsigned)((cols + kBlk - 1) / kBlk), (unsigned)((rows + kBlk - 1) / kBlk)),
                       256, 0, st, static_cast<const __nv_bfloat16*>(W), rows, cols, codes, scales);
}

}  // namespace lora
