// E4M3 operands with one scale per block of 128: quantisation of activations (1 x 128 blocks) and
// of a frozen weight (128 x 128 blocks). Memory-bound: 2 bytes read and 1 written per element.
#include "block_e4m3.cuh"

namespace lora {

namespace {

constexpr int kBlk = LORA_SCALE_BLOCK;

// One 1 x 128 block per 8 lanes: two 16-byte loads, the maximum over the lanes, a 16-byte store.
// Enough small CTAs hide the loads; two or four blocks per lane ran slower (4096 x 4096: 9.1 us with
// one, 9.8 and 11.7; 8192 x 14336: 51.8 us, 6.8 TB/s), as did 16 lanes per block (12.2). A CTA's
// blocks lie in a slab of kQuantRows rows, so that a block's row comes from a 32-bit division (with
// 64-bit ones the kernel was bound by its index arithmetic: 45 us).
constexpr int kQuantBlocks = 256 / 8;   // of a CTA
constexpr int kQuantRows = 1024;
__global__ void __launch_bounds__(256) k_block_quant(const __nv_bfloat16* __restrict__ src,
                                                     int64_t rows, int64_t K, uint32_t nkb,
                                                     uint8_t* __restrict__ codes,
                                                     float* __restrict__ scales, int64_t ld_row,
                                                     int64_t ld_kb) {
  grid_dep_sync();
  const int sub = threadIdx.x & 7;
  const int64_t row0 = (int64_t)blockIdx.y * kQuantRows;
  const uint32_t blocks = (uint32_t)(rows - row0 < kQuantRows ? rows - row0 : kQuantRows) * nkb;
  const uint32_t b = blockIdx.x * kQuantBlocks + (threadIdx.x >> 3), r = b / nkb, kb = b - r * nkb;
  const int64_t row = row0 + r, col = (int64_t)kb * kBlk + sub * 16;
  const bool in = b < blocks && col < K;   // K % 16 == 0
  const uint4* p = reinterpret_cast<const uint4*>(src + row * K + col);
  const uint4 v0 = in ? __ldg(p) : make_uint4(0, 0, 0, 0);
  const uint4 v1 = in ? __ldg(p + 1) : make_uint4(0, 0, 0, 0);
  float m = fmaxf(amax8(v0), amax8(v1));
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (b >= blocks) return;
  float rcp, sc;
  block_scales(m, rcp, sc);
  if (sub == 0) scales[row * ld_row + kb * ld_kb] = sc;
  if (!in) return;
  const uint2 c0 = encode8(v0, rcp), c1 = encode8(v1, rcp);
  *reinterpret_cast<uint4*>(codes + row * K + col) = make_uint4(c0.x, c0.y, c1.x, c1.y);
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
        dim3((unsigned)((slab * nkb + kQuantBlocks - 1) / kQuantBlocks),
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
