// E4M3 codes and the scale of a block of 128.
//
// A block x (fp32, each operation rounded): amax = max |x|, r = 448 (1 / amax), codes = e4m3(x r)
// rounded to nearest even with saturation, scale = amax (1 / 448); r = scale = 1 when amax is 0 or
// r is not finite. The factors are products with a reciprocal, not quotients: x / amax of two
// bf16 numbers often lies on a tie between two codes, so the last bit of r decides codes.
#pragma once

#include <cuda_fp8.h>

#include "lora_kernels.h"

namespace lora {

__device__ __forceinline__ void block_scales(float amax, float& rcp, float& scale) {
  rcp = __fmul_rn(__fdiv_rn(1.f, amax), 448.f);
  if (amax > 0.f && isfinite(rcp)) {
    scale = __fmul_rn(amax, 1.f / 448.f);
  } else {
    rcp = 1.f;
    scale = 1.f;
  }
}

// E4M3 codes of 8 bf16 values (one 16-byte vector) times rcp
__device__ __forceinline__ uint2 encode8(const uint4& v, float rcp) {
  const uint32_t h[4] = {v.x, v.y, v.z, v.w};
  uint32_t w[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 f = make_float2(__fmul_rn(__uint_as_float(h[e] << 16), rcp),
                                 __fmul_rn(__uint_as_float(h[e] & 0xFFFF0000u), rcp));
    w[e] = __nv_cvt_float2_to_fp8x2(f, __NV_SATFINITE, __NV_E4M3);
  }
  return make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
}

// max |x| of 8 bf16 values, two at a time (a maximum of bf16 values is one of them; NaNs are passed
// over, and reach their row through their codes)
__device__ __forceinline__ float amax8(const uint4& v) {
  const uint32_t h[4] = {v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu, v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu};
  __nv_bfloat162 m = *reinterpret_cast<const __nv_bfloat162*>(&h[0]);
#pragma unroll
  for (int e = 1; e < 4; ++e) m = __hmax2(m, *reinterpret_cast<const __nv_bfloat162*>(&h[e]));
  return fmaxf(__low2float(m), __high2float(m));
}

}  // namespace lora
