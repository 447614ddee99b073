// Microscaled 4-bit arithmetic shared by the quantisers and the MXFP4 kernels.
#pragma once

#include <cuda_fp8.h>

#include "ptx.cuh"

namespace moe {

// Eight E2M1 codes of f[0..7] * r, input 0 in the lowest nibble: nearest even,
// saturating at 6.
__device__ __forceinline__ uint32_t e2m1x8(const float* f, float r) {
  uint32_t w;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(w)
      : "f"(f[0] * r), "f"(f[1] * r), "f"(f[2] * r), "f"(f[3] * r), "f"(f[4] * r), "f"(f[5] * r), "f"(f[6] * r),
        "f"(f[7] * r));
  return w;
}

// Largest magnitude of n values as fp32 bits: the bits order like the values,
// infinity and then NaN above every finite number.
template <int n>
__device__ __forceinline__ uint32_t amax_bits(const float* f) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < n; ++i) m = max(m, __float_as_uint(f[i]) & 0x7fffffffu);
  return m;
}

// E8M0 byte of an MXFP4 block whose largest magnitude has fp32 bits `m`:
// floor(log2) - 2 + 127, at least 0; 127 (scale 1) for zero; 255 (NaN) for a
// block with an infinity or a NaN.
__device__ __forceinline__ uint32_t e8m0_of(uint32_t m) {
  const uint32_t eb = m >> 23;
  if (eb == 255u) return 255u;
  if (m == 0u) return 127u;
  return eb > 2u ? eb - 2u : 0u;
}

// 2^(127 - byte), a normal fp32 number for every finite byte that e8m0_of gives.
__device__ __forceinline__ float e8m0_rcp(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }

// Value of an E8M0 byte: 2^(byte - 127), 255 is NaN.
__device__ __forceinline__ float e8m0_value(uint32_t byte) {
  return byte == 255u ? __uint_as_float(0x7fffffffu) : byte == 0u ? 0x1p-127f : __uint_as_float(byte << 23);
}

__device__ __forceinline__ float e4m3_value(uint32_t byte) {
  return __half2float(__half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)byte, __NV_E4M3)));
}

}  // namespace moe
