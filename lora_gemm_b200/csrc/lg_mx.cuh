// Device helpers of the OCP Microscaling (MX) formats: the blocked scale
// layout, block exponents and the 4- and 8-bit codes of eight values at a time
// (four neighbouring lanes hold one block of 32).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp4.h>
#include <cuda_fp8.h>
#include <stdint.h>

namespace lg {

// Byte offset of the scale of (row, block of 32 along K) in the blocked
// layout: 128 rows x 4 blocks are 512 contiguous bytes.
__device__ __forceinline__ int64_t mx_scale_offset(int64_t row, int block, int k_groups) {
  const int r = (int)(row & 127);
  return (((row >> 7) * k_groups + (block >> 2)) << 9) + 16 * (r & 31) + 4 * (r >> 5) + (block & 3);
}

// The largest magnitude among a block's bf16 values as an FP32 word: eight
// packed values of this lane and those of the three lanes beside it.  An
// unsigned maximum of the magnitudes' bits, two at a time: NaN and infinity,
// whose exponent field is all ones, stay on top.
__device__ __forceinline__ uint32_t mx_block_max(const uint32_t (&w)[4]) {
  uint32_t m = __vmaxu2(__vmaxu2(w[0] & 0x7FFF7FFFu, w[1] & 0x7FFF7FFFu),
                        __vmaxu2(w[2] & 0x7FFF7FFFu, w[3] & 0x7FFF7FFFu));
  m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 1));
  m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 2));
  return max(m << 16, m & 0xFFFF0000u);
}

// 2^-e as an FP32 number, e in [-127, 127] (2^-127 is subnormal).
__device__ __forceinline__ float mx_inverse_scale(int e) {
  return e == 127 ? __uint_as_float(0x00400000u) : __uint_as_float((uint32_t)(127 - e) << 23);
}

// MXFP4 scale byte of a block whose largest magnitude has the FP32 word amax:
// e = floor(log2 amax) - 2, at least -127 (zero and FP32 subnormals, whose
// exponent field is 0, end there too), plus 127; 255 for NaN or infinity.
__device__ __forceinline__ uint32_t mxfp4_scale_byte(uint32_t amax) {
  const int field = (int)(amax >> 23);
  return field == 255 ? 255u : (uint32_t)max(field - 2, 0);
}

// The E2M1 codes of eight bf16 values (packed pairs) under scale byte sb,
// value k in bits 4k..4k+3.  The product with 2^-e is exact wherever it
// matters: a result below FP32's normal range rounds to code 0 either way.
__device__ __forceinline__ uint32_t mxfp4_codes8(const uint32_t (&w)[4], uint32_t sb) {
  if (sb == 255u) return 0u;
  const float inv = mx_inverse_scale((int)sb - 127);
  float v[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16) * inv;
    v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u) * inv;
  }
  uint32_t out;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(out)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return out;
}

// MXFP8 (E4M3) scale byte by lg_mx_quantize's rule: e = floor(log2 amax) - 8
// clamped to [-127, 127], -127 for zero.
__device__ __forceinline__ uint32_t mxfp8_scale_byte(float amax) {
  int e = -127;
  if (amax > 0.f) {
    int ex;
    frexpf(amax, &ex);  // amax = m 2^ex, m in [0.5, 1): floor(log2 amax) = ex - 1
    e = min(max(ex - 1 - 8, -127), 127);
  }
  return (uint32_t)(e + 127);
}

// The E4M3 codes of eight bf16 values under scale byte sb.
__device__ __forceinline__ uint2 mxfp8_codes8(const uint32_t (&w)[4], uint32_t sb) {
  const float inv = mx_inverse_scale((int)sb - 127);
  uint32_t out[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 v = make_float2(__uint_as_float(w[i] << 16) * inv, __uint_as_float(w[i] & 0xFFFF0000u) * inv);
    out[i / 2] |= (uint32_t)__nv_cvt_float2_to_fp8x2(v, __NV_SATFINITE, __NV_E4M3) << (16 * (i & 1));
  }
  return make_uint2(out[0], out[1]);
}

}  // namespace lg
