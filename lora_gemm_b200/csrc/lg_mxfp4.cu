// MXFP4 quantization of bf16 rows along K and its inverse.  The block rule is
// the OCP Microscaling one: 32 consecutive values along K share the scale 2^e,
// e = floor(log2 max|v|) - 2 (2 is the exponent of E2M1's largest value, 6),
// each value becomes the E2M1 code of v 2^-e.
//
// Both directions move 2 + 17/32 bytes per value and compute next to nothing:
// HBM bounds them, the instructions per value come next.  Rows are contiguous and
// K a multiple of 128, so both tensors are flat sequences of 128-value groups,
// whatever K: sixteen lanes take a group (eight values each), a warp 32
// consecutive 16-byte pieces at a time and four such loads before the first use.
// Only a group's scale word needs its row: one multiplication by the divisor's
// reciprocal, in one lane per group.  The words are scattered (16 bytes apart
// for neighbouring rows) and meet their sectors' others in L2.
#include "lg_internal.h"
#include "lg_mx.cuh"

namespace lg {

namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;
constexpr int kStep = kThreads / 16;       // groups the CTA has at a time
constexpr int kGroups = kStep * kUnroll;  // groups of a CTA

// n / d for n < 2^31: shift = 31 + ceil(log2 d), mul = floor(2^shift / d) + 1
// (below 2^32; mul d - 2^shift <= d <= 2^(shift - 31), so the quotient is exact).
struct Divide {
  uint32_t d, mul, shift;
};
Divide divide_by(uint32_t d) {
  uint32_t l = 0;
  while ((1u << l) < d) ++l;
  const uint64_t pow = (uint64_t)1 << (31 + l);
  return Divide{d, (uint32_t)(pow / d + 1), 31 + l};
}

// Byte offset of the four scales of flat group i = row * k_groups + kg.
template <typename Index>
__device__ __forceinline__ int64_t scale_word(Index i, const Divide& dv) {
  Index row;
  if constexpr (sizeof(Index) == 8) row = i / (Index)dv.d;
  else row = (Index)(((uint64_t)i * dv.mul) >> dv.shift);
  const uint32_t kg = (uint32_t)(i - row * (Index)dv.d), r = (uint32_t)row & 127u;
  return ((int64_t)((row >> 7) * (Index)dv.d + kg) << 9) + 16 * (r & 31) + 4 * (r >> 5);
}

__device__ __forceinline__ uint4 load_stream(const void* p) {
  uint4 v;
  asm("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

// Sixteen lanes have the words of kUnroll groups, four apart in p: lane p of
// them takes group p's.
__device__ __forceinline__ uint32_t own_word(const uint32_t (&word)[kUnroll], int lane16) {
  uint32_t w = word[0];
#pragma unroll
  for (int p = 1; p < kUnroll; ++p) w = lane16 == p ? word[p] : w;
  return w;
}

// One CTA per kThreads / 16 * kUnroll groups.  Groups [0, groups) hold values,
// [groups, padded) are the padding rows', whose scale bytes are 0.  Index is
// 32 bits wide where the groups allow it.
template <typename Index>
__global__ void __launch_bounds__(kThreads) k_mxfp4_quantize(const uint16_t* __restrict__ in, Index groups, Index padded,
                                                             const Divide dv, uint8_t* __restrict__ codes,
                                                             uint8_t* __restrict__ scales) {
  const int lane16 = threadIdx.x & 15;
  const Index first = (Index)blockIdx.x * kGroups;
  const Index g0 = first + (threadIdx.x >> 4);
  const uint16_t* src = in + (int64_t)g0 * 128 + lane16 * 8;
  uint32_t* dst = reinterpret_cast<uint32_t*>(codes) + (int64_t)g0 * 16 + lane16;
  const bool whole = first + kGroups <= groups;  // of the CTA
  uint4 q[kUnroll];
#pragma unroll
  for (int p = 0; p < kUnroll; ++p) {
    q[p] = make_uint4(0, 0, 0, 0);
    if (whole || g0 + p * kStep < groups) q[p] = load_stream(src + p * (kStep * 128));
  }
  uint32_t word[kUnroll];
#pragma unroll
  for (int p = 0; p < kUnroll; ++p) {
    const bool live = whole || g0 + p * kStep < groups;
    const uint32_t w[4] = {q[p].x, q[p].y, q[p].z, q[p].w};
    uint32_t sb = mxfp4_scale_byte(mx_block_max(w));
    if (live) dst[p * (kStep * 16)] = mxfp4_codes8(w, sb);
    if (!live) sb = 0;
    // The group's four bytes, in all of its lanes.
    sb <<= 8 * (lane16 >> 2);
    sb |= __shfl_xor_sync(0xffffffffu, sb, 4);
    word[p] = sb | __shfl_xor_sync(0xffffffffu, sb, 8);
  }
  const Index g = g0 + lane16 * kStep;
  if (lane16 < kUnroll && g < padded) {
    *reinterpret_cast<uint32_t*>(scales + scale_word<Index>(g, dv)) = own_word(word, lane16);
  }
}

template <typename Index>
__global__ void __launch_bounds__(kThreads) k_mxfp4_dequantize(const uint8_t* __restrict__ codes,
                                                               const uint8_t* __restrict__ scales, Index groups,
                                                               const Divide dv, uint16_t* __restrict__ out) {
  const int lane16 = threadIdx.x & 15;
  const Index first = (Index)blockIdx.x * kGroups;
  const Index g0 = first + (threadIdx.x >> 4);
  const uint32_t* src = reinterpret_cast<const uint32_t*>(codes) + (int64_t)g0 * 16 + lane16;
  uint16_t* dst = out + (int64_t)g0 * 128 + lane16 * 8;
  const bool whole = first + kGroups <= groups;
  uint32_t c[kUnroll];
#pragma unroll
  for (int p = 0; p < kUnroll; ++p) {
    c[p] = 0;
    if (whole || g0 + p * kStep < groups) c[p] = __ldg(src + p * (kStep * 16));
  }
  uint32_t mine = 0;
  const Index g = g0 + lane16 * kStep;
  if (lane16 < kUnroll && g < groups) mine = __ldg(reinterpret_cast<const uint32_t*>(scales + scale_word<Index>(g, dv)));
#pragma unroll
  for (int p = 0; p < kUnroll; ++p) {
    const uint32_t word = __shfl_sync(0xffffffffu, mine, p, 16);
    if (!whole && g0 + p * kStep >= groups) continue;
    const uint32_t s = (word >> (8 * (lane16 >> 2))) & 255u;
    // 2^e: the byte is FP32's own exponent field but for 0 (2^-127, subnormal)
    // and 255 (NaN).
    const float f = s == 255u ? __uint_as_float(0x7FFFFFFFu) : __uint_as_float(s == 0u ? 0x00400000u : s << 23);
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __half2_raw h = __nv_cvt_fp4x2_to_halfraw2((__nv_fp4x2_storage_t)(c[p] >> (8 * i)), __NV_E2M1);
      const float2 v = __half22float2(__half2(h));
      // Exact: two significant bits times a power of two.
      const __nv_bfloat162 b = __floats2bfloat162_rn(v.x * f, v.y * f);
      w[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
    *reinterpret_cast<uint4*>(dst + p * (kStep * 128)) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

}  // namespace

cudaError_t launch_mxfp4_quantize(const uint16_t* in, int64_t rows, int K, uint8_t* codes, uint8_t* scales,
                                  cudaStream_t s) {
  const int64_t groups = rows * (K / 128), padded = (rows + 127) / 128 * 128 * (K / 128);
  const Divide dv = divide_by((uint32_t)(K / 128));
  const unsigned grid = (unsigned)((padded + kGroups - 1) / kGroups);
  if (padded < ((int64_t)1 << 31) - kGroups) {
    k_mxfp4_quantize<uint32_t><<<grid, kThreads, 0, s>>>(in, (uint32_t)groups, (uint32_t)padded, dv, codes, scales);
  } else {
    k_mxfp4_quantize<int64_t><<<grid, kThreads, 0, s>>>(in, groups, padded, dv, codes, scales);
  }
  return cudaGetLastError();
}

cudaError_t launch_mxfp4_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows, int K, uint16_t* out,
                                    cudaStream_t s) {
  const int64_t groups = rows * (K / 128);
  const Divide dv = divide_by((uint32_t)(K / 128));
  const unsigned grid = (unsigned)((groups + kGroups - 1) / kGroups);
  if (groups < ((int64_t)1 << 31) - kGroups) {
    k_mxfp4_dequantize<uint32_t><<<grid, kThreads, 0, s>>>(codes, scales, (uint32_t)groups, dv, out);
  } else {
    k_mxfp4_dequantize<int64_t><<<grid, kThreads, 0, s>>>(codes, scales, groups, dv, out);
  }
  return cudaGetLastError();
}

}  // namespace lg
