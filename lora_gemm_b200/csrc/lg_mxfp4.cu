// MXFP4 quantization of bf16 rows along K and its inverse.  The block rule is
// the OCP Microscaling one: 32 consecutive values along K share the scale 2^e,
// e = floor(log2 max|v|) - 2 (2 is the exponent of E2M1's largest value, 6),
// each value becomes the E2M1 code of v 2^-e.
//
// Both directions move 2 + 17/32 bytes per value and compute next to nothing:
// HBM bounds them.  A CTA takes tiles of 128 rows x 128 values, the group of
// the blocked scale layout, so that a group's 512 scale bytes leave (or enter)
// through shared memory as one contiguous piece; 16 lanes cover a row's 256
// bytes, eight rows per thread, all loads issued before the first use.
#include "lg_internal.h"
#include "lg_mx.cuh"

namespace lg {

namespace {

constexpr int kThreads = 256;
constexpr int kRowsPerPass = kThreads / 16;
constexpr int kPasses = 128 / kRowsPerPass;

__device__ __forceinline__ uint4 load_stream(const void* p) {
  uint4 v;
  asm("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

__global__ void __launch_bounds__(kThreads) k_mxfp4_quantize(const uint16_t* __restrict__ in, int64_t rows, int K,
                                                             int64_t tiles, uint8_t* __restrict__ codes,
                                                             uint8_t* __restrict__ scales) {
  __shared__ uint32_t sf[128];  // one group's scale bytes, word 4 (r mod 32) + r / 32 for row r
  const int k_groups = K / 128;
  const int lane16 = threadIdx.x & 15;
  const int row0 = threadIdx.x >> 4;
  for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x) {
    const int64_t g = t / k_groups;
    const int kg = (int)(t - g * k_groups);
    const uint16_t* src = in + (g * 128 + row0) * K + kg * 128 + lane16 * 8;
    uint4 q[kPasses];
#pragma unroll
    for (int p = 0; p < kPasses; ++p) {
      q[p] = make_uint4(0, 0, 0, 0);
      if (g * 128 + row0 + p * kRowsPerPass < rows) q[p] = load_stream(src + (int64_t)p * kRowsPerPass * K);
    }
#pragma unroll
    for (int p = 0; p < kPasses; ++p) {
      const int r = row0 + p * kRowsPerPass;
      const uint32_t w[4] = {q[p].x, q[p].y, q[p].z, q[p].w};
      const uint32_t sb = mxfp4_scale_byte(mx_block_max(mx_abs_max8(w)));
      const bool live = g * 128 + r < rows;
      if (live) {
        *reinterpret_cast<uint32_t*>(codes + ((g * 128 + r) * K + kg * 128) / 2 + lane16 * 4) = mxfp4_codes8(w, sb);
      }
      if ((lane16 & 3) == 0) {
        reinterpret_cast<uint8_t*>(sf)[16 * (r & 31) + 4 * (r >> 5) + (lane16 >> 2)] = live ? (uint8_t)sb : 0;
      }
    }
    __syncthreads();
    if (threadIdx.x < 32) {
      reinterpret_cast<uint4*>(scales + (t << 9))[threadIdx.x] = reinterpret_cast<const uint4*>(sf)[threadIdx.x];
    }
    __syncthreads();
  }
}

__global__ void __launch_bounds__(kThreads) k_mxfp4_dequantize(const uint8_t* __restrict__ codes,
                                                               const uint8_t* __restrict__ scales, int64_t rows,
                                                               int K, int64_t tiles, uint16_t* __restrict__ out) {
  const int k_groups = K / 128;
  const int lane16 = threadIdx.x & 15;
  const int row0 = threadIdx.x >> 4;
  for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x) {
    const int64_t g = t / k_groups;
    const int kg = (int)(t - g * k_groups);
    uint32_t c[kPasses], s[kPasses];
#pragma unroll
    for (int p = 0; p < kPasses; ++p) {
      const int r = row0 + p * kRowsPerPass;
      c[p] = s[p] = 0;
      if (g * 128 + r < rows) {
        c[p] = __ldg(reinterpret_cast<const uint32_t*>(codes + ((g * 128 + r) * K + kg * 128) / 2 + lane16 * 4));
        s[p] = __ldg(scales + (t << 9) + 16 * (r & 31) + 4 * (r >> 5) + (lane16 >> 2));
      }
    }
#pragma unroll
    for (int p = 0; p < kPasses; ++p) {
      const int r = row0 + p * kRowsPerPass;
      if (g * 128 + r >= rows) continue;
      // 2^e: the byte is FP32's own exponent field but for 0 (2^-127,
      // subnormal) and 255 (NaN).
      const float f = s[p] == 255u ? __uint_as_float(0x7FFFFFFFu)
                                   : __uint_as_float(s[p] == 0u ? 0x00400000u : s[p] << 23);
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const __half2_raw h = __nv_cvt_fp4x2_to_halfraw2((__nv_fp4x2_storage_t)(c[p] >> (8 * i)), __NV_E2M1);
        const float2 v = __half22float2(__half2(h));
        // Exact: two significant bits times a power of two.
        const __nv_bfloat162 b = __floats2bfloat162_rn(v.x * f, v.y * f);
        w[i] = *reinterpret_cast<const uint32_t*>(&b);
      }
      *reinterpret_cast<uint4*>(out + (g * 128 + r) * K + kg * 128 + lane16 * 8) = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
}

// Four CTAs of 256 threads per SM hold 128 KB of loads in flight.
int tile_grid(int64_t tiles, int sm_count) {
  const int64_t most = (int64_t)sm_count * 8;
  return (int)(tiles < most ? tiles : most);
}

}  // namespace

cudaError_t launch_mxfp4_quantize(const uint16_t* in, int64_t rows, int K, uint8_t* codes, uint8_t* scales,
                                  int sm_count, cudaStream_t s) {
  const int64_t tiles = (rows + 127) / 128 * (K / 128);
  k_mxfp4_quantize<<<tile_grid(tiles, sm_count), kThreads, 0, s>>>(in, rows, K, tiles, codes, scales);
  return cudaGetLastError();
}

cudaError_t launch_mxfp4_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows, int K, uint16_t* out,
                                    int sm_count, cudaStream_t s) {
  const int64_t tiles = (rows + 127) / 128 * (K / 128);
  k_mxfp4_dequantize<<<tile_grid(tiles, sm_count), kThreads, 0, s>>>(codes, scales, rows, K, tiles, out);
  return cudaGetLastError();
}

}  // namespace lg
