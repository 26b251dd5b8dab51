// What the pipelined tensor-core kernels share: bounded mbarrier waits with the
// device error word of their translation unit, and the host-side tensor maps
// of their operands.
#pragma once

#include <mutex>

#include <cudaTypedefs.h>

#include "../../include/lora_gemm.h"
#include "lg_device.cuh"

namespace lg {
namespace {

// One word per translation unit (device code is not linked across them);
// lg_get_last_device_error reads them all.
__device__ int g_device_error;

constexpr uint64_t TEARDOWN_LIMIT_NS = 200ull * 1000ull * 1000ull;
constexpr int BK = 64;    // bf16 K elements per stage: one 128-byte swizzle span
constexpr int BKQ = 128;  // K elements of a scale group (MXFP8: of a stage, 128-byte rows)
constexpr int Y_BOX = 32;

__device__ __forceinline__ void record_timeout(volatile int* abort_flag) {
  *abort_flag = 1;
  atomicCAS(&g_device_error, 0, (int)LG_ERR_DEVICE_TIMEOUT);
}

// Wait for the phase of `bar` with parity `parity` to complete, giving up
// after limit_ns or as soon as another warp of the CTA has given up.  With
// `cluster_scope` the wait acquires at cluster scope (peers' writes made
// before their release-arrive become visible).
__device__ __noinline__ bool wait_slow(uint32_t bar, uint32_t parity, uint64_t limit_ns, volatile int* abort_flag,
                                       bool cluster_scope) {
  const uint64_t t0 = globaltimer_ns();
  // Sleep in slices of at most 20 us (woken early when the phase completes),
  // never past the wait's own limit.
  const uint32_t hint = (uint32_t)(limit_ns < 20000ull ? limit_ns : 20000ull);
  for (;;) {
    if (cluster_scope ? mbar_try_wait_cluster_sleep(bar, parity, hint) : mbar_try_wait_sleep(bar, parity, hint))
      return true;
    if (*abort_flag) return false;
    if (globaltimer_ns() - t0 >= limit_ns) {
      record_timeout(abort_flag);
      return false;
    }
  }
}
__device__ __forceinline__ bool wait_bounded(uint32_t bar, uint32_t parity, uint64_t limit_ns,
                                             volatile int* abort_flag, bool cluster_scope = false) {
  if (cluster_scope ? mbar_try_wait_cluster(bar, parity) : mbar_try_wait(bar, parity)) return true;
  return wait_slow(bar, parity, limit_ns, abort_flag, cluster_scope);
}

// Teardown wait: ignores the abort flag, gives up after limit_ns.
__device__ __noinline__ void wait_teardown(uint32_t bar, uint32_t parity, volatile int* abort_flag,
                                           uint64_t limit_ns = TEARDOWN_LIMIT_NS) {
  if (mbar_try_wait(bar, parity)) return;
  const uint64_t t0 = globaltimer_ns();
  while (!mbar_try_wait(bar, parity)) {
    if (globaltimer_ns() - t0 >= limit_ns) {
      record_timeout(abort_flag);
      return;
    }
  }
}

// Polls a phase without being held by the hardware, as a plain try_wait may for
// microseconds; for limits below that time.  One below the timer's own step gives
// up at the first look.
__device__ __noinline__ bool wait_polled(uint32_t bar, uint32_t parity, uint64_t limit_ns, volatile int* abort_flag) {
  const uint64_t t0 = globaltimer_ns();
  for (;;) {
    if (mbar_test_wait_cluster(bar, parity)) return true;
    if (*abort_flag) return false;
    if (limit_ns < 1000ull || globaltimer_ns() - t0 >= limit_ns) {
      record_timeout(abort_flag);
      return false;
    }
  }
}
// wait_bounded, but exact about short limits.
__device__ __forceinline__ bool wait_limited(uint32_t bar, uint32_t parity, uint64_t limit_ns, volatile int* abort_flag,
                                             bool cluster_scope = false) {
  if (limit_ns < 20000ull) return wait_polled(bar, parity, limit_ns, abort_flag);
  return wait_bounded(bar, parity, limit_ns, abort_flag, cluster_scope);
}

// Every lane's wait succeeded: the warp goes on, or gives up, as one.
__device__ __forceinline__ bool all_waited(bool ok) { return __all_sync(0xffffffffu, ok); }

// One lane of the (converged) warp, always the same.
__device__ __forceinline__ bool elect_lane() {
  uint32_t yes;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(yes));
  return yes != 0;
}

__device__ __forceinline__ void fence_proxy_async_smem() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

__device__ __forceinline__ void advance(uint32_t& stage, uint32_t& phase, uint32_t stages) {
  if (++stage == stages) {
    stage = 0;
    phase ^= 1;
  }
}

inline PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess) {
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    }
  });
  return fn;
}

// Row-major bf16 matrix [outer, inner] read as tiles of box_outer rows x 64
// columns with the 128-byte swizzle; out-of-range rows read as zero.
inline bool make_map(PFN_cuTensorMapEncodeTiled_v12000 enc, CUtensorMap* m, const void* base, uint64_t inner,
              uint64_t outer, uint32_t box_outer) {
  cuuint64_t dims[2] = {inner, outer};
  cuuint64_t strides[1] = {inner * 2};
  cuuint32_t box[2] = {(cuuint32_t)BK, box_outer};
  cuuint32_t elem_strides[2] = {1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, elem_strides,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Row-major codes [outer, inner bytes] (E4M3, or packed E2M1) read as tiles of
// box_outer rows x 128 bytes with the 128-byte swizzle (the layout of the bf16 tiles above).
inline bool make_map_codes(PFN_cuTensorMapEncodeTiled_v12000 enc, CUtensorMap* m, const void* base, uint64_t inner,
                    uint64_t outer, uint32_t box_outer) {
  cuuint64_t dims[2] = {inner, outer};
  cuuint64_t strides[1] = {inner};
  cuuint32_t box[2] = {(cuuint32_t)BKQ, box_outer};
  cuuint32_t elem_strides[2] = {1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, elem_strides,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Row-major FP32 matrix [outer, inner] read as tiles of box_outer rows x 32
// columns with the 128-byte swizzle, rounded to nearest TF32 values (ten fraction
// bits) on the way: the tensor core itself cuts the further bits off, which made a
// sum of products 7e-4 too small.  Out-of-range rows read as zero.
inline bool make_map_tf32(PFN_cuTensorMapEncodeTiled_v12000 enc, CUtensorMap* m, const void* base, uint64_t inner,
                          uint64_t outer, uint32_t box_outer) {
  cuuint64_t dims[2] = {inner, outer};
  cuuint64_t strides[1] = {inner * 4};
  cuuint32_t box[2] = {32, box_outer};
  cuuint32_t elem_strides[2] = {1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_TFLOAT32, 2, const_cast<void*>(base), dims, strides, box, elem_strides,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// MX scales (the blocked layout of lg_mx_quantize) viewed as rows of 256
// bytes: a 512-byte group is a box of two rows (box_rows: several groups in a
// row).  Groups past the end read as zero.
inline bool make_map_scales(PFN_cuTensorMapEncodeTiled_v12000 enc, CUtensorMap* m, const void* base, uint64_t groups,
                            uint32_t box_rows = 2) {
  cuuint64_t dims[2] = {256, groups * 2};
  cuuint64_t strides[1] = {256};
  cuuint32_t box[2] = {256, box_rows};
  cuuint32_t elem_strides[2] = {1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, elem_strides,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_NONE,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Row-major bf16 y [rows, cols] written in 32 x 32 boxes from 64-byte-swizzled
// shared memory; the store clips rows and columns outside the matrix.
inline bool make_store_map(PFN_cuTensorMapEncodeTiled_v12000 enc, CUtensorMap* m, void* base, uint64_t cols,
                    uint64_t rows) {
  cuuint64_t dims[2] = {cols, rows};
  cuuint64_t strides[1] = {cols * 2};
  cuuint32_t box[2] = {(cuuint32_t)Y_BOX, (cuuint32_t)Y_BOX};
  cuuint32_t elem_strides[2] = {1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, base, dims, strides, box, elem_strides,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The error word of this translation unit: read and clear (synchronous).
inline cudaError_t take_device_error(int* value) {
  int v = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_device_error, sizeof(int));
  if (e != cudaSuccess) return e;
  if (v != 0) {
    const int zero = 0;
    e = cudaMemcpyToSymbol(g_device_error, &zero, sizeof(int));
  }
  *value = v;
  return e;
}

}  // namespace
}  // namespace lg
