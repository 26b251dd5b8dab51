// Internal host-side interface between the C ABI layer (lg_api.cu) and the
// kernel translation units.  Not part of the public ABI.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace lg {

constexpr int kMaxAdapters = 8;

struct MergeAParams {
  const float* A[kMaxAdapters];
  float scale[kMaxAdapters];
  int row_off[kMaxAdapters + 1];  // prefix sums of the ranks
  int n_adapters;
  int d_in;
};

struct MergeBParams {
  const float* B[kMaxAdapters];
  int col_off[kMaxAdapters + 1];
  int n_adapters;
  int d_out;
};

// Grid size for a grid-stride elementwise kernel over `work` items.
int elementwise_grid(int64_t work, int sm_count);

cudaError_t launch_philox_u32(uint32_t* out, int64_t n_blocks, uint64_t seed, uint64_t block_offset, int sm_count,
                              cudaStream_t s);
cudaError_t launch_philox_normal(float* eps, int64_t n, uint64_t seed, uint64_t offset, int sm_count,
                                 cudaStream_t s);
cudaError_t launch_renoise(const float* up, float* x, int64_t n, float sigma, uint64_t seed, uint64_t offset,
                           int sm_count, cudaStream_t s);
cudaError_t launch_euler(float* x, const float* v, int64_t n, float dt, int sm_count, cudaStream_t s);
cudaError_t launch_merge(const MergeAParams& pa, const MergeBParams& pb, float* A_cat, float* B_cat, int sm_count,
                         cudaStream_t s);
// FP32 -> bf16 (RNE) of A_cat [R, K] and B_cat [N, R] into dstA / dstB.
cudaError_t launch_prep_bf16(const float* A_cat, const float* B_cat, uint16_t* dstA, uint16_t* dstB,
                             int64_t nA, int64_t nB, int sm_count, cudaStream_t s);

// MXFP8 quantization of bf16 rows [rows, K] along K (K % 128 == 0): E4M3
// codes [rows, K] and E8M0 scales in the 128 x 128 blocked layout.
cudaError_t launch_mx_quantize(const uint16_t* in, int64_t rows, int K, uint8_t* codes, uint8_t* scales,
                               int sm_count, cudaStream_t s);

// MXFP4 quantization of bf16 rows [rows, K] along K (K % 128 == 0): packed
// E2M1 codes [rows, K / 2] and E8M0 scales in the blocked layout; and back.
cudaError_t launch_mxfp4_quantize(const uint16_t* in, int64_t rows, int K, uint8_t* codes, uint8_t* scales,
                                  cudaStream_t s);
cudaError_t launch_mxfp4_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows, int K, uint16_t* out,
                                    cudaStream_t s);

// Block norms; fields as in lg_block_norm_args / lg_block_norm_backward_args.
struct BlockNormLaunch {
  const void* h;
  const void* b;
  const float* gate;
  const float* scale;
  const float* shift;
  void* h_out;
  void* n;
  void* codes;
  void* scales;
  int64_t M, segment_tokens;
  int D;
  bool fp32;
  int post, pre, codes_format;
  float alpha, eps;
};
cudaError_t launch_block_norm(const BlockNormLaunch& p, cudaStream_t s);

struct BlockNormBackwardLaunch {
  const void* dn;
  const void* dh_out;
  const void* h_out;
  const void* b;
  const float* gate;
  const float* scale;
  void* dh;
  void* db;
  float* dgate;
  float* dscale;
  float* dshift;
  float* workspace;
  int64_t M, segment_tokens;
  int D;
  bool fp32;
  int post, pre;
  float alpha, eps;
  uint64_t wait_limit_ns;
};
// Bytes of partial column sums (0: none are needed); M >= 1.
size_t block_norm_backward_workspace(int64_t M, int D, int64_t segment_tokens);
// *kernels: launches made.
cudaError_t launch_block_norm_backward(const BlockNormBackwardLaunch& p, int* kernels, cudaStream_t s);

// Merged-LoRA linear (tcgen05 kernel).  Factors already in bf16.
struct LinearLaunch {
  const void* x;
  const void* W;
  const uint16_t* A_bf16;  // [R, K]
  const uint16_t* B_bf16;  // [N, R]
  void* y;
  int64_t M;
  int K, N, R;
  int sm_count;
  uint64_t wait_limit_ns;
  // MX base term: codes and blocked E8M0 scales of x [M, K] and W [N, K] --
  // E4M3 for the panel kernel (mx, lg_lora_linear_mxfp8), packed E2M1 for the
  // tile and few-token kernels (lg_lora_linear_mxfp4); x above stays the bf16
  // activations (the LoRA path reads them), W is unused.
  bool mx = false;
  const void* xq = nullptr;
  const void* xsf = nullptr;
  const void* wq = nullptr;
  const void* wsf = nullptr;
  // Fused SwiGLU (MXFP8 only): N = 2 ffn (gate rows, then up rows); the
  // MXFP8 codes [M, ffn] and blocked scales of silu(gate) * up replace y.
  int ffn = 0;
  void* q_codes = nullptr;
  void* q_scales = nullptr;
  // Fused Euler update (bf16 layer only): y is not
  // written; z [M / eu_frame, N, eu_frame] += eu_dt v, bf16 copy to eu_zb.
  float* eu_z = nullptr;
  void* eu_zb = nullptr;
  int64_t eu_frame = 0;
  float eu_dt = 0.f;
};
// Returns cudaSuccess or the failing CUDA error; *driver_failed is set when
// the tensor-map encoder (driver API) is missing or rejects a map.
cudaError_t launch_lora_linear(const LinearLaunch& p, cudaStream_t s, bool* driver_failed);

// lg_lora_linear_mxfp4 for few tokens: FP32 factors as they are, h a workspace
// of M * R floats.  *kernels: launches made.
bool few_tokens(int64_t M);
cudaError_t launch_lora_linear_few(const LinearLaunch& p, const float* A_cat, const float* B_cat, float* h,
                                   int* kernels, cudaStream_t s, bool* driver_failed);

// CTAs per cluster sharing one panel in lg_lora_linear (0: chosen per shape).
void set_cluster_override(int g);
// MMA variant of lg_lora_linear: 1 single-SM, 2 SM pair (0: chosen per shape).
void set_variant_override(int v);

// Device error word of the current device: read and clear (synchronous on s).
cudaError_t read_and_clear_device_error(cudaStream_t s, int* value);

// The same for the error words of the MXFP4 and norm kernels (no synchronization
// before).  A word is a copy of 9 us: one whose kernels the process has never
// launched is not read.
cudaError_t take_tile_error(int* value);
cudaError_t take_few_error(int* value);
cudaError_t take_norm_error(int* value);

// lg_lora_linear_mxfp4 on output tiles: h = x A^T into `h` (workspace, M * R
// bf16) and y = deq(x) deq(W)^T + h B^T, the factors in bf16.  *kernels:
// launches made.
cudaError_t launch_lora_linear_tiles(const LinearLaunch& p, uint16_t* h, int* kernels, cudaStream_t s,
                                     bool* driver_failed);

// The driver's process-unique id of the calling thread's current CUDA
// context.  False when no context is current or the driver cannot say; a
// per-device cache keyed on this id notices a context that was destroyed
// and recreated (cudaDeviceReset) or a different context made current.
bool current_context_id(unsigned long long* id);

// Lets `kernel` use up to `bytes` of dynamic shared memory in the current
// context; asks the runtime once per context and kernel.  `bytes` is the same in
// every call for a kernel.
cudaError_t allow_shared_memory(const void* kernel, int bytes);

// Every check lg_lora_linear makes on its arguments except those on the
// workspace, then (for M > 0) the current device's compute capability, in
// the same order and with the same status codes; launches nothing.  Returns
// an lg_status value.
int check_lora_linear(const void* x, const void* W, const float* A_cat, const float* B_cat, const void* y,
                      int64_t M, int K, int N, int R);

}  // namespace lg
