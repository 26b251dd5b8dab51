// lg_lora_linear_mxfp4 for few tokens (M <= 128): bound by reading the weights
// and factors once, 17/32 bytes per weight and 4 per factor (past 64 tokens A_cat
// a second time, from L2).
//
// The tile kernel would multiply 256 token rows, give each SM pair whole
// columns of K, and read the factors twice (a pass copies them to bf16): 129 x
// 7168 -> 7168 at rank 576 takes it 45 us, 128 tokens take 40 here and one token
// 16.5 (9.5 without adapters).  Here the weights are the wide
// operand and the tokens the narrow one, and K is split:
//
//   k_few_down  h = x A_cat^T: a cluster of eight CTAs per 16 ranks, K spread
//               over its warps (mma.sync straight from registers: the FP32
//               factors are rounded on the way, which no tensor-memory operand
//               path does), partial sums joined through distributed shared
//               memory.
//   k_few_up    y = deq(x) deq(W)^T + h B_cat^T: 128 outputs per cluster of S
//               CTAs that split K and the ranks; tcgen05 with the weights as the
//               128-row operand and the tokens as its N (16 to 128): MXFP4
//               stages of 256 K, then TF32 stages of 32 ranks that take the
//               FP32 B_cat and h, rounded by the loads.  All loads are TMA,
//               100 KB of them in flight per CTA; the CTAs' accumulators are
//               joined in the order of their ranks through distributed shared
//               memory.
//
// k_few_up is launched as a programmatic dependent and waits for k_few_down only
// before its first load of h: it reads weights beside it on the SMs that have room.
// At rank 192 k_few_down's 96 CTAs leave most of them free; at rank 576 it has 288,
// whose 114 to 128 registers for each of 256 threads leave next to none, and the
// two run one after the other.
//
// A_cat is rounded to bf16, h and B_cat to TF32: one product each, as in the
// library's other layers, against an FP32 evaluation of the adapters' term a
// difference of 0.0018 in y (relative Frobenius; y's own rounding is 0.0016, and the
// base term's 4-bit codes move it by 0.16).  As pairs of bf16 parts, two products
// for h and three for y, the term would be FP32's: 17.9 us instead of 16.4 for one
// token 7168 -> 7168 at rank 576, 102 instead of 92 for 128 x 28672 -> 7168.
#include <atomic>

#include <cuda_bf16.h>

#include "lg_internal.h"
#include "lg_pipeline.cuh"

namespace lg {

namespace {

std::atomic<bool> g_launched{false};  // so that the error word may be set

constexpr int kDownCluster = 8;
constexpr int kDownRows = 16;  // ranks per cluster

constexpr int kUpRows = 128;     // outputs per cluster: the MMA's M
constexpr int kUpThreads = 192;  // loads, MMAs, four epilogue warps
constexpr int kUpStagesMax = 8;
constexpr uint32_t kUpClusterMax = 8;
constexpr uint32_t kUpWBytes = kUpRows * 128;
constexpr uint32_t kSfBytes = 1024;  // scales of 128 rows x 256 K

__device__ __forceinline__ float4 ld_stream4(const float* p) {
  float4 v;
  asm volatile("ld.global.L1::no_allocate.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "l"(p));
  return v;
}
// FP32 values -> bf16 pairs, rounded to nearest (as the other layers round the
// factors for the tensor cores).
__device__ __forceinline__ uint32_t round2(float a, float b) {
  const __nv_bfloat162 p = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&p);
}
__device__ __forceinline__ void round8(const float4& a, const float4& b, uint32_t (&h)[4]) {
  h[0] = round2(a.x, a.y);
  h[1] = round2(a.z, a.w);
  h[2] = round2(b.x, b.y);
  h[3] = round2(b.z, b.w);
}
__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
      "%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

struct DownArgs {
  const uint16_t* x;  // [M, K] bf16
  const float* A;     // [R, K]
  float* h;           // [M, R]
  int M, K, R;
};

// NG groups of eight tokens, up to 64 (the tokens past 64 are a second row of
// clusters: 70 x 7168, rank 576, 35.7 us against 37.3 with sixteen groups).  The
// eight warps of eight CTAs split K 64 ways, so that a warp has few batches of
// loads to wait for.
template <int NG>
struct DownCfg {
  static constexpr int kWarps = 8;
  static constexpr int kBatch = NG <= 2 ? 4 : 2;  // steps whose loads are in flight together
};

// h[m, r0 .. r0 + 15]: cluster blockIdx.x / 8; its warps take every 64th step of
// 32 K.
template <int NG>
__global__ void __cluster_dims__(kDownCluster, 1, 1) __launch_bounds__(DownCfg<NG>::kWarps * 32, 2)
    k_few_down(DownArgs a) {
  constexpr int W = DownCfg<NG>::kWarps, U = DownCfg<NG>::kBatch;
  __shared__ float sums[W][NG * 8][kDownRows];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  // Tokens from 64 blockIdx.y on.
  a.x += (int64_t)blockIdx.y * 64 * a.K;
  a.h += (int64_t)blockIdx.y * 64 * a.R;
  a.M -= (int)blockIdx.y * 64;
  if (a.M > NG * 8) a.M = NG * 8;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const uint32_t rank = cluster_ctarank();
  const int r0 = (int)(blockIdx.x / kDownCluster) * kDownRows;
  const int steps = a.K / 32;
  float acc[NG][4];
#pragma unroll
  for (int n = 0; n < NG; ++n) {
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[n][e] = 0.f;
  }
  const float* pa = a.A + (int64_t)(r0 + g) * a.K + t * 8;
  const uint16_t* px = a.x + (int64_t)g * a.K + t * 8;
  for (int s0 = (int)rank * W + warp; s0 < steps; s0 += U * kDownCluster * W) {
    float4 w[U][2][2];
    uint4 x[U][NG];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int s = s0 + u * kDownCluster * W;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        w[u][i][0] = w[u][i][1] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (s < steps) {
          const float* p = pa + (int64_t)i * 8 * a.K + s * 32;
          w[u][i][0] = ld_stream4(p);
          w[u][i][1] = ld_stream4(p + 4);
        }
      }
#pragma unroll
      for (int n = 0; n < NG; ++n) {
        x[u][n] = make_uint4(0, 0, 0, 0);
        if (s < steps && n * 8 + g < a.M) x[u][n] = __ldg(reinterpret_cast<const uint4*>(px + (int64_t)n * 8 * a.K + s * 32));
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      uint32_t v[2][4];
#pragma unroll
      for (int i = 0; i < 2; ++i) round8(w[u][i][0], w[u][i][1], v[i]);
#pragma unroll
      for (int n = 0; n < NG; ++n) {
        mma_bf16(acc[n], v[0][0], v[1][0], v[0][1], v[1][1], x[u][n].x, x[u][n].y);
        mma_bf16(acc[n], v[0][2], v[1][2], v[0][3], v[1][3], x[u][n].z, x[u][n].w);
      }
    }
  }
#pragma unroll
  for (int n = 0; n < NG; ++n) {
#pragma unroll
    for (int e = 0; e < 4; ++e) sums[warp][n * 8 + 2 * t + (e & 1)][8 * (e >> 1) + g] = acc[n][e];
  }
  __syncthreads();
  // The CTA's own sum, warp by warp, then the cluster's, CTA by CTA.
  for (int i = threadIdx.x; i < a.M * kDownRows; i += W * 32) {
    float* p = &sums[0][0][0] + i;
    float v = p[0];
#pragma unroll
    for (int k = 1; k < W; ++k) v += p[k * NG * 8 * kDownRows];
    p[0] = v;
  }
  cluster_barrier();
  for (int i = (int)rank * W * 32 + threadIdx.x; i < a.M * kDownRows; i += kDownCluster * W * 32) {
    const uint32_t at = smem_u32(&sums[0][0][0] + i);
    float v = 0.f;
#pragma unroll
    for (int c = 0; c < kDownCluster; ++c) {
      float p;
      asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(p) : "r"(mapa_shared(at, (uint32_t)c)) : "memory");
      v += p;
    }
    a.h[(int64_t)(i / kDownRows) * a.R + r0 + i % kDownRows] = v;
  }
  // No CTA leaves while a peer may still read its sums.
  cluster_barrier();
}

// NT: tokens, rounded up to the MMA's N.
template <int NT>
struct UpCfg {
  static constexpr uint32_t kX = NT * 128;
  static constexpr uint32_t kStage = kUpWBytes + kX + 2 * kSfBytes;
  // Two CTAs per SM.
  static constexpr int kStages = (int)(104 * 1024 / kStage) < kUpStagesMax ? (int)(104 * 1024 / kStage) : kUpStagesMax;
  static constexpr uint32_t kSums = NT * kUpRows * 4;  // over the ring, once it is done
  static constexpr uint32_t kRing = kStage * kStages > kSums ? kStage * kStages : kSums;
  static constexpr uint32_t kSfCols = 16;  // TMEM columns of a stage's scales: W at 4 g, x at 8 + 4 g
  static constexpr uint32_t kSfBufs = 4;
  static constexpr uint32_t kCols = NT + kSfBufs * kSfCols <= 128 ? 128 : 256;  // TMEM columns allocated
  static_assert(NT + kSfBufs * kSfCols <= kCols && kStages >= 3, "few-token layout");
};

struct UpControl {
  uint64_t full[kUpStagesMax];
  uint64_t empty[kUpStagesMax];
  uint64_t done;  // every MMA has finished
  uint32_t tmem_base;
  int abort_flag;
};

struct UpArgs {
  uint16_t* y;
  int M, N;
  int q_stages, q_groups;  // 256-K stages of the base term, 128-K scale groups
  int h_stages;            // 32-rank stages of the adapters' term
  unsigned long long wait_limit_ns;
};

// CTA `rank` of a cluster of S takes stages rank, rank + S, ... of the base term,
// then of the adapters' term.
template <int NT>
__global__ void __launch_bounds__(kUpThreads)
    k_few_up(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_x,
             const __grid_constant__ CUtensorMap tm_sw, const __grid_constant__ CUtensorMap tm_sx,
             const __grid_constant__ CUtensorMap tm_b, const __grid_constant__ CUtensorMap tm_h, const UpArgs a) {
  using C = UpCfg<NT>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  UpControl* ctl = reinterpret_cast<UpControl*>(base + C::kRing);
  const uint32_t smem = smem_u32(base);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint32_t S;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(S));
  const uint32_t rank = cluster_ctarank();
  const int tile = (int)cluster_id_x();
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(smem_u32(&ctl->full[s]), 1);
      mbar_init(smem_u32(&ctl->empty[s]), 1);
    }
    mbar_init(smem_u32(&ctl->done), 1);
    ctl->abort_flag = 0;
    fence_mbarrier_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&ctl->tmem_base), C::kCols);
    tmem_relinquish();
    tc_fence_before();
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl->tmem_base;
  volatile int* abort_flag = &ctl->abort_flag;
  const uint32_t full0 = smem_u32(&ctl->full[0]), empty0 = smem_u32(&ctl->empty[0]), done = smem_u32(&ctl->done);
  const uint32_t stages = (uint32_t)C::kStages;

  if (warp == 0) {
    uint32_t stage = 0, phase = 0;
    uint64_t fills = 0;
    bool ok = true;
    for (int kb = (int)rank; kb < a.q_stages; kb += (int)S) {
      if (!all_waited(wait_limited(empty0 + 8 * stage, phase ^ 1, a.wait_limit_ns, abort_flag))) {
        ok = false;
        break;
      }
      const uint32_t st = smem + stage * C::kStage, bar = full0 + 8 * stage;
      if (elect_lane()) {
        mbar_arrive_expect_tx(bar, C::kStage);
        tma_load_2d(st, &tm_w, bar, kb * 128, tile * kUpRows);
        tma_load_2d(st + kUpWBytes, &tm_x, bar, kb * 128, 0);
        // Two 512-byte groups each; past an odd last group: bytes that no MMA reads.
        tma_load_2d(st + kUpWBytes + C::kX, &tm_sw, bar, 0, 2 * (tile * a.q_groups + 2 * kb));
        tma_load_2d(st + kUpWBytes + C::kX + kSfBytes, &tm_sx, bar, 0, 2 * (2 * kb));
      }
      __syncwarp();
      ++fills;
      advance(stage, phase, stages);
    }
    // Also where no stage needs h: the grid does not end before k_few_down.
    if (a.h_stages > 0) asm volatile("griddepcontrol.wait;" ::: "memory");
    for (int kb = (int)rank; ok && kb < a.h_stages; kb += (int)S) {
      if (!all_waited(wait_limited(empty0 + 8 * stage, phase ^ 1, a.wait_limit_ns, abort_flag))) {
        ok = false;
        break;
      }
      const uint32_t st = smem + stage * C::kStage, bar = full0 + 8 * stage;
      if (elect_lane()) {
        mbar_arrive_expect_tx(bar, kUpWBytes + C::kX);
        tma_load_2d(st, &tm_b, bar, kb * 32, tile * kUpRows);
        tma_load_2d(st + kUpWBytes, &tm_h, bar, kb * 32, 0);
      }
      __syncwarp();
      ++fills;
      advance(stage, phase, stages);
    }
    // Every copy has landed before the ring is used for the sums.
    for (uint32_t s = 0; s < stages; ++s) {
      const uint64_t fs = fills / stages + (s < fills % stages ? 1 : 0);
      if (fs) wait_teardown(full0 + 8 * s, (uint32_t)((fs - 1) & 1), abort_flag);
    }
  } else if (warp == 1) {
    uint32_t stage = 0, phase = 0, sf_buf = 0;
    uint32_t any = 0;  // 0 until the first MMA, which clears the accumulator
    bool ok = true;
    for (int kb = (int)rank; kb < a.q_stages; kb += (int)S) {
      if (!all_waited(wait_limited(full0 + 8 * stage, phase, a.wait_limit_ns, abort_flag))) {
        ok = false;
        break;
      }
      tc_fence_after();
      const uint32_t st = smem + stage * C::kStage;
      const uint64_t dw = sw128_kmajor_desc(st), dx = sw128_kmajor_desc(st + kUpWBytes);
      const uint32_t sf = tmem + NT + C::kSfCols * sf_buf;
      const uint32_t src = st + kUpWBytes + C::kX;
      const int groups = min(2, a.q_groups - 2 * kb);
      if (elect_lane()) {
        for (int g = 0; g < groups; ++g) {
          tmem_cp_32x128b_x4(sf + 4 * g, plain_rows16_desc(src + g * 512));
          tmem_cp_32x128b_x4(sf + 8 + 4 * g, plain_rows16_desc(src + kSfBytes + g * 512));
        }
        for (int g = 0; g < groups; ++g) {
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            umma_mxf4(tmem, dw + 2 * (2 * g + k), dx + 2 * (2 * g + k), idesc_mxf4(kUpRows, NT, 2u * k, 2u * k),
                      sf + 4 * g, sf + 8 + 4 * g, any | (uint32_t)(g | k));
          }
        }
        umma_commit(empty0 + 8 * stage);
      }
      __syncwarp();
      any = 1;
      if (++sf_buf == C::kSfBufs) sf_buf = 0;
      advance(stage, phase, stages);
    }
    for (int kb = (int)rank; ok && kb < a.h_stages; kb += (int)S) {
      if (!all_waited(wait_limited(full0 + 8 * stage, phase, a.wait_limit_ns, abort_flag))) {
        ok = false;
        break;
      }
      tc_fence_after();
      const uint32_t st = smem + stage * C::kStage;
      const uint64_t dw = sw128_kmajor_desc(st), dx = sw128_kmajor_desc(st + kUpWBytes);
      if (elect_lane()) {
#pragma unroll
        for (int k = 0; k < 4; ++k)  // K = 8 each: 32 bytes
          umma_tf32(tmem, dw + 2 * k, dx + 2 * k, idesc_tf32(kUpRows, NT), any | (uint32_t)k);
        umma_commit(empty0 + 8 * stage);
      }
      __syncwarp();
      any = 1;
      advance(stage, phase, stages);
    }
    if (elect_lane()) umma_commit(done);
    __syncwarp();
  }
  // Every MMA has finished and every load has landed: the ring is free.
  wait_teardown(done, 0, abort_flag, a.wait_limit_ns + TEARDOWN_LIMIT_NS);
  __syncthreads();
  tc_fence_after();
  const bool some = (int)rank < a.q_stages || (int)rank < a.h_stages;  // this CTA had a stage
  if (warp >= 2) {
    const int row = 32 * (warp & 3) + lane;  // TMEM lane: output row of the tile
    float* sums = reinterpret_cast<float*>(base) + row;
#pragma unroll
    for (int c = 0; c < NT / 16; ++c) {
      uint32_t v[16];
      tmem_ld_32x32b_x16(tmem + ((uint32_t)(32 * (warp & 3)) << 16) + 16 * c, v);
      tmem_wait_ld();
#pragma unroll
      for (int i = 0; i < 16; ++i) sums[(16 * c + i) * kUpRows] = some ? __uint_as_float(v[i]) : 0.f;
    }
    tc_fence_before();
  }
  cluster_barrier();
  // Token m goes to CTA m mod S: four outputs per lane, summed in rank order (all
  // the peers' values on their way before the first is used).
  for (int m = (int)rank + (int)S * warp; m < a.M; m += (int)S * (kUpThreads / 32)) {
    const uint32_t at = smem + (uint32_t)(m * kUpRows + 4 * lane) * 4;
    uint32_t p[kUpClusterMax][4];
#pragma unroll
    for (uint32_t c = 0; c < kUpClusterMax; ++c) {
      p[c][0] = p[c][1] = p[c][2] = p[c][3] = 0;
      if (c < S) ld_shared_cluster_v4(mapa_shared(at, c), p[c][0], p[c][1], p[c][2], p[c][3]);
    }
    float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (uint32_t c = 0; c < kUpClusterMax; ++c) {
      t.x += __uint_as_float(p[c][0]);
      t.y += __uint_as_float(p[c][1]);
      t.z += __uint_as_float(p[c][2]);
      t.w += __uint_as_float(p[c][3]);
    }
    const int n = tile * kUpRows + 4 * lane;
    if (n < a.N) *reinterpret_cast<uint2*>(a.y + (int64_t)m * a.N + n) = make_uint2(round2(t.x, t.y), round2(t.z, t.w));
  }
  // No CTA leaves while a peer may still read its sums.
  cluster_barrier();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kCols);
  }
}

// CTAs that split a row tile's stages: as many as two per SM hold, of at least
// three stages each.
int up_split(int tiles, int steps, int sm_count) {
  int s = 1;
  while (s < (int)kUpClusterMax && tiles * s * 2 <= 2 * sm_count && steps >= 3 * 2 * s) s *= 2;
  return s;
}

template <int NT>
cudaError_t up_launch(const LinearLaunch& p, const float* B_cat, const float* h, cudaStream_t s, bool* driver_failed,
                      PFN_cuTensorMapEncodeTiled_v12000 enc) {
  using C = UpCfg<NT>;
  CUtensorMap tm_w, tm_x, tm_sw, tm_sx, tm_b, tm_h;
  const uint64_t groups = (uint64_t)p.K / BKQ;
  bool ok = make_map_codes(enc, &tm_w, p.wq, (uint64_t)p.K / 2, (uint64_t)p.N, kUpRows) &&
            make_map_codes(enc, &tm_x, p.xq, (uint64_t)p.K / 2, (uint64_t)p.M, NT) &&
            make_map_scales(enc, &tm_sw, p.wsf, (uint64_t)((p.N + 127) / 128) * groups, 4) &&
            make_map_scales(enc, &tm_sx, p.xsf, (uint64_t)((p.M + 127) / 128) * groups, 4);
  tm_b = tm_h = tm_w;  // never read without adapters
  if (p.R > 0) {
    ok = ok && make_map_tf32(enc, &tm_b, B_cat, (uint64_t)p.R, (uint64_t)p.N, kUpRows) &&
         make_map_tf32(enc, &tm_h, h, (uint64_t)p.R, (uint64_t)p.M, NT);
  }
  if (!ok) {
    *driver_failed = true;
    return cudaErrorInvalidValue;
  }
  UpArgs a;
  a.y = reinterpret_cast<uint16_t*>(p.y);
  a.M = (int)p.M;
  a.N = p.N;
  a.q_stages = (p.K + 255) / 256;
  a.q_groups = (int)groups;
  a.h_stages = p.R / 32;
  a.wait_limit_ns = p.wait_limit_ns;
  constexpr int smem = (int)(1024 + C::kRing + sizeof(UpControl));
  cudaError_t e = allow_shared_memory((const void*)k_few_up<NT>, smem);
  if (e != cudaSuccess) return e;
  const int tiles = (p.N + kUpRows - 1) / kUpRows;
  const int split = up_split(tiles, a.q_stages + a.h_stages, p.sm_count);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(tiles * split), 1, 1);
  cfg.blockDim = dim3(kUpThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)split;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = p.R > 0 ? 2 : 1;  // without adapters nothing waits for the kernel before
  g_launched.store(true);
  return cudaLaunchKernelEx(&cfg, k_few_up<NT>, tm_w, tm_x, tm_sw, tm_sx, tm_b, tm_h, a);
}

template <int NG>
cudaError_t down_launch(const LinearLaunch& p, const float* A_cat, float* h, cudaStream_t s) {
  const DownArgs d{reinterpret_cast<const uint16_t*>(p.x), A_cat, h, (int)p.M, p.K, p.R};
  k_few_down<NG><<<dim3(p.R / kDownRows * kDownCluster, (p.M + 63) / 64), DownCfg<NG>::kWarps * 32, 0, s>>>(d);
  return cudaGetLastError();
}

}  // namespace

cudaError_t take_few_error(int* value) {
  *value = 0;
  return g_launched.load() ? take_device_error(value) : cudaSuccess;
}

bool few_tokens(int64_t M) { return M <= 128; }

cudaError_t launch_lora_linear_few(const LinearLaunch& p, const float* A_cat, const float* B_cat, float* h,
                                   int* kernels, cudaStream_t s, bool* driver_failed) {
  *kernels = 0;
  *driver_failed = false;
  PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
  if (!enc) {
    *driver_failed = true;
    return cudaErrorNotSupported;
  }
  cudaError_t e = cudaSuccess;
  if (p.R > 0) {
    if (p.M <= 8) e = down_launch<1>(p, A_cat, h, s);
    else if (p.M <= 16) e = down_launch<2>(p, A_cat, h, s);
    else if (p.M <= 32) e = down_launch<4>(p, A_cat, h, s);
    else e = down_launch<8>(p, A_cat, h, s);
    if (e != cudaSuccess) return e;
    *kernels = 1;
  }
  if (p.M <= 16) e = up_launch<16>(p, B_cat, h, s, driver_failed, enc);
  else if (p.M <= 32) e = up_launch<32>(p, B_cat, h, s, driver_failed, enc);
  else if (p.M <= 64) e = up_launch<64>(p, B_cat, h, s, driver_failed, enc);
  else e = up_launch<128>(p, B_cat, h, s, driver_failed, enc);
  if (e == cudaSuccess) *kernels += 1;
  return e;
}

}  // namespace lg
