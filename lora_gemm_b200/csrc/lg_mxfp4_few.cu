// lg_lora_linear_mxfp4 for few tokens (M <= 64): bound by reading the weights
// and factors once, 17/32 bytes per weight and 4 per factor.
//
// The panel kernel gives each SM pair a 256-token panel and computes
// h = x A_cat^T once per panel and SM pair: with one panel that is every
// pair reading all of A_cat, behind a pass that copies the factors to bf16
// (1 x 7168 -> 7168, rank 576: 148 us, 6 % of HBM).  Here the weights are the
// wide operand and the tokens the narrow one:
//
//   k_few_down  h = x A_cat^T: a cluster of eight CTAs per 16 ranks, K spread
//               over its 32 warps, partial sums joined through distributed
//               shared memory.
//   k_few_up    y = deq(x) deq(W)^T + h B_cat^T: a CTA per 32 outputs, K spread
//               over its eight warps, each with a ring of cp.async stages of
//               its own; the warps' sums are joined in a fixed order.
//
// k_few_up is launched as a programmatic dependent: it reads weights while
// k_few_down still runs and waits for h only before the adapters' term.
//
// The products run on mma.sync (m16n8k16, weights as the 16-row operand): at 8
// to 64 tokens the warp's own registers feed it as fast as HBM delivers, without
// the tensor-memory round trip, and a block's scale is applied to its FP32 sum.
// E2M1 codes become f16 (exact); the sum of a block's 32 products is exact in
// FP32 (multiples of 1/4 below 2^11), so the scales 2^(e_x + e_w) go in without
// rounding.  K may be permuted freely within a block as long as both operands
// agree: each lane takes eight consecutive codes, one 32-bit word.
#include <cuda_bf16.h>

#include "lg_internal.h"

namespace lg {

namespace {

constexpr int kUpWarps = 8;
constexpr int kUpRows = 32;                   // outputs per CTA
constexpr int kStageRows = kUpRows * 64;      // bytes of W codes per stage: 128 K
constexpr int kDownWarps = 4;
constexpr int kDownCluster = 8;
constexpr int kDownRows = 16;                 // ranks per cluster

__device__ __forceinline__ uint32_t s_addr(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ float4 ld_stream4(const float* p) {
  float4 v;
  asm volatile("ld.global.L1::no_allocate.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "l"(p));
  return v;
}

// Eight E2M1 codes -> four f16 pairs, exact.
__device__ __forceinline__ void decode8(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
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
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
      "%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 2^(byte - 127): byte 0 is the subnormal 2^-127, 255 is NaN.
__device__ __forceinline__ float e8m0(uint32_t byte) {
  return byte == 255u ? __uint_as_float(0x7FFFFFFFu) : __uint_as_float(byte == 0u ? 0x00400000u : byte << 23);
}
// All four scale bytes of a word are in [63, 190]: the product of two such
// scales is 2^-128 .. 2^126, exact in FP32.
__device__ __forceinline__ bool plain_scales(uint32_t w) {
  const uint32_t v = w + 0x01010101u;
  return ((v ^ (v << 1)) & 0x80808080u) == 0x80808080u;
}

struct UpArgs {
  const uint8_t* xq;
  const uint8_t* xsf;
  const uint8_t* wq;
  const uint8_t* wsf;
  const float* B;       // [N, R]
  const uint16_t* h;    // [M, R] bf16
  uint16_t* y;
  int M, K, N, R;
};

// NG: groups of eight tokens.
template <int NG>
struct UpCfg {
  static constexpr int kX = NG * 8 * 64;                                // x codes per stage
  static constexpr int kStage = kStageRows + kUpRows * 4 + kX + NG * 8 * 4;  // + W scale words, x scale words
  // Two CTAs per SM (227 KB shared, 128 registers a thread) keep 16 warps and
  // over 80 KB of copies in flight.
  static constexpr int kStages = NG == 1 ? 4 : (NG <= 4 ? 3 : 2);
  static constexpr int kWarp = kStage * kStages;
  static constexpr int kSums = kUpWarps * kUpRows * NG * 8 * 4;
  static constexpr int kSmem = kUpWarps * kWarp > kSums ? kUpWarps * kWarp : kSums;
};

__device__ __forceinline__ uint64_t pair2(float a, float b) {
  uint64_t v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(a), "f"(b));
  return v;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t v;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(v) : "l"(a), "l"(b));
  return v;
}
// (c, c1) += (d, d1) * s, two FP32 lanes in one instruction.
__device__ __forceinline__ void fma2(float& c, float& c1, float d, float d1, uint64_t s) {
  uint64_t v = pair2(c, c1);
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(v) : "l"(pair2(d, d1)), "l"(s));
  asm("mov.b64 {%0, %1}, %2;" : "=f"(c), "=f"(c1) : "l"(v));
}

// One stage of 128 K: acc += deq(W) deq(x)^T.  PLAIN: every scale's exponent
// field is in [63, 190] (plain_scales), so a scale is its byte in FP32's
// exponent field and the product of two is exact.
template <int NG, bool PLAIN>
__device__ __forceinline__ void up_stage(uint32_t st, uint32_t xc, int g, int t, const uint32_t (&ws)[4],
                                         const uint32_t (&xs)[NG][2], float (&acc)[2][NG][4]) {
#pragma unroll
  for (int c = 0; c < 4; ++c) {  // the four blocks of 32
    uint32_t w[4][4];
    float sw[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = i * 8 + g;
      decode8(lds32(st + r * 64 + ((c ^ ((r >> 1) & 3)) << 4) + t * 4), w[i]);
      sw[i] = PLAIN ? __uint_as_float((c == 3 ? ws[i] >> 1 : ws[i] << (23 - 8 * c)) & 0x7F800000u)
                    : e8m0((ws[i] >> (8 * c)) & 255u);
    }
#pragma unroll
    for (int n = 0; n < NG; ++n) {
      uint32_t x[4];
      const int r = n * 8 + g;
      decode8(lds32(xc + r * 64 + ((c ^ ((r >> 1) & 3)) << 4) + t * 4), x);
      float sx[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        sx[e] = PLAIN ? __uint_as_float((c == 3 ? xs[n][e] >> 1 : xs[n][e] << (23 - 8 * c)) & 0x7F800000u)
                      : e8m0((xs[n][e] >> (8 * c)) & 255u);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float d[4] = {0.f, 0.f, 0.f, 0.f};
        mma_f16(d, w[2 * i][0], w[2 * i + 1][0], w[2 * i][1], w[2 * i + 1][1], x[0], x[1]);
        mma_f16(d, w[2 * i][2], w[2 * i + 1][2], w[2 * i][3], w[2 * i + 1][3], x[2], x[3]);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float(&o)[4] = acc[i][n];
          const float s = sw[2 * i + e];
          if (PLAIN) {
            fma2(o[2 * e], o[2 * e + 1], d[2 * e], d[2 * e + 1], mul2(pair2(sx[0], sx[1]), pair2(s, s)));
          } else {
            // The smaller scale first: no step leaves FP32's range unless the
            // result does.  (fminf drops a NaN, the sum s + sx keeps it.)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const float lo = fminf(s, sx[k]), hi = s + sx[k] == s + sx[k] ? fmaxf(s, sx[k]) : s + sx[k];
              o[2 * e + k] += (d[2 * e + k] * lo) * hi;
            }
          }
        }
      }
    }
  }
}

template <int NG>
__global__ void __launch_bounds__(kUpWarps * 32, 2) k_few_up(const UpArgs a) {
  using C = UpCfg<NG>;
  extern __shared__ __align__(16) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int n0 = blockIdx.x * kUpRows;
  // The steps of this CTA: groups of 128 K, then 16 ranks of the adapters'
  // term each.  Warp w takes steps w, w + 8, ...
  const int groups = a.K / 128;
  const int steps = groups + a.R / 16;
  const int64_t row_bytes = a.K / 2;
  const uint32_t ring = s_addr(smem) + warp * C::kWarp;
  bool waited = false;

  // Stage layout: W codes [32 rows][64 B] (or 16 FP32 ranks of B_cat), 16-byte
  // piece c of row r at c ^ ((r / 2) mod 4): no bank conflicts when eight rows
  // are read at one piece; W scale words [32]; x codes [NG * 8][64 B] (or 32 B
  // of h) likewise; x scale words.
  constexpr uint32_t kWs = kStageRows, kXc = kWs + kUpRows * 4, kXs = kXc + C::kX;
  auto fetch = [&](int step, int stage) {
    const uint32_t st = ring + stage * C::kStage;
    if (step < groups) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = i * 8 + g;
        copy16(st + r * 64 + ((t ^ ((r >> 1) & 3)) << 4), a.wq + (n0 + r) * row_bytes + step * 64 + t * 16);
      }
      // Row r of a group of 128 has its four scale bytes at 16 (r mod 32) + 4 (r / 32).
      copy4(st + kWs + lane * 4,
            a.wsf + (((int64_t)(n0 >> 7) * groups + step) << 9) + 16 * lane + 4 * ((n0 & 127) >> 5));
#pragma unroll
      for (int n = 0; n < NG; ++n) {
        const int r = n * 8 + g;
        if (r < a.M) copy16(st + kXc + r * 64 + ((t ^ ((r >> 1) & 3)) << 4), a.xq + r * row_bytes + step * 64 + t * 16);
      }
#pragma unroll
      for (int n = 0; n < (NG + 3) / 4; ++n) {
        const int r = n * 32 + lane;
        if (r < a.M && r < NG * 8) copy4(st + kXs + r * 4, a.xsf + ((int64_t)step << 9) + 16 * lane + 4 * n);
      }
    } else if (step < steps) {
      const int r0 = (step - groups) * 16;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = i * 8 + g;
        copy16(st + r * 64 + ((t ^ ((r >> 1) & 3)) << 4), a.B + (int64_t)(n0 + r) * a.R + r0 + t * 4);
      }
      if (!waited) asm volatile("griddepcontrol.wait;" ::: "memory");  // h is there
      waited = true;
#pragma unroll
      for (int n = 0; n < (NG + 1) / 2; ++n) {
        const int r = n * 16 + (lane >> 1), c = lane & 1;
        if (r < a.M && r < NG * 8)
          copy16(st + kXc + r * 64 + ((c ^ ((r >> 1) & 3)) << 4), a.h + (int64_t)r * a.R + r0 + c * 8);
      }
    }
    copy_commit();
  };
  // Tokens past M: codes (or h) 0 under scale 1, never overwritten.
  for (int st = 0; st < C::kStages; ++st) {
    uint8_t* base = smem + warp * C::kWarp + st * C::kStage;
    for (int i = lane; i < C::kX / 16; i += 32) reinterpret_cast<uint4*>(base + kXc)[i] = make_uint4(0, 0, 0, 0);
    for (int i = lane; i < NG * 8; i += 32) reinterpret_cast<uint32_t*>(base + kXs)[i] = 0x7F7F7F7Fu;
  }
  __syncwarp();
#pragma unroll
  for (int s = 0; s < C::kStages; ++s) fetch(warp + s * kUpWarps, s);

  float acc[2][NG][4];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
#pragma unroll
    for (int n = 0; n < NG; ++n) {
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[i][n][e] = 0.f;
    }
  }
  int stage = 0;
  for (int step = warp; step < steps; step += kUpWarps) {
    copy_wait<C::kStages - 1>();
    __syncwarp();  // every lane's pieces of this stage have landed
    const uint32_t st = ring + stage * C::kStage;
    if (step < groups) {
      uint32_t ws[4];  // scale words of rows g, g + 8, g + 16, g + 24
#pragma unroll
      for (int i = 0; i < 4; ++i) ws[i] = lds32(st + kWs + (i * 8 + g) * 4);
      uint32_t xs[NG][2];  // of tokens 8 n + 2 t and + 1
      bool plain = plain_scales(ws[0]) && plain_scales(ws[1]) && plain_scales(ws[2]) && plain_scales(ws[3]);
#pragma unroll
      for (int n = 0; n < NG; ++n) {
        xs[n][0] = lds32(st + kXs + (n * 8 + 2 * t) * 4);
        xs[n][1] = lds32(st + kXs + (n * 8 + 2 * t + 1) * 4);
        plain = plain && plain_scales(xs[n][0]) && plain_scales(xs[n][1]);
      }
      if (__all_sync(0xffffffffu, plain)) {
        up_stage<NG, true>(st, st + kXc, g, t, ws, xs, acc);
      } else {
        up_stage<NG, false>(st, st + kXc, g, t, ws, xs, acc);
      }
    } else {
      // 16 ranks: lane t has ranks 4 t .. 4 t + 3 of its rows and tokens.
      uint32_t w[4][2];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = i * 8 + g;
        float4 v;
        asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                     : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                     : "r"(st + r * 64 + ((t ^ ((r >> 1) & 3)) << 4))
                     : "memory");
        w[i][0] = round2(v.x, v.y);
        w[i][1] = round2(v.z, v.w);
      }
#pragma unroll
      for (int n = 0; n < NG; ++n) {
        const int r = n * 8 + g;
        uint32_t x0, x1;
        asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];"
                     : "=r"(x0), "=r"(x1)
                     : "r"(st + kXc + r * 64 + (((t >> 1) ^ ((r >> 1) & 3)) << 4) + (t & 1) * 8)
                     : "memory");
#pragma unroll
        for (int i = 0; i < 2; ++i) mma_bf16(acc[i][n], w[2 * i][0], w[2 * i + 1][0], w[2 * i][1], w[2 * i + 1][1], x0, x1);
      }
    }
    __syncwarp();  // the stage has been read by every lane
    fetch(step + C::kStages * kUpWarps, stage);
    if (++stage == C::kStages) stage = 0;
  }
  copy_wait<0>();
  // Also where no adapter step was this warp's: the grid ends after k_few_down.
  if (a.R > 0 && !waited) asm volatile("griddepcontrol.wait;" ::: "memory");

  // Join the warps' sums in their order: [warp][token][32 outputs].
  __syncthreads();  // every warp is done with its ring
  float* sums = reinterpret_cast<float*>(smem);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
#pragma unroll
    for (int n = 0; n < NG; ++n) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        sums[(warp * NG * 8 + n * 8 + 2 * t + (e & 1)) * kUpRows + 16 * i + 8 * (e >> 1) + g] = acc[i][n][e];
      }
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < a.M * (kUpRows / 2); i += kUpWarps * 32) {
    const int m = i / (kUpRows / 2), r = i % (kUpRows / 2) * 2;
    float2 v = make_float2(0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kUpWarps; ++w) {
      const float2 p = *reinterpret_cast<const float2*>(&sums[(w * NG * 8 + m) * kUpRows + r]);
      v.x += p.x;
      v.y += p.y;
    }
    *reinterpret_cast<__nv_bfloat162*>(a.y + (int64_t)m * a.N + n0 + r) = __floats2bfloat162_rn(v.x, v.y);
  }
}

struct DownArgs {
  const uint16_t* x;  // [M, K] bf16
  const float* A;     // [R, K]
  uint16_t* h;        // [M, R] bf16
  int M, K, R;
};

// h[m, r0 .. r0 + 15]: cluster blockIdx.x / 8, its 32 warps take every 32nd
// step of 32 K.
template <int NG>
__global__ void __cluster_dims__(kDownCluster, 1, 1) __launch_bounds__(kDownWarps * 32) k_few_down(const DownArgs a) {
  __shared__ float sums[kDownWarps][NG * 8][kDownRows];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  uint32_t rank;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
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
#pragma unroll 4
  for (int s = (int)rank * kDownWarps + warp; s < steps; s += kDownCluster * kDownWarps) {
    uint32_t w[2][4];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float* p = pa + (int64_t)i * 8 * a.K + s * 32;
      round8(ld_stream4(p), ld_stream4(p + 4), w[i]);
    }
#pragma unroll
    for (int n = 0; n < NG; ++n) {
      uint4 x = make_uint4(0, 0, 0, 0);
      if (n * 8 + g < a.M) x = __ldg(reinterpret_cast<const uint4*>(px + (int64_t)n * 8 * a.K + s * 32));
      mma_bf16(acc[n], w[0][0], w[1][0], w[0][1], w[1][1], x.x, x.y);
      mma_bf16(acc[n], w[0][2], w[1][2], w[0][3], w[1][3], x.z, x.w);
    }
  }
#pragma unroll
  for (int n = 0; n < NG; ++n) {
#pragma unroll
    for (int e = 0; e < 4; ++e) sums[warp][n * 8 + 2 * t + (e & 1)][8 * (e >> 1) + g] = acc[n][e];
  }
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
  // Each CTA joins an eighth of the cluster's M x 16 sums, CTA by CTA and warp
  // by warp.
  for (int i = (int)rank * kDownWarps * 32 + threadIdx.x; i < a.M * kDownRows; i += kDownCluster * kDownWarps * 32) {
    const int m = i / kDownRows, r = i % kDownRows;
    float v = 0.f;
#pragma unroll
    for (int c = 0; c < kDownCluster; ++c) {
      uint32_t peer;
      asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(peer) : "r"(s_addr(&sums[0][m][r])), "r"(c));
#pragma unroll
      for (int w = 0; w < kDownWarps; ++w) {
        float p;
        asm volatile("ld.shared::cluster.f32 %0, [%1];"
                     : "=f"(p)
                     : "r"(peer + (uint32_t)(w * NG * 8 * kDownRows * 4))
                     : "memory");
        v += p;
      }
    }
    // Rounded to bf16 as the other layers round h for the up-projection.
    a.h[(int64_t)m * a.R + r0 + r] = __bfloat16_as_ushort(__float2bfloat16_rn(v));
  }
  // No CTA leaves while a peer may still read its sums.
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

template <int NG>
cudaError_t few_launch(const LinearLaunch& p, const float* A_cat, const float* B_cat, uint16_t* h, int* kernels,
                       cudaStream_t s) {
  using C = UpCfg<NG>;
  *kernels = 0;
  // A constant, so that calls from several host threads cannot lower it.
  cudaError_t e = cudaFuncSetAttribute((const void*)k_few_up<NG>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (e != cudaSuccess) return e;
  if (p.R > 0) {
    const DownArgs d{reinterpret_cast<const uint16_t*>(p.x), A_cat, h, (int)p.M, p.K, p.R};
    k_few_down<NG><<<p.R / kDownRows * kDownCluster, kDownWarps * 32, 0, s>>>(d);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    *kernels = 1;
  }
  const UpArgs u{reinterpret_cast<const uint8_t*>(p.xq), reinterpret_cast<const uint8_t*>(p.xsf),
                 reinterpret_cast<const uint8_t*>(p.wq), reinterpret_cast<const uint8_t*>(p.wsf),
                 B_cat, h, reinterpret_cast<uint16_t*>(p.y), (int)p.M, p.K, p.N, p.R};
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p.N / kUpRows), 1, 1);
  cfg.blockDim = dim3(kUpWarps * 32, 1, 1);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = p.R > 0 ? 1 : 0;  // without adapters nothing waits for the kernel before
  e = cudaLaunchKernelEx(&cfg, k_few_up<NG>, u);
  if (e == cudaSuccess) *kernels += 1;
  return e;
}

}  // namespace

bool few_tokens(int64_t M) { return M <= 64; }

cudaError_t launch_lora_linear_few(const LinearLaunch& p, const float* A_cat, const float* B_cat, uint16_t* h,
                                   int* kernels, cudaStream_t s) {
  if (p.M <= 8) return few_launch<1>(p, A_cat, B_cat, h, kernels, s);
  if (p.M <= 16) return few_launch<2>(p, A_cat, B_cat, h, kernels, s);
  if (p.M <= 24) return few_launch<3>(p, A_cat, B_cat, h, kernels, s);
  if (p.M <= 32) return few_launch<4>(p, A_cat, B_cat, h, kernels, s);
  if (p.M <= 48) return few_launch<6>(p, A_cat, B_cat, h, kernels, s);
  return few_launch<8>(p, A_cat, B_cat, h, kernels, s);
}

}  // namespace lg
