// The norms between two transformer blocks, with the gate, the scaled residual
// and the modulation, forward and backward:
//
//   h' = alpha h + gate * N_post(b),   n = N_pre(h') (1 + scale) + shift
//
// (RMS or layer norms over the D values of a row; gate, scale and shift per
// segment of rows).  Both directions touch every row once and are bound by
// HBM; the statistics are sums over the row held in registers, FP32 but for the
// forward's last additions (row_sum).  Squares are FP32's: a row whose sum of
// squares passes 3.4e38 has an infinite deviation.
//
// Forward: one row per group of warps, each thread holding CH chunks of eight
// consecutive values, 64 registers so that four CTAs of a 7168-wide row share an
// SM.  Every product and sum of the formula rounds by itself, in its order (but for the
// squares, which are fused into their sum), so that a row agrees to the bit with the
// formula in elementary FP32 operations wherever the deviations do, and with it the
// codes, which a last bit can flip: of 65,536 rows of 7168 (random streams) 20 codes
// differ from such an evaluation's, 72 with fused multiply-adds and FP32 row sums.
// The row's data are read and written past L1, which is left to the modulation
// vectors: 3 x 4 D bytes that every row of a segment reads again (more than the
// row itself), and that the rows resident on an SM share there, in 256-bit loads.
// 66601 x 7168 bf16: 640 us without codes (91 % of measured HBM), 750 us with
// MXFP4 codes (83 %: issue slots, the quantizer's share).
//
// Backward: with x^ a normalised row, r its reciprocal deviation and g the
// gradient there, the input's gradient is
//
//   RMS:    r (g - x^ mean(g x^))
//   layer:  r (g - mean g - x^ mean(g x^))
//
// A CTA takes consecutive rows of one segment, each thread always the same
// columns, so the column sums dgate, dscale and dshift stay in registers over
// the CTA's rows; one partial row per CTA goes to the workspace and a second
// kernel adds the partials of a segment in a fixed order.
#include <atomic>
#include <initializer_list>

#include "lg_internal.h"
#include "lg_mx.cuh"
#include "lg_pipeline.cuh"

namespace lg {

namespace {

constexpr int kNone = 0, kLayer = 2;  // LG_NORM_NONE, LG_NORM_LAYER (LG_NORM_RMS needs no test)
constexpr int kCodesMxfp4 = 2;  // LG_CODES_MXFP4; any other nonzero format is MXFP8
constexpr int kMaxWarps = 32;  // of a row in one CTA

std::atomic<bool> g_launched{false};  // a kernel that waits, so that the error word may be set

// Eight consecutive values of a row as FP32; loads and stores of the stream
// data do not allocate in L1.
__device__ __forceinline__ uint4 ld_stream(const void* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p)
               : "memory");
  return v;
}
__device__ __forceinline__ void st_stream(void* p, uint4 v) {
  asm volatile("st.global.L1::no_allocate.v4.u32 [%0], {%1, %2, %3, %4};" ::"l"(p), "r"(v.x), "r"(v.y), "r"(v.z),
               "r"(v.w)
               : "memory");
}
__device__ __forceinline__ void st_stream(void* p, uint32_t v) {
  asm volatile("st.global.L1::no_allocate.u32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}
__device__ __forceinline__ void st_stream(void* p, uint2 v) {
  asm volatile("st.global.L1::no_allocate.v2.u32 [%0], {%1, %2};" ::"l"(p), "r"(v.x), "r"(v.y) : "memory");
}
__device__ __forceinline__ void unpack8(uint4 q, float (&v)[8]) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&b);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Two FP32 values in a register pair, for the instructions that work on both
// (the backward pass; the forward one, which waits for memory, ran slower so).
struct F2 {
  uint64_t v;
};
__device__ __forceinline__ F2 f2(float a, float b) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 split(F2 a) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a.v));
  return r;
}
__device__ __forceinline__ F2 operator+(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 operator*(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 fma(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
// Eight bf16 values as four pairs.
__device__ __forceinline__ void unpack8(uint4 q, F2 (&v)[4]) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = f2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
}
__device__ __forceinline__ uint4 pack8(const F2 (&v)[4]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 p = split(v[i]);
    const __nv_bfloat162 b = __floats2bfloat162_rn(p.x, p.y);
    w[i] = *reinterpret_cast<const uint32_t*>(&b);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Eight FP32 values of a thread are 32 bytes: one 256-bit access where the
// pointers allow it (`wide`).  As two of 128 bits, each takes every second half
// of its warp's sectors, and both take the passes of the whole.
__device__ __forceinline__ void ld_stream8(const float* p, bool wide, uint4& a, uint4& b) {
  if (wide) {
    asm volatile("ld.global.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(a.x), "=r"(a.y), "=r"(a.z), "=r"(a.w), "=r"(b.x), "=r"(b.y), "=r"(b.z), "=r"(b.w)
                 : "l"(p)
                 : "memory");
  } else {
    a = ld_stream(p);
    b = ld_stream(p + 4);
  }
}
__device__ __forceinline__ void st_stream8(float* p, bool wide, uint4 a, uint4 b) {
  if (wide) {
    asm volatile("st.global.L1::no_allocate.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(a.x), "r"(a.y),
                 "r"(a.z), "r"(a.w), "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
                 : "memory");
  } else {
    st_stream(p, a);
    st_stream(p + 4, b);
  }
}

// Raw bits of eight stream values: 16 bytes (bf16) or 32 (FP32).
template <bool FP32>
struct Raw8 {
  uint4 q[FP32 ? 2 : 1];
  __device__ __forceinline__ void load(const void* base, int64_t at, bool wide) {
    if constexpr (FP32) ld_stream8(reinterpret_cast<const float*>(base) + at, wide, q[0], q[1]);
    else q[0] = ld_stream(reinterpret_cast<const uint16_t*>(base) + at);
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < (FP32 ? 2 : 1); ++i) q[i] = make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    if constexpr (FP32) {
      v[0] = __uint_as_float(q[0].x), v[1] = __uint_as_float(q[0].y);
      v[2] = __uint_as_float(q[0].z), v[3] = __uint_as_float(q[0].w);
      v[4] = __uint_as_float(q[1].x), v[5] = __uint_as_float(q[1].y);
      v[6] = __uint_as_float(q[1].z), v[7] = __uint_as_float(q[1].w);
    } else {
      unpack8(q[0], v);
    }
  }
  __device__ __forceinline__ void get(F2 (&v)[4]) const {
    if constexpr (FP32) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        v[2 * i] = f2(__uint_as_float(q[i].x), __uint_as_float(q[i].y));
        v[2 * i + 1] = f2(__uint_as_float(q[i].z), __uint_as_float(q[i].w));
      }
    } else {
      unpack8(q[0], v);
    }
  }
};
// Stores eight values in the stream's type; the scalar form's v becomes what was
// stored.
template <bool FP32>
__device__ __forceinline__ void store_stream8(void* base, int64_t at, bool wide, float (&v)[8]) {
  if constexpr (FP32) {
    st_stream8(reinterpret_cast<float*>(base) + at, wide,
               make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])),
               make_uint4(__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]), __float_as_uint(v[7])));
  } else {
    const uint4 q = pack8(v);
    st_stream(reinterpret_cast<uint16_t*>(base) + at, q);
    unpack8(q, v);
  }
}
template <bool FP32>
__device__ __forceinline__ void store_stream8(void* base, int64_t at, bool wide, const F2 (&v)[4]) {
  if constexpr (FP32) {
    uint4 q[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float2 a = split(v[2 * i]), b = split(v[2 * i + 1]);
      q[i] = make_uint4(__float_as_uint(a.x), __float_as_uint(a.y), __float_as_uint(b.x), __float_as_uint(b.y));
    }
    st_stream8(reinterpret_cast<float*>(base) + at, wide, q[0], q[1]);
  } else {
    st_stream(reinterpret_cast<uint16_t*>(base) + at, pack8(v));
  }
}
// Eight values of a segment's modulation row (cached), or `other` without one.
__device__ __forceinline__ void load_mod8(const float* base, int64_t at, bool wide, float other, float (&v)[8]) {
  if (!base) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = other;
  } else if (wide) {
    asm("ld.global.nc.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7])
        : "l"(base + at));
  } else {
    const float4 a = __ldg(reinterpret_cast<const float4*>(base + at));
    const float4 b = __ldg(reinterpret_cast<const float4*>(base + at + 4));
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
    v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  }
}

// Sum over each `n` lanes that differ in the low bits, n a power of two.
template <typename T>
__device__ __forceinline__ T lane_sum(T v, int n) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    if (o < n) v += __shfl_xor_sync(0xffffffffu, v, o);
  }
  return v;
}

// Sum over the `warps` warps of a row.  The roundings of its last additions are
// not averaged over others and move the whole row, so those are FP64's (they
// cost 14 us of 750 at 66601 x 7168).  Each call of a row has shared memory of
// its own (`slot`): no barrier is needed before the next call.
__device__ __forceinline__ double row_sum(float v, int warps, float* slot) {
  if (warps == 1) return lane_sum((double)v, 32);
  v = lane_sum(v, 32);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (lane == 0) slot[warp] = v;
  __syncthreads();
  const int n = 2 << (31 - __clz(warps - 1));  // `warps`, up to a power of two
  const int w = lane & (n - 1);
  return lane_sum(w < warps ? (double)slot[w] : 0.0, n);
}

struct NormArgs {
  const void* h;
  const void* b;
  const float* gate;
  const float* scale;
  const float* shift;
  void* h_out;
  void* n;
  uint8_t* codes;
  uint8_t* scales;
  int64_t M;
  int64_t rows;  // M, or with codes M rounded up to 128 (the padding's scale bytes are 0)
  int64_t seg;
  int D, post, pre, format;
  bool wide_stream, wide_mods;  // 32-byte aligned
  float alpha, eps;
};

// Normalises the row's values in place; `live` masks chunks past D.
template <int CH>
__device__ __forceinline__ void normalise(float (&v)[CH][8], const bool (&live)[CH], int kind, float eps, float d,
                                          int warps, float (*slot)[kMaxWarps]) {
  if (kind == kLayer) {
    float s = 0.f;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      float p = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) p += v[c][i];  // chunks past D hold zeros
      s += p;
    }
    const float mean = (float)row_sum(s, warps, slot[0]) / d;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[c][i] = live[c] ? v[c][i] - mean : 0.f;
    }
  }
  float q = 0.f;
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    float p = 0.f;  // short chains: their roundings are what moves r
#pragma unroll
    for (int i = 0; i < 8; ++i) p = fmaf(v[c][i], v[c][i], p);
    q += p;
  }
  const float r = rsqrtf((float)row_sum(q, warps, slot[1]) / d + eps);
#pragma unroll
  for (int c = 0; c < CH; ++c) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[c][i] *= r;
  }
}

// blockDim.x = 32 * warps for one row, or (ONE) several rows of one warp each.  A
// warp has CH * 256 consecutive columns, so that a thread's chunks lie 256 columns
// apart and every array needs one address.
template <bool FP32, int CH, bool ONE>
__global__ void __launch_bounds__(ONE ? 128 : (CH == 4 ? 512 : 1024), ONE || FP32 || CH < 4 ? 1 : 2) k_block_norm(const NormArgs a) {
  __shared__ float slots[4][kMaxWarps];
  const int warps = ONE ? 1 : (int)blockDim.x >> 5;
  const int t = ONE ? (int)threadIdx.x & 31 : (int)threadIdx.x;
  const int64_t row = ONE ? (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5) : (int64_t)blockIdx.x;
  if (row >= a.rows) return;
  if (row >= a.M) {  // the scale bytes of rows past M
    for (int kb = t; kb < a.D / 32; kb += 32 * warps) a.scales[mx_scale_offset(row, kb, a.D / 128)] = 0;
    return;
  }
  const int col = (t >> 5) * (CH * 256) + (t & 31) * 8;  // of chunk 0
  const int64_t at = row * a.D + col;
  const int64_t mod = row / a.seg * a.D + col;
  bool live[CH];
  Raw8<FP32> raw[CH];
  float v[CH][8];
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    live[c] = col + 256 * c < a.D;
    raw[c].zero();
    if (live[c]) raw[c].load(a.h, at + 256 * c, a.wide_stream);
  }
  if (a.b) {
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      uint4 q = make_uint4(0, 0, 0, 0);
      if (live[c]) q = ld_stream(reinterpret_cast<const uint16_t*>(a.b) + at + 256 * c);
      unpack8(q, v[c]);
    }
    if (a.post != kNone) normalise<CH>(v, live, a.post, a.eps, (float)a.D, warps, slots);
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      if (!live[c]) continue;
      float g[8], h[8];
      load_mod8(a.gate, mod + 256 * c, a.wide_mods, 1.0f, g);
      raw[c].get(h);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[c][i] = __fadd_rn(__fmul_rn(g[i], v[c][i]), __fmul_rn(a.alpha, h[i]));
      store_stream8<FP32>(a.h_out, at + 256 * c, a.wide_stream, v[c]);
    }
  } else {
#pragma unroll
    for (int c = 0; c < CH; ++c) raw[c].get(v[c]);
  }
  if (a.pre == kNone) return;
  normalise<CH>(v, live, a.pre, a.eps, (float)a.D, warps, slots + 2);
  // Chunk c's K group is 2 c after chunk 0's: 1024 bytes on.
  uint8_t* sf = a.scales + mx_scale_offset(row, col / 128 * 4, a.D / 128);
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    uint4 q = make_uint4(0, 0, 0, 0);
    if (live[c]) {
      float s[8], f[8];
      load_mod8(a.scale, mod + 256 * c, a.wide_mods, 0.0f, s);
      load_mod8(a.shift, mod + 256 * c, a.wide_mods, 0.0f, f);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[c][i] = __fadd_rn(__fmul_rn(v[c][i], 1.0f + s[i]), f[i]);
      q = pack8(v[c]);
      if (a.n) st_stream(reinterpret_cast<uint16_t*>(a.n) + at + 256 * c, q);
    }
    if (a.format != 0) {
      // D is a multiple of 128 here, so four lanes hold one block, all live or all not.
      const uint32_t w[4] = {q.x, q.y, q.z, q.w};
      uint32_t sb;
      if (a.format == kCodesMxfp4) {
        sb = mxfp4_scale_byte(mx_block_max(w));
        if (live[c]) st_stream(a.codes + at / 2 + 128 * c, mxfp4_codes8(w, sb));
      } else {
        float m = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          m = fmaxf(m, fmaxf(fabsf(__uint_as_float(w[i] << 16)), fabsf(__uint_as_float(w[i] & 0xFFFF0000u))));
        }
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
        sb = mxfp8_scale_byte(m);
        if (live[c]) st_stream(a.codes + at + 256 * c, mxfp8_codes8(w, sb));
      }
      // The four bytes of a K group from its 16 lanes, one store.
      sb |= __shfl_down_sync(0xffffffffu, sb, 4) << 8;
      sb |= __shfl_down_sync(0xffffffffu, sb, 8) << 16;
      if (live[c] && (t & 15) == 0) st_stream(sf + 1024 * c, sb);
    }
  }
}

// ---------------------------------------------------------------------------
// Backward.
// ---------------------------------------------------------------------------
constexpr int kBackStagesMax = 4;
// A backward CTA: at most 448 threads (of eight columns each), two per SM, so 72
// registers a thread.  FP32 rows hold more of them (spills at 72): where one CTA
// of up to 256 threads has the row, three per SM, 80 registers (33001 x 1024: 156
// us against 198); a wider row on more CTAs of that size loses more to their
// meeting (33001 x 7168 on four: 1227 us against 946 on two; 33001 x 4096, where
// two are 256 threads wide as well, would gain: 549 on two of these, 684 now).
constexpr int kBackThreads = 448;
constexpr int kBackSmem = 106 * 1024;  // modulation and row stages
template <bool FP32, int SPLIT>
struct Back {
  static constexpr bool kNarrow = FP32 && SPLIT == 1;
  static constexpr int kThreads = kNarrow ? 256 : kBackThreads;
  static constexpr int kCtas = kNarrow ? 3 : 2;
  static constexpr int kSmem = kNarrow ? 70 * 1024 : kBackSmem;
};

struct BackArgs {
  const void* dn;
  const void* dh_out;
  const void* h;
  const void* b;
  const float* gate;
  const float* scale;
  void* dh;
  void* db;
  float* sums[3];     // dgate, dscale, dshift: rows of `sum_stride` floats, one per chunk (or per segment, direct)
  int64_t sum_stride;
  int64_t M;
  int64_t seg;
  int64_t seg_chunks;   // chunks of a full segment; the last segment may have fewer
  int64_t segments;
  int64_t chunk_rows;
  int D, post, pre, stages;
  bool wide;  // dh is 32-byte aligned
  float alpha, eps;
  unsigned long long wait_limit_ns;
};

__device__ __forceinline__ uint32_t smem_addr(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Wait until at most n (0 .. 3) of this thread's newest groups are in flight.
__device__ __forceinline__ void cp_async_wait(int n) {
  if (n == 0) asm volatile("cp.async.wait_group 0;" ::: "memory");
  else if (n == 1) asm volatile("cp.async.wait_group 1;" ::: "memory");
  else if (n == 2) asm volatile("cp.async.wait_group 2;" ::: "memory");
  else asm volatile("cp.async.wait_group 3;" ::: "memory");
}

__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// One 32-bit value into a CTA of the cluster, counted on that CTA's mbarrier: the
// barrier's completion makes it visible, without a fence that would also wait
// for this thread's stores to global memory.
__device__ __forceinline__ void store_async(uint32_t cluster_addr, float v, uint32_t cluster_bar) {
  asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.b32 [%0], %1, [%2];" ::"r"(cluster_addr),
               "r"(__float_as_uint(v)), "r"(cluster_bar)
               : "memory");
}

// What the warps of a row's CTAs need to meet: the places of their sums, and the
// mbarrier that counts their arrival (SPLIT > 1).  A pair of these alternates
// from row to row: a CTA writes a peer's slot for the next row but one only
// after that peer's warps have all sent the row between, having read this one.
// Sums of N <= 8 values over all threads of the SPLIT CTAs that share a row, in
// every thread.  Within a warp each step exchanges half of the eight values a
// lane still holds with the lane whose bit differs (9 shuffles instead of 40):
// value i ends in lanes 4 i .. 4 i + 3.  Every warp leaves its sums in all
// SPLIT CTAs' slot, at the same place, so that all add them up in the same order.
template <int SPLIT>
struct Slots {
  static constexpr int kWarps = SPLIT * (SPLIT == 8 ? 8 : 14);  // at most, of a row
  static constexpr int kReads = (kWarps + 3) / 4;
  float v[8][68];  // 64 warps and four more: eight rows of four reads fall into 32 banks
  uint64_t bar;
};
// False when the wait for the peers ran out.
template <int SPLIT, int N>
__device__ __forceinline__ bool row_group_sums(float (&sum)[N], int warps, uint32_t rank, Slots<SPLIT>& slot,
                                               uint32_t parity, uint64_t limit_ns, volatile int* abort_flag) {
  bool ok = true;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = i < N ? sum[i] : 0.f;
#pragma unroll
  for (int half = 4; half >= 1; half >>= 1) {
    const bool up = lane & (4 * half);
#pragma unroll
    for (int i = 0; i < half; ++i) {
      const float give = up ? v[i] : v[i + half];
      const float keep = up ? v[i + half] : v[i];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, give, 4 * half);
    }
  }
  float total = v[0];
  total += __shfl_xor_sync(0xffffffffu, total, 2);
  total += __shfl_xor_sync(0xffffffffu, total, 1);
  if (SPLIT > 1 || warps > 1) {
    const int idx = lane >> 2, sub = lane & 3;
    float* mine = &slot.v[idx][(int)rank * warps + warp];
    if constexpr (SPLIT == 1) {
      if (sub == 0) *mine = total;
      __syncthreads();
    } else {
      const uint32_t bar = smem_u32(&slot.bar);
      if (threadIdx.x == 0) mbar_arrive_expect_tx(bar, (uint32_t)(SPLIT * warps * 8 * 4));
      if (sub == 0) {
        const uint32_t at = smem_u32(mine);
#pragma unroll
        for (uint32_t c = 0; c < SPLIT; ++c) store_async(mapa_shared(at, c), total, mapa_shared(bar, c));
      }
      ok = wait_limited(bar, parity, limit_ns, abort_flag, true);
      __syncwarp();
    }
    // A fixed number of reads: places that no warp writes hold zero.
    total = 0.f;
#pragma unroll
    for (int w = 0; w < Slots<SPLIT>::kReads; ++w) total += slot.v[idx][4 * w + sub];
    total += __shfl_xor_sync(0xffffffffu, total, 2);
    total += __shfl_xor_sync(0xffffffffu, total, 1);
  }
#pragma unroll
  for (int i = 0; i < N; ++i) sum[i] = __shfl_sync(0xffffffffu, total, 4 * i);
  return ok;
}
// The two halves of N pairs added up.
template <int N>
__device__ __forceinline__ void fold(const F2 (&p)[N], float (&q)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float2 h = split(p[i]);
    q[i] = h.x + h.y;
  }
}

// A cluster of SPLIT CTAs: consecutive rows of one segment; every thread always
// has the same eight columns.  A row of 7168 is two CTAs of 448 threads rather
// than one of 896: the three column sums fill the registers of an SM either way
// (one CTA of 896 threads, or two of 448), but two CTAs of different clusters are
// at different points of their rows, and one works while the other waits for its
// row's sums.  Rows arrive through a ring of shared-memory stages filled by
// cp.async: every thread copies and reads its own 16-byte pieces, so the ring
// needs no barrier, and the rows in flight cost no registers.  Gate and scale
// are laid out in shared memory by thread (read in place, a thread's eight FP32
// values are 32 bytes from its neighbour's and every load takes twice the passes).
//
// Without a layer norm all row sums come from one pass.  With x, b the rows, g =
// dn (1 + scale), t = gate:
//   rx^2 = D / sum x^2, ru^2 = D / sum b^2 (+ eps),   k = rx^2 mean(g x)
//   dh' = dh_out + rx (g - mean g) - k x^,   x^ = rx x,   w = t dh',  u = ru b
//   sum w u = ru (sum t b dh_out + rx (sum t b g - mean g sum t b) - k rx sum t b x)
//   db = ru (w - mean w - u mean(w u))
// so the second norm's sums need no second pass over the first one's result
// (mean g and mean w belong to layer norms).  k is taken as rx (rx mean(g x)), no
// power of rx by itself: a row's rx may be 1e15 or 1e-15, and its cube is no FP32
// number then, while k has the size of the gradient itself.  A layer norm's row is centred
// first, so that its squares are those of centred values (a mean far above the
// deviation would cancel in FP32): its mean takes a pass.  After a layer norm on
// the block's output the second norm's sums are taken from dh' itself, in a pass
// of their own: that is eight sums less to hold than the closed form.
template <bool FP32, int SPLIT, bool PRE_L, bool POST_L>
__global__ void __launch_bounds__(Back<FP32, SPLIT>::kThreads, Back<FP32, SPLIT>::kCtas) k_block_norm_backward(const BackArgs a) {
  constexpr int W = FP32 ? 2 : 1;              // 16-byte pieces of eight stream values
  constexpr int PIECES = 2 * W + 2;            // h, dh_out, dn, b
  extern __shared__ uint4 shared[];            // [4][T] scale and gate, then [stages][PIECES][T]
  constexpr int PASSES = 1 + (PRE_L ? 1 : 0) + (POST_L ? 1 : 0);
  __shared__ Slots<SPLIT> slots[2][PASSES];
  const int T = (int)blockDim.x, warps = T >> 5, t = (int)threadIdx.x;
  uint32_t rank = 0;
  if constexpr (SPLIT > 1) asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  const int64_t chunk = blockIdx.x / SPLIT;
  int64_t s = chunk / a.seg_chunks;
  if (s >= a.segments) s = a.segments - 1;
  const int64_t first = s * a.seg + (chunk - s * a.seg_chunks) * a.chunk_rows;
  int64_t last = first + a.chunk_rows;
  if (last > (s + 1) * a.seg) last = (s + 1) * a.seg;
  if (last > a.M) last = a.M;
  const float inv_d = 1.0f / (float)a.D;
  const int col = ((int)rank * T + t) * 8;
  const bool live = col < a.D;

  uint4* ring = shared + 4 * T;
  auto piece = [&](int stage, int k) { return &ring[(stage * PIECES + k) * T + t]; };
  // The stream's pieces: bf16, each thread its own 16 bytes.  FP32, a warp's 1024
  // bytes in two runs of 512: lane l copies pieces (l mod 2) of the threads l / 2
  // and 16 + l / 2 of its warp, and the warp meets before and after reading.
  auto fetch_stream = [&](const void* base, int64_t at, int stage, int k) {
    if constexpr (FP32) {
      const int lane = t & 31;
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        const int to = (t & ~31) + 16 * w + (lane >> 1);  // thread
        const int c = ((int)rank * T + to) * 8 + 4 * (lane & 1);
        if (c < a.D)
          cp_async16(smem_addr(&ring[(stage * PIECES + k + (lane & 1)) * T + to]),
                     reinterpret_cast<const float*>(base) + (at - col) + c);
      }
    } else {
      if (live) cp_async16(smem_addr(piece(stage, k)), reinterpret_cast<const uint16_t*>(base) + at);
    }
  };
  auto fetch = [&](int64_t row, int stage) {
    if (row < last) {
      const int64_t at = row * a.D + col;
      if (a.dn) {
        fetch_stream(a.h, at, stage, 0);
        if (live) cp_async16(smem_addr(piece(stage, 2 * W)), reinterpret_cast<const uint16_t*>(a.dn) + at);
      }
      if (a.dh_out) fetch_stream(a.dh_out, at, stage, W);
      if (a.b && live) cp_async16(smem_addr(piece(stage, 2 * W + 1)), reinterpret_cast<const uint16_t*>(a.b) + at);
    }
    cp_async_commit();  // a group per row, empty past the last one
  };

  F2 acc[3][4];
#pragma unroll
  for (int k = 0; k < 3; ++k) {
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[k][i] = f2(0.f, 0.f);
  }
  // Pieces of absent inputs and of columns past D read as zero.
  for (int st = 0; st < a.stages; ++st) {
#pragma unroll
    for (int k = 0; k < PIECES; ++k) *piece(st, k) = make_uint4(0, 0, 0, 0);
  }
  __syncwarp();
  for (int st = 0; st < a.stages; ++st) fetch(first + st, st);
  // Scale in pieces 0 and 1 of this thread, gate in 2 and 3.
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float* m = k < 2 ? a.scale : a.gate;
    float4 v = k < 2 ? make_float4(0.f, 0.f, 0.f, 0.f) : make_float4(1.f, 1.f, 1.f, 1.f);
    if (m && live) v = __ldg(reinterpret_cast<const float4*>(m + s * a.D + col + 4 * (k & 1)));
    reinterpret_cast<float4*>(shared)[k * T + t] = v;
  }
  auto scale_at = [&](F2 (&v)[4]) {
    const ulonglong2 x = reinterpret_cast<const ulonglong2*>(shared)[t];
    const ulonglong2 y = reinterpret_cast<const ulonglong2*>(shared)[T + t];
    v[0].v = x.x, v[1].v = x.y, v[2].v = y.x, v[3].v = y.y;
  };
  auto gate_at = [&](F2 (&v)[4]) {
    const ulonglong2 x = reinterpret_cast<const ulonglong2*>(shared)[2 * T + t];
    const ulonglong2 y = reinterpret_cast<const ulonglong2*>(shared)[3 * T + t];
    v[0].v = x.x, v[1].v = x.y, v[2].v = y.x, v[3].v = y.y;
  };
  for (int i = t; i < (int)(sizeof(slots) / 4); i += T) reinterpret_cast<float*>(slots)[i] = 0.f;
  __shared__ int abort_word;
  if (t == 0) abort_word = 0;
  volatile int* abort_flag = &abort_word;
  __syncthreads();
  if constexpr (SPLIT > 1) {
    if (t == 0) {
      for (int k = 0; k < 2 * PASSES; ++k) mbar_init(smem_u32(&slots[0][0].bar) + k * (uint32_t)sizeof(Slots<SPLIT>), 1);
      fence_mbarrier_init();
    }
    cluster_barrier();  // every CTA's slots and barriers are ready
  }

  int buf = 0, stage = 0;
  for (int64_t row = first; row < last; ++row, buf ^= 1) {
    cp_async_wait(a.stages - 1);
    if constexpr (FP32) __syncwarp();
    Raw8<FP32> rx8, rd8;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      rx8.q[w] = *piece(stage, w);
      rd8.q[w] = *piece(stage, W + w);
    }
    const uint4 rn8 = *piece(stage, 2 * W), rb8 = *piece(stage, 2 * W + 1);
    if constexpr (FP32) __syncwarp();
    fetch(row + a.stages, stage);
    if (++stage == a.stages) stage = 0;

    Slots<SPLIT>* slot = slots[buf];
    const uint32_t parity = (uint32_t)((row - first) >> 1) & 1u;
    bool ok = true;
    const F2 zero = f2(0.f, 0.f);
    float mx = 0.f, mu = 0.f, rx = 0.f, ru = 1.f, k = 0.f, mg = 0.f, mw = 0.f, mwu = 0.f;

    if constexpr (POST_L) {
      // The mean of b with, layer pre-norm: the means of x and g; else the sums of x.
      F2 p[3] = {zero, zero, zero};
      if (live) {
        F2 x[4], g[4], u[4], sc[4];
        rx8.get(x);
        unpack8(rn8, g);
        unpack8(rb8, u);
        scale_at(sc);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const F2 w = fma(g[i], sc[i], g[i]);
          p[0] = p[0] + u[i];
          p[1] = PRE_L ? p[1] + x[i] : fma(x[i], x[i], p[1]);
          p[2] = PRE_L ? p[2] + w : fma(w, x[i], p[2]);
        }
      }
      float q[3];
      fold(p, q);
      ok = row_group_sums<SPLIT>(q, warps, rank, slot[0], parity, a.wait_limit_ns, abort_flag) && ok;
      mu = q[0] * inv_d;
      if constexpr (PRE_L) {
        mx = q[1] * inv_d;
        mg = q[2] * inv_d;
        const F2 nmx = f2(-mx, -mx);
        F2 s[2] = {zero, zero};
        if (live) {
          F2 x[4], g[4], sc[4];
          rx8.get(x);
          unpack8(rn8, g);
          scale_at(sc);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            x[i] = x[i] + nmx;
            s[0] = fma(x[i], x[i], s[0]);
            s[1] = fma(fma(g[i], sc[i], g[i]), x[i], s[1]);
          }
        }
        float r[2];
        fold(s, r);
        ok = row_group_sums<SPLIT>(r, warps, rank, slot[PASSES - 1], parity, a.wait_limit_ns, abort_flag) && ok;
        q[1] = r[0];
        q[2] = r[1];
      }
      if (a.dn) {
        rx = rsqrtf(q[1] * inv_d + a.eps);
        k = rx * (rx * (q[2] * inv_d));
      }
    } else {
      if constexpr (PRE_L) {
        F2 p[2] = {zero, zero};
        if (live) {
          F2 x[4], g[4], sc[4];
          rx8.get(x);
          unpack8(rn8, g);
          scale_at(sc);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            p[0] = p[0] + x[i];
            p[1] = p[1] + fma(g[i], sc[i], g[i]);
          }
        }
        float q[2];
        fold(p, q);
        ok = row_group_sums<SPLIT>(q, warps, rank, slot[0], parity, a.wait_limit_ns, abort_flag) && ok;
        mx = q[0] * inv_d;
        mg = q[1] * inv_d;
      }
      const F2 nmx = f2(-mx, -mx);
      F2 p[PRE_L ? 7 : 6];
#pragma unroll
      for (int i = 0; i < (PRE_L ? 7 : 6); ++i) p[i] = zero;
      if (live) {
        F2 x[4], d[4], g[4], u[4], sc[4], gt[4];
        rx8.get(x);
        rd8.get(d);
        unpack8(rn8, g);
        unpack8(rb8, u);
        scale_at(sc);
        gate_at(gt);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if constexpr (PRE_L) x[i] = x[i] + nmx;
          acc[2][i] = acc[2][i] + g[i];
          const F2 w = fma(g[i], sc[i], g[i]);
          const F2 tb = gt[i] * u[i];
          p[0] = fma(x[i], x[i], p[0]);
          p[1] = fma(u[i], u[i], p[1]);
          p[2] = fma(w, x[i], p[2]);
          p[3] = fma(tb, d[i], p[3]);
          p[4] = fma(tb, w, p[4]);
          p[5] = fma(tb, x[i], p[5]);
          if constexpr (PRE_L) p[6] = p[6] + tb;
        }
      }
      float q[PRE_L ? 7 : 6];
      fold(p, q);
      ok = row_group_sums<SPLIT>(q, warps, rank, slot[PASSES - 1], parity, a.wait_limit_ns, abort_flag) && ok;
      if (a.dn) {
        rx = rsqrtf(q[0] * inv_d + a.eps);
        k = rx * (rx * (q[2] * inv_d));
      }
      if (a.post != kNone) {
        ru = rsqrtf(q[1] * inv_d + a.eps);
        float swu = q[3] + rx * q[4] - k * (rx * q[5]);
        if constexpr (PRE_L) swu -= rx * mg * q[6];
        mwu = ru * swu * inv_d;
      }
    }

    const F2 rx2 = f2(rx, rx), nk2 = f2(-k, -k), nmx2 = f2(-mx, -mx), nmg2 = f2(-rx * mg, -rx * mg);
    const F2 alpha2 = f2(a.alpha, a.alpha), nmu2 = f2(-mu, -mu);
    F2 d[4];
    // dh', from the row's data and statistics.
    auto stream_gradient = [&](F2 (&x)[4], F2 (&g)[4], const F2 (&sc)[4]) {
      rd8.get(d);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (PRE_L) x[i] = x[i] + nmx2;
        x[i] = x[i] * rx2;
        acc[1][i] = fma(g[i], x[i], acc[1][i]);
        d[i] = fma(rx2, fma(g[i], sc[i], g[i]), d[i]);
        if constexpr (PRE_L) d[i] = d[i] + nmg2;
        d[i] = fma(nk2, x[i], d[i]);
      }
    };
    if constexpr (POST_L) {
      F2 p[3] = {zero, zero, zero};
      if (live) {
        F2 x[4], g[4], u[4], sc[4], gt[4];
        rx8.get(x);
        unpack8(rn8, g);
        scale_at(sc);
        stream_gradient(x, g, sc);
        unpack8(rb8, u);
        gate_at(gt);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          acc[2][i] = acc[2][i] + g[i];
          u[i] = u[i] + nmu2;
          const F2 w = gt[i] * d[i];
          p[0] = fma(u[i], u[i], p[0]);
          p[1] = fma(w, u[i], p[1]);
          p[2] = p[2] + w;
        }
      }
      float q[3];
      fold(p, q);
      ok = row_group_sums<SPLIT>(q, warps, rank, slot[1], parity, a.wait_limit_ns, abort_flag) && ok;
      ru = rsqrtf(q[0] * inv_d + a.eps);
      mwu = ru * q[1] * inv_d;
      mw = q[2] * inv_d;
    }
    // A wait that ran out is recorded; the warp sends no more, so its peers' waits run out too.
    if (SPLIT > 1 && !__all_sync(0xffffffffu, ok)) break;
    const F2 ru2 = f2(ru, ru), nmw2 = f2(-ru * mw, -ru * mw), nmwu2 = f2(-ru * mwu, -ru * mwu);
    if (live) {
      F2 x[4], g[4], u[4], sc[4], gt[4];
      if constexpr (!POST_L) {
        rx8.get(x);
        unpack8(rn8, g);
        scale_at(sc);
        stream_gradient(x, g, sc);
      }
      unpack8(rb8, u);
      gate_at(gt);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (POST_L) u[i] = u[i] + nmu2;
        u[i] = u[i] * ru2;
        acc[0][i] = fma(d[i], u[i], acc[0][i]);
        const F2 w = (ru2 * gt[i]) * d[i];
        u[i] = fma(nmwu2, u[i], w);
        if constexpr (POST_L) u[i] = u[i] + nmw2;
      }
      if (!POST_L && a.post == kNone) {
        // Without a norm b takes no part in db, also where 0 b is not 0 (a select in
        // the line above instead: 582 -> 600 us at 33001 x 7168).
        gate_at(gt);
#pragma unroll
        for (int i = 0; i < 4; ++i) u[i] = gt[i] * d[i];
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) d[i] = d[i] * alpha2;
      const int64_t at = row * a.D + col;
      if (a.dh) store_stream8<FP32>(a.dh, at, a.wide, d);
      if (a.db) st_stream(reinterpret_cast<uint16_t*>(a.db) + at, pack8(u));
    }
  }
  cp_async_wait(0);
  if constexpr (SPLIT > 1) {
    // No CTA leaves while a peer may still send it sums.  A CTA whose waits all
    // came to an end has everything that was sent to it.  One that gave up does not
    // know, and the barrier, after which nobody sends, does not wait for what is on
    // its way: one thread keeps the CTA's shared memory for the microseconds that
    // takes, and more.
    cluster_barrier();
    if (t == 0 && *abort_flag) {
      const uint64_t t0 = globaltimer_ns();
      while (globaltimer_ns() - t0 < 200000ull) {
      }
    }
  }
  if (!live) return;
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    if (!a.sums[k]) continue;
    float4* o = reinterpret_cast<float4*>(a.sums[k] + chunk * a.sum_stride + col);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float2 x = split(acc[k][2 * i]), y = split(acc[k][2 * i + 1]);
      o[i] = make_float4(x.x, x.y, y.x, y.y);
    }
  }
}

struct SumArgs {
  const float* sums;  // [chunks][3][D]
  float* out[3];
  int64_t seg_chunks, segments, chunks;
  int D;
};

// out_k[s] = the sum of a segment's partials: eight warps take every eighth
// chunk of 128 columns, then add up in the order of the warps.
__global__ void __launch_bounds__(256) k_segment_sums(const SumArgs a) {
  __shared__ float4 part[8][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int col = ((int)blockIdx.x * 32 + lane) * 4;
  float* out = a.out[blockIdx.z];
  if (!out) return;
  for (int64_t s = blockIdx.y; s < a.segments; s += gridDim.y) {
    const int64_t c0 = s * a.seg_chunks;
    const int64_t c1 = s + 1 < a.segments ? c0 + a.seg_chunks : a.chunks;
    float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
    if (col < a.D) {
      const float* src = a.sums + blockIdx.z * a.D + col;
#pragma unroll 8
      for (int64_t i = c0 + warp; i < c1; i += 8) {
        const float4 v = __ldg(reinterpret_cast<const float4*>(src + i * 3 * a.D));
        t.x += v.x;
        t.y += v.y;
        t.z += v.z;
        t.w += v.w;
      }
    }
    part[warp][lane] = t;
    __syncthreads();
    if (warp == 0 && col < a.D) {
#pragma unroll
      for (int w = 1; w < 8; ++w) {
        const float4 v = part[w][lane];
        t.x += v.x;
        t.y += v.y;
        t.z += v.z;
        t.w += v.w;
      }
      *reinterpret_cast<float4*>(out + s * a.D + col) = t;
    }
    __syncthreads();
  }
}

bool aligned32(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 31u) == 0; }

template <bool FP32, int CH>
cudaError_t norm_launch(const NormArgs& a, int warps, cudaStream_t s) {
  k_block_norm<FP32, CH, false><<<(unsigned)a.rows, 32 * warps, 0, s>>>(a);
  return cudaGetLastError();
}
// Rows of one warp, four to a CTA.
template <bool FP32, int CH>
cudaError_t narrow_launch(const NormArgs& a, cudaStream_t s) {
  k_block_norm<FP32, CH, true><<<(unsigned)((a.rows + 3) / 4), 128, 0, s>>>(a);
  return cudaGetLastError();
}

template <bool FP32>
cudaError_t norm_dispatch(const NormArgs& a, cudaStream_t s) {
  // Chunks of eight values per thread: four where the row is wide (66601 x 7168 at
  // two: 850 us against 641), two up to 2048 (66601 x 1024 at four: 97 us against
  // 95).  By the width alone, so that a row's bits do not depend on how many rows
  // come with it; one chunk per thread would save a single row of 7168 1.2 of 6.0 us.
  if (a.D <= 256) return narrow_launch<FP32, 1>(a, s);
  if (a.D <= 512) return narrow_launch<FP32, 2>(a, s);
  if (a.D <= 2048) return norm_launch<FP32, 2>(a, (a.D + 511) / 512, s);
  return norm_launch<FP32, 4>(a, (a.D + 1023) / 1024, s);
}

// CTAs that share a row in the backward pass, and their threads.
template <bool FP32>
int back_split(int D) {
  if (D / 8 <= Back<FP32, 1>::kThreads) return 1;
  int split = 2;
  while ((D / 8 + split - 1) / split > kBackThreads) split *= 2;
  return split;
}
template <bool FP32>
int back_threads(int D) {
  const int split = back_split<FP32>(D);
  return 32 * ((D / 8 + 32 * split - 1) / (32 * split));
}

// How the backward pass splits its rows: `per` chunks of `rows` rows in a full
// segment, `total` in all.  A chunk stays within a segment.
struct Chunks {
  int64_t segments, rows, per, total;
};
template <bool FP32>
Chunks back_chunks(int64_t M, int D, int64_t seg) {
  if (seg > M) seg = M;
  Chunks c;
  c.segments = (M + seg - 1) / seg;
  const int64_t rest = M - (c.segments - 1) * seg;
  // The clusters that the threads of 148 SMs hold (at most eight CTAs each).  A
  // chunk's partial sums cost as much traffic as about one of its rows, and its
  // rows follow one another: not less than four of them.  This counts threads
  // alone: it is one wave where a CTA has near 448 of them, and up to two where
  // the shared memory of their rings holds fewer CTAs than that (of the planned
  // 7, 3 and 3 per SM 5, 2 and 2 fit at bf16 widths of 1024, 4096 and 16384:
  // 33001 x 4096 takes 457 us, 33001 x 7168 584).
  const int split = back_split<FP32>(D), threads = back_threads<FP32>(D);
  const int64_t resident = (split == 1 ? Back<FP32, 1>::kCtas * Back<FP32, 1>::kThreads : 2 * kBackThreads) / threads;
  const int64_t target = 148 * (resident > 8 ? 8 : resident) / split;
  c.rows = (M + target - 1) / target;
  if (c.rows < 4) c.rows = 4;
  if (c.rows > seg) c.rows = seg;
  for (;;) {
    c.per = (seg + c.rows - 1) / c.rows;
    c.total = (c.segments - 1) * c.per + (rest + c.rows - 1) / c.rows;
    // Segments' ragged ends may open a second wave: take longer chunks.
    if (c.total <= target || c.rows >= seg || c.segments >= target) break;
    c.rows += (c.rows + 31) / 32;
    if (c.rows > seg) c.rows = seg;
  }
  return c;
}

}  // namespace

cudaError_t launch_block_norm(const BlockNormLaunch& p, cudaStream_t s) {
  NormArgs a;
  a.h = p.h;
  a.b = p.b;
  a.gate = p.gate;
  a.scale = p.scale;
  a.shift = p.shift;
  a.h_out = p.h_out;
  a.n = p.n;
  a.codes = reinterpret_cast<uint8_t*>(p.codes);
  a.scales = reinterpret_cast<uint8_t*>(p.scales);
  a.M = p.M;
  a.rows = p.codes_format != 0 ? (p.M + 127) / 128 * 128 : p.M;
  a.seg = p.segment_tokens;
  a.D = p.D;
  a.post = p.post;
  a.pre = p.pre;
  a.format = p.codes_format;
  a.wide_stream = aligned32(p.h) && aligned32(p.h_out);
  a.wide_mods = aligned32(p.gate) && aligned32(p.scale) && aligned32(p.shift);
  a.alpha = p.alpha;
  a.eps = p.eps;
  return p.fp32 ? norm_dispatch<true>(a, s) : norm_dispatch<false>(a, s);
}

size_t block_norm_backward_workspace(int64_t M, int D, int64_t segment_tokens) {
  // The larger of the two stream types'.  One chunk per segment: nothing to add up.
  size_t most = 0;
  for (const Chunks& c : {back_chunks<false>(M, D, segment_tokens), back_chunks<true>(M, D, segment_tokens)}) {
    const size_t bytes = c.per == 1 ? 0 : (size_t)c.total * 3 * D * sizeof(float);
    if (bytes > most) most = bytes;
  }
  return most;
}

namespace {

template <bool FP32, int SPLIT, bool PRE_L, bool POST_L>
cudaError_t back_launch(BackArgs& a, int64_t chunks, int T, cudaStream_t s) {
  const size_t mods = (size_t)64 * T, stage = (size_t)(FP32 ? 6 : 4) * 16 * T;
  int stages = (int)((Back<FP32, SPLIT>::kSmem - mods) / stage);
  if (stages > kBackStagesMax) stages = kBackStagesMax;
  if (stages > a.chunk_rows) stages = (int)a.chunk_rows;
  a.stages = stages;
  const cudaError_t e = allow_shared_memory((const void*)k_block_norm_backward<FP32, SPLIT, PRE_L, POST_L>, Back<FP32, SPLIT>::kSmem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(chunks * SPLIT), 1, 1);
  cfg.blockDim = dim3((unsigned)T, 1, 1);
  cfg.dynamicSmemBytes = mods + stage * stages;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = SPLIT;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = SPLIT > 1 ? 1 : 0;
  if (SPLIT > 1) g_launched.store(true);
  return cudaLaunchKernelEx(&cfg, k_block_norm_backward<FP32, SPLIT, PRE_L, POST_L>, (const BackArgs)a);
}

template <bool FP32, int SPLIT>
cudaError_t back_kind(BackArgs& a, int64_t chunks, int T, cudaStream_t s) {
  const bool pre = a.pre == kLayer, post = a.post == kLayer;
  if (post) {
    return pre ? back_launch<FP32, SPLIT, true, true>(a, chunks, T, s) : back_launch<FP32, SPLIT, false, true>(a, chunks, T, s);
  }
  return pre ? back_launch<FP32, SPLIT, true, false>(a, chunks, T, s) : back_launch<FP32, SPLIT, false, false>(a, chunks, T, s);
}

template <bool FP32>
cudaError_t back_dispatch(BackArgs& a, int64_t chunks, cudaStream_t s) {
  const int T = back_threads<FP32>(a.D);
  switch (back_split<FP32>(a.D)) {
    case 1: return back_kind<FP32, 1>(a, chunks, T, s);
    case 2: return back_kind<FP32, 2>(a, chunks, T, s);
    case 4: return back_kind<FP32, 4>(a, chunks, T, s);
    default: return back_kind<FP32, 8>(a, chunks, T, s);
  }
}

}  // namespace

cudaError_t launch_block_norm_backward(const BlockNormBackwardLaunch& p, int* kernels, cudaStream_t s) {
  const Chunks c = p.fp32 ? back_chunks<true>(p.M, p.D, p.segment_tokens) : back_chunks<false>(p.M, p.D, p.segment_tokens);
  BackArgs a;
  a.dn = p.dn;
  a.dh_out = p.dh_out;
  a.h = p.h_out;
  a.b = p.b;
  a.gate = p.gate;
  a.scale = p.scale;
  a.dh = p.dh;
  a.db = p.db;
  a.M = p.M;
  a.seg = p.segment_tokens < p.M ? p.segment_tokens : p.M;
  a.seg_chunks = c.per;
  a.segments = c.segments;
  a.chunk_rows = c.rows;
  a.D = p.D;
  a.post = p.post;
  a.pre = p.pre;
  a.alpha = p.alpha;
  a.eps = p.eps;
  a.wide = aligned32(p.dh);
  a.wait_limit_ns = p.wait_limit_ns;
  float* const out[3] = {p.dgate, p.dscale, p.dshift};
  const bool direct = c.per == 1;
  for (int k = 0; k < 3; ++k) a.sums[k] = !out[k] ? nullptr : (direct ? out[k] : p.workspace + (int64_t)k * p.D);
  a.sum_stride = direct ? p.D : 3 * (int64_t)p.D;
  *kernels = 1;
  cudaError_t e = p.fp32 ? back_dispatch<true>(a, c.total, s) : back_dispatch<false>(a, c.total, s);
  if (e != cudaSuccess || direct || (!out[0] && !out[1] && !out[2])) return e;
  SumArgs m;
  m.sums = p.workspace;
  for (int k = 0; k < 3; ++k) m.out[k] = out[k];
  m.seg_chunks = c.per;
  m.segments = c.segments;
  m.chunks = c.total;
  m.D = p.D;
  const dim3 grid((unsigned)((p.D + 127) / 128), (unsigned)(c.segments < 65535 ? c.segments : 65535), 3);
  k_segment_sums<<<grid, 256, 0, s>>>(m);
  *kernels = 2;
  return cudaGetLastError();
}

cudaError_t take_norm_error(int* value) {
  *value = 0;
  return g_launched.load() ? take_device_error(value) : cudaSuccess;
}

}  // namespace lg
