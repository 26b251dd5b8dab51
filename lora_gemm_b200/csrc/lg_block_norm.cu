// The norms between two transformer blocks, with the gate, the scaled residual
// and the modulation, forward and backward:
//
//   h' = alpha h + gate * N_post(b),   n = N_pre(h') (1 + scale) + shift
//
// (RMS or layer norms over the D values of a row; gate, scale and shift per
// segment of rows).  Both directions touch every row once and are bound by
// HBM; the statistics are FP32 sums over the row held in registers.
//
// Forward: one row per group of warps, each thread holding CH chunks of eight
// consecutive values.  The row's data are read and written past L1, which is
// left to the modulation vectors: 3 x 4 D bytes that every row of a segment
// reads again (more than the row itself), and that the rows resident on an SM
// share there.
//
// Backward: with u = N_post(b), x^ = N_pre(h'), r the reciprocal deviation of
// a norm and g its output's gradient, the input's gradient is
//
//   RMS:    r (g - x^ mean(g x^))
//   layer:  r (g - mean g - x^ mean(g x^))
//
// A CTA takes consecutive rows of one segment, each thread always the same
// columns, so the column sums dgate, dscale and dshift stay in registers over
// the CTA's rows; one partial row per CTA goes to the workspace and a second
// kernel adds the partials of a segment in a fixed order.
#include "lg_internal.h"
#include "lg_mx.cuh"

namespace lg {

namespace {

constexpr int kNone = 0, kLayer = 2;  // LG_NORM_NONE, LG_NORM_LAYER (LG_NORM_RMS needs no test)
constexpr int kCodesMxfp4 = 2;  // LG_CODES_MXFP4; any other nonzero format is MXFP8
constexpr int kMaxWarps = 32;

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

// Raw bits of eight stream values: 16 bytes (bf16) or 32 (FP32).
template <bool FP32>
struct Raw8 {
  uint4 q[FP32 ? 2 : 1];
  __device__ __forceinline__ void load(const void* base, int64_t at) {
    if constexpr (FP32) {
      q[0] = ld_stream(reinterpret_cast<const float*>(base) + at);
      q[1] = ld_stream(reinterpret_cast<const float*>(base) + at + 4);
    } else {
      q[0] = ld_stream(reinterpret_cast<const uint16_t*>(base) + at);
    }
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
};
// Stores eight values in the stream's type; v becomes what was stored.
template <bool FP32>
__device__ __forceinline__ void store_stream8(void* base, int64_t at, float (&v)[8]) {
  if constexpr (FP32) {
    float* p = reinterpret_cast<float*>(base) + at;
    st_stream(p, make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])));
    st_stream(p + 4,
              make_uint4(__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]), __float_as_uint(v[7])));
  } else {
    const uint4 q = pack8(v);
    st_stream(reinterpret_cast<uint16_t*>(base) + at, q);
    unpack8(q, v);
  }
}
// Eight values of a segment's modulation row (cached), or `other` without one.
__device__ __forceinline__ void load_mod8(const float* base, int64_t at, float other, float (&v)[8]) {
  if (base) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(base + at));
    const float4 b = __ldg(reinterpret_cast<const float4*>(base + at + 4));
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
    v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = other;
  }
}

// Sums of N values over the `warps` warps of a row (one warp: shuffles alone).
// Each call of a row has shared memory of its own (`slot`): no barrier is
// needed before the next call.
template <int N>
__device__ __forceinline__ void row_sums(float (&v)[N], int warps, float (*slot)[kMaxWarps]) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
  }
  if (warps == 1) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (lane == 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) slot[i][warp] = v[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) {
    v[i] = lane < warps ? slot[i][lane] : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
  }
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
  float alpha, eps;
};

// Normalises the row's values in place; `live` masks chunks past D.
template <int CH>
__device__ __forceinline__ void normalise(float (&v)[CH][8], const bool (&live)[CH], int kind, float eps, int D,
                                          int warps, float (*slot)[kMaxWarps]) {
  if (kind == kLayer) {
    float s[1] = {0.f};
#pragma unroll
    for (int c = 0; c < CH; ++c) {
#pragma unroll
      for (int i = 0; i < 8; ++i) s[0] += v[c][i];  // chunks past D hold zeros
    }
    row_sums<1>(s, warps, slot);
    const float mean = s[0] / (float)D;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[c][i] = live[c] ? v[c][i] - mean : 0.f;
    }
  }
  float q[1] = {0.f};
#pragma unroll
  for (int c = 0; c < CH; ++c) {
#pragma unroll
    for (int i = 0; i < 8; ++i) q[0] = fmaf(v[c][i], v[c][i], q[0]);
  }
  row_sums<1>(q, warps, slot + 1);
  const float r = 1.0f / sqrtf(q[0] / (float)D + eps);
#pragma unroll
  for (int c = 0; c < CH; ++c) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[c][i] *= r;
  }
}

// blockDim.x = 32 * warps for one row, or (ONE) several rows of one warp each.
template <bool FP32, int CH, bool ONE>
__global__ void __launch_bounds__(ONE ? 128 : 1024) k_block_norm(const NormArgs a) {
  __shared__ float slots[4][kMaxWarps];
  const int warps = ONE ? 1 : (int)blockDim.x >> 5;
  const int t = ONE ? (int)threadIdx.x & 31 : (int)threadIdx.x;
  const int T = 32 * warps;
  const int64_t row = ONE ? (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5) : (int64_t)blockIdx.x;
  if (row >= a.rows) return;
  if (row >= a.M) {  // the scale bytes of rows past M
    for (int kb = t; kb < a.D / 32; kb += T) a.scales[mx_scale_offset(row, kb, a.D / 128)] = 0;
    return;
  }
  const int64_t at = row * a.D;
  const int64_t mod = row / a.seg * a.D;
  bool live[CH];
  Raw8<FP32> raw[CH];
  float v[CH][8];
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int col = (c * T + t) * 8;
    live[c] = col < a.D;
    raw[c].zero();
    if (live[c]) raw[c].load(a.h, at + col);
  }
  if (a.b) {
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      uint4 q = make_uint4(0, 0, 0, 0);
      if (live[c]) q = ld_stream(reinterpret_cast<const uint16_t*>(a.b) + at + (c * T + t) * 8);
      unpack8(q, v[c]);
    }
    if (a.post != kNone) normalise<CH>(v, live, a.post, a.eps, a.D, warps, slots);
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      if (!live[c]) continue;
      const int col = (c * T + t) * 8;
      float g[8], h[8];
      load_mod8(a.gate, mod + col, 1.0f, g);
      raw[c].get(h);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[c][i] = fmaf(g[i], v[c][i], a.alpha * h[i]);
      store_stream8<FP32>(a.h_out, at + col, v[c]);
    }
  } else {
#pragma unroll
    for (int c = 0; c < CH; ++c) raw[c].get(v[c]);
  }
  if (a.pre == kNone) return;
  normalise<CH>(v, live, a.pre, a.eps, a.D, warps, slots + 2);
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int col = (c * T + t) * 8;
    uint4 q = make_uint4(0, 0, 0, 0);
    if (live[c]) {
      float s[8], f[8];
      load_mod8(a.scale, mod + col, 0.0f, s);
      load_mod8(a.shift, mod + col, 0.0f, f);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[c][i] = fmaf(v[c][i], 1.0f + s[i], f[i]);
      q = pack8(v[c]);
      if (a.n) st_stream(reinterpret_cast<uint16_t*>(a.n) + at + col, q);
    }
    if (a.format != 0) {
      // D is a multiple of 128 here, so four lanes hold one block, all live or all not.
      const uint32_t w[4] = {q.x, q.y, q.z, q.w};
      uint32_t sb;
      if (a.format == kCodesMxfp4) {
        sb = mxfp4_scale_byte(mx_block_max(mx_abs_max8(w)));
        if (live[c]) *reinterpret_cast<uint32_t*>(a.codes + (at + col) / 2) = mxfp4_codes8(w, sb);
      } else {
        float m = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          m = fmaxf(m, fmaxf(fabsf(__uint_as_float(w[i] << 16)), fabsf(__uint_as_float(w[i] & 0xFFFF0000u))));
        }
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
        sb = mxfp8_scale_byte(m);
        if (live[c]) *reinterpret_cast<uint2*>(a.codes + at + col) = mxfp8_codes8(w, sb);
      }
      // The four bytes of a K group from its 16 lanes, one store.
      sb |= __shfl_down_sync(0xffffffffu, sb, 4) << 8;
      sb |= __shfl_down_sync(0xffffffffu, sb, 8) << 16;
      if (live[c] && (t & 15) == 0) {
        *reinterpret_cast<uint32_t*>(a.scales + mx_scale_offset(row, col / 32, a.D / 128)) = sb;
      }
    }
  }
}

struct BackArgs {
  const void* dn;
  const void* dh_out;
  const void* h;
  const void* b;
  const float* gate;
  const float* scale;
  void* dh;
  void* db;
  float* sums;        // [chunks][3][D] partials (dgate, dscale, dshift)
  int64_t M;
  int64_t seg;
  int64_t seg_chunks;   // chunks per segment
  int64_t chunk_rows;
  int D, post, pre;
  float alpha, eps;
};

template <bool FP32, int CH>
__global__ void __launch_bounds__(1024) k_block_norm_backward(const BackArgs a) {
  __shared__ float slots[2][8][kMaxWarps];  // alternating rows: a row's last reads and the next row's writes
  const int warps = (int)blockDim.x >> 5;
  const int T = (int)blockDim.x;
  const int64_t s = blockIdx.x / a.seg_chunks;
  const int64_t first = s * a.seg + (blockIdx.x - s * a.seg_chunks) * a.chunk_rows;
  int64_t last = first + a.chunk_rows;
  if (last > (s + 1) * a.seg) last = (s + 1) * a.seg;
  if (last > a.M) last = a.M;
  const float inv_d = 1.0f / (float)a.D;
  float acc[3][CH][8];
#pragma unroll
  for (int k = 0; k < 3; ++k) {
#pragma unroll
    for (int c = 0; c < CH; ++c) {
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[k][c][i] = 0.f;
    }
  }
  int buf = 0;
  for (int64_t row = first; row < last; ++row, buf ^= 1) {
    const int64_t at = row * a.D;
    float (*slot)[kMaxWarps] = slots[buf];
    float x[CH][8], g[CH][8], u[CH][8], d[CH][8];
    bool live[CH];
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int col = (c * T + (int)threadIdx.x) * 8;
      live[c] = col < a.D;
      Raw8<FP32> rx, rd;
      uint4 rn = make_uint4(0, 0, 0, 0), rb = make_uint4(0, 0, 0, 0);
      rx.zero();
      rd.zero();
      if (live[c]) {
        if (a.dn) {
          rx.load(a.h, at + col);
          rn = ld_stream(reinterpret_cast<const uint16_t*>(a.dn) + at + col);
        }
        if (a.dh_out) rd.load(a.dh_out, at + col);
        if (a.b) rb = ld_stream(reinterpret_cast<const uint16_t*>(a.b) + at + col);
      }
      rx.get(x[c]);
      rd.get(d[c]);
      unpack8(rn, g[c]);
      unpack8(rb, u[c]);
    }
    // Layer norms: the means first, so that the squares are those of centred
    // values (a mean far above the deviation would cancel in FP32).
    if (a.pre == kLayer || a.post == kLayer) {
      float m[2] = {0.f, 0.f};
#pragma unroll
      for (int c = 0; c < CH; ++c) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          m[0] += x[c][i];
          m[1] += u[c][i];
        }
      }
      row_sums<2>(m, warps, slot);
      const float mx = a.pre == kLayer ? m[0] * inv_d : 0.f;
      const float mu = a.post == kLayer ? m[1] * inv_d : 0.f;
#pragma unroll
      for (int c = 0; c < CH; ++c) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          x[c][i] = live[c] ? x[c][i] - mx : 0.f;
          u[c][i] = live[c] ? u[c][i] - mu : 0.f;
        }
      }
    }
    // Squares of both rows, and the sums of g and g x with g = dn (1 + scale).
    float q[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      if (!live[c]) continue;
      const int col = (c * T + (int)threadIdx.x) * 8;
      float sc[8];
      load_mod8(a.scale, s * a.D + col, 0.f, sc);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        acc[2][c][i] += g[c][i];
        const float w = g[c][i] * (1.0f + sc[i]);
        q[0] = fmaf(x[c][i], x[c][i], q[0]);
        q[1] = fmaf(u[c][i], u[c][i], q[1]);
        q[2] = fmaf(w, x[c][i], q[2]);
        q[3] += w;
      }
    }
    row_sums<4>(q, warps, slot + 2);
    const float rx = 1.0f / sqrtf(q[0] * inv_d + a.eps);
    const float ru = a.post == kNone ? 1.0f : 1.0f / sqrtf(q[1] * inv_d + a.eps);
    const float mgx = q[2] * inv_d * rx;  // mean of g x^
    const float mg = a.pre == kLayer ? q[3] * inv_d : 0.f;
    float p[2] = {0.f, 0.f};
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      if (!live[c]) continue;
      const int col = (c * T + (int)threadIdx.x) * 8;
      float sc[8], gt[8];
      load_mod8(a.scale, s * a.D + col, 0.f, sc);
      load_mod8(a.gate, s * a.D + col, 1.f, gt);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float xh = x[c][i] * rx;
        acc[1][c][i] = fmaf(g[c][i], xh, acc[1][c][i]);
        if (a.dn) d[c][i] = fmaf(rx, g[c][i] * (1.0f + sc[i]) - mg - xh * mgx, d[c][i]);
        u[c][i] *= ru;
        acc[0][c][i] = fmaf(d[c][i], u[c][i], acc[0][c][i]);
        const float w = gt[i] * d[c][i];
        p[0] = fmaf(w, u[c][i], p[0]);
        p[1] += w;
        x[c][i] = w;
      }
    }
    if (a.dh) {
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        if (!live[c]) continue;
#pragma unroll
        for (int i = 0; i < 8; ++i) d[c][i] *= a.alpha;
        store_stream8<FP32>(a.dh, at + (c * T + (int)threadIdx.x) * 8, d[c]);
      }
    }
    if (a.db) {
      float mwu = 0.f, mw = 0.f;
      if (a.post != kNone) {
        row_sums<2>(p, warps, slot + 6);
        mwu = p[0] * inv_d;
        mw = a.post == kLayer ? p[1] * inv_d : 0.f;
      }
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        if (!live[c]) continue;
#pragma unroll
        for (int i = 0; i < 8; ++i) x[c][i] = ru * (x[c][i] - mw - u[c][i] * mwu);
        st_stream(reinterpret_cast<uint16_t*>(a.db) + at + (c * T + (int)threadIdx.x) * 8, pack8(x[c]));
      }
    }
  }
  float* out = a.sums + (int64_t)blockIdx.x * 3 * a.D;
#pragma unroll
  for (int k = 0; k < 3; ++k) {
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int col = (c * T + (int)threadIdx.x) * 8;
      if (col >= a.D) continue;
      float4* o = reinterpret_cast<float4*>(out + (int64_t)k * a.D + col);
      o[0] = make_float4(acc[k][c][0], acc[k][c][1], acc[k][c][2], acc[k][c][3]);
      o[1] = make_float4(acc[k][c][4], acc[k][c][5], acc[k][c][6], acc[k][c][7]);
    }
  }
}

// out_k[s] = the sum of a segment's partials, in the order of its chunks.
__global__ void __launch_bounds__(128) k_segment_sums(const float* __restrict__ sums, int64_t seg_chunks, int D,
                                                      float* __restrict__ o0, float* __restrict__ o1,
                                                      float* __restrict__ o2, int64_t S) {
  const int col = (blockIdx.x * 128 + threadIdx.x) * 4;
  if (col >= D) return;
  float* out = blockIdx.z == 0 ? o0 : (blockIdx.z == 1 ? o1 : o2);
  if (!out) return;
  for (int64_t s = blockIdx.y; s < S; s += gridDim.y) {
    const float* src = sums + (s * seg_chunks * 3 + blockIdx.z) * D + col;
    float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
    for (int64_t i = 0; i < seg_chunks; ++i) {
      const float4 v = __ldg(reinterpret_cast<const float4*>(src + i * 3 * D));
      t.x += v.x;
      t.y += v.y;
      t.z += v.z;
      t.w += v.w;
    }
    *reinterpret_cast<float4*>(out + s * D + col) = t;
  }
}

template <bool FP32, int CH>
cudaError_t norm_launch(const NormArgs& a, int warps, cudaStream_t s) {
  if (warps == 1) {
    k_block_norm<FP32, CH, true><<<(unsigned)((a.rows + 3) / 4), 128, 0, s>>>(a);
  } else {
    k_block_norm<FP32, CH, false><<<(unsigned)a.rows, 32 * warps, 0, s>>>(a);
  }
  return cudaGetLastError();
}

template <bool FP32>
cudaError_t norm_dispatch(const NormArgs& a, cudaStream_t s) {
  // Up to 1024 values a lane's four chunks hold a row; wider rows take more warps.
  if (a.D <= 256) return norm_launch<FP32, 1>(a, 1, s);
  if (a.D <= 512) return norm_launch<FP32, 2>(a, 1, s);
  return norm_launch<FP32, 4>(a, (a.D + 1023) / 1024, s);
}

// Rows per CTA of the backward pass.
constexpr int64_t kChunkRows = 64;

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
  a.alpha = p.alpha;
  a.eps = p.eps;
  return p.fp32 ? norm_dispatch<true>(a, s) : norm_dispatch<false>(a, s);
}

int64_t block_norm_backward_chunks(int64_t M, int64_t segment_tokens, int64_t* per_segment) {
  const int64_t S = (M + segment_tokens - 1) / segment_tokens;
  const int64_t rows = segment_tokens < M ? segment_tokens : M;
  *per_segment = (rows + kChunkRows - 1) / kChunkRows;
  return S * *per_segment;
}

cudaError_t launch_block_norm_backward(const BlockNormBackwardLaunch& p, int* kernels, cudaStream_t s) {
  BackArgs a;
  a.dn = p.dn;
  a.dh_out = p.dh_out;
  a.h = p.h_out;
  a.b = p.b;
  a.gate = p.gate;
  a.scale = p.scale;
  a.dh = p.dh;
  a.db = p.db;
  a.sums = p.workspace;
  a.M = p.M;
  a.seg = p.segment_tokens < p.M ? p.segment_tokens : p.M;
  const int64_t chunks = block_norm_backward_chunks(p.M, a.seg, &a.seg_chunks);
  a.chunk_rows = kChunkRows;
  a.D = p.D;
  a.post = p.post;
  a.pre = p.pre;
  a.alpha = p.alpha;
  a.eps = p.eps;
  const int T = 32 * ((p.D / 8 + 31) / 32);
  *kernels = 1;
  if (p.D <= 8192) {
    if (p.fp32) k_block_norm_backward<true, 1><<<(unsigned)chunks, T, 0, s>>>(a);
    else k_block_norm_backward<false, 1><<<(unsigned)chunks, T, 0, s>>>(a);
  } else {
    const int T2 = 32 * ((p.D / 8 + 63) / 64);
    if (p.fp32) k_block_norm_backward<true, 2><<<(unsigned)chunks, T2, 0, s>>>(a);
    else k_block_norm_backward<false, 2><<<(unsigned)chunks, T2, 0, s>>>(a);
  }
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  if (p.dgate || p.dscale || p.dshift) {
    const int64_t S = chunks / a.seg_chunks;
    const dim3 grid((unsigned)((p.D / 4 + 127) / 128), (unsigned)(S < 65535 ? S : 65535), 3);
    k_segment_sums<<<grid, 128, 0, s>>>(a.sums, a.seg_chunks, p.D, p.dgate, p.dscale, p.dshift, S);
    *kernels = 2;
    e = cudaGetLastError();
  }
  return e;
}

}  // namespace lg
