// lg_lora_linear_mxfp4 on output tiles:
//
//   D[M, N] = deq(aq) deq(bq)^T  (MXFP4, optional)  +  a b^T  (bf16, optional)
//
// one kernel for both products of the layer: h = x A_cat^T (bf16 part alone,
// its N the ranks) and y = deq(x) deq(W)^T + h B_cat^T (both parts into one
// accumulator).
//
// The panel kernel of the bf16 and MXFP8 layers keeps h on the chip: an SM pair
// owns 256 tokens, computes their h and then all their output columns.  In
// 4 bits the base term takes a quarter of the bf16 time, and what the panel
// costs weighs more: tokens that do not fill every cluster's panel leave SMs
// idle (20 panels on 33 clusters: 60 %), and its tensor memory is full of h,
// with room for four scale buffers.  So here h goes through memory (2 x 2 M R
// bytes, under 1 % of the time at R = 576) and any SM pair takes any tile:
//
//   * persistent CTA pairs (tcgen05.mma cta_group::2, M = 256 tokens x TN
//     columns), all 148 SMs; each CTA loads its 128 token rows and half of the
//     tile's TN weight rows per stage by TMA into 128-byte swizzled rows: 256 K
//     in 4 bits, with the stage's scales behind them, or 64 K in bf16.
//   * TMEM: TN <= 192 keeps two accumulators, so a tile's epilogue runs under
//     the next tile's products; the rest holds the scales of four stages.  The
//     thread that issues the MMAs also issues the scale copies (tcgen05.cp):
//     tcgen05 executes one thread's copies and MMAs in order, so neither needs
//     a wait of its own.
//   * A_cat, h and B_cat are rounded to bf16, as in the other layers: against an
//     FP32 evaluation of the adapters' term a difference of 0.0022 in y (relative
//     Frobenius; y's own rounding is 0.0016, and the base term's 4-bit codes move
//     it by 0.16).  Pairs of bf16 parts instead would take a second product for h
//     and two more for y: 0.5 of 1.6 ms at 16384 x 28672 -> 7168, rank 576, by the
//     rate.
//   * tiles run over blocks of eight panels, panels fastest: the 74 tiles in
//     flight share eight panels of x and nine tiles of W in L2.
//   * the second launch is a programmatic dependent of the first: its 4-bit
//     part runs on SMs that h does not fill, and its producers wait for h only
//     before their first load of it.
//
// Warp 0 loads, warp 1 owns tensor memory and issues copies and MMAs from one
// thread, warps 2-9 are the epilogue (bf16, TMA stores).  Every mbarrier wait
// is bounded, as in the panel kernel.
#include <atomic>

#include "lg_internal.h"
#include "lg_pipeline.cuh"

namespace lg {

namespace {

std::atomic<bool> g_launched{false};  // so that the error word may be set

constexpr int BM = 128;  // token rows per CTA
constexpr uint32_t A_BYTES = BM * 128;
constexpr uint32_t SF_GROUP = 512;  // scales of 128 rows x 128 K
constexpr int THREADS = 320;
constexpr int EPI_WARPS = 8;
constexpr int MAX_STAGES = 8;
constexpr uint32_t TMEM_COLS = 512;
constexpr uint32_t Y_WARP_BYTES = Y_BOX * Y_BOX * 2;
constexpr uint32_t Y_BYTES = EPI_WARPS * Y_WARP_BYTES;
constexpr size_t MAX_SMEM = 232448;
constexpr int RASTER = 8;  // panels per block of tiles

template <int TN>
struct Cfg {
  static constexpr int ACCS = TN <= 192 ? 2 : 1;
  static constexpr int W_GROUPS = TN > 128 ? 2 : 1;  // 128-row scale groups a tile's columns touch
  static constexpr uint32_t SF_COL = ACCS * TN;
  static constexpr uint32_t SF_K = 4 + 4 * W_GROUPS;     // TMEM columns of one 128-K group's scales
  static constexpr uint32_t SF_STAGE_COLS = 32;          // two groups, padded
  static constexpr uint32_t SF_BUFS = (TMEM_COLS - SF_COL) / SF_STAGE_COLS < 4 ? (TMEM_COLS - SF_COL) / SF_STAGE_COLS : 4;
  static constexpr uint32_t B_ROWS = TN / 2;
  static constexpr uint32_t B_BYTES = B_ROWS * 128;
  static constexpr uint32_t SF_BYTES = 2 * (1 + W_GROUPS) * SF_GROUP;
  static constexpr uint32_t STAGE = A_BYTES + B_BYTES + SF_BYTES;
  static constexpr int HALF = TN / 2;  // accumulator columns per epilogue warp
  static_assert(TN % 64 == 0 && HALF % 32 == 0 && SF_BUFS >= 2 && 2 * SF_K <= SF_STAGE_COLS, "tile layout");
  static_assert(STAGE % 1024 == 0, "stages must stay 1024-byte aligned");
};

struct Control {
  uint64_t full[MAX_STAGES];   // a stage's loads have landed (both CTAs', counted on the leader)
  uint64_t empty[MAX_STAGES];  // the MMAs are done with a stage
  uint64_t acc_full[2];        // a tile's accumulator is complete
  uint64_t acc_empty[2];       // the epilogue has drained it (on the leader)
  uint64_t drain;              // every MMA and copy has finished
  uint32_t tmem_base;
  int abort_flag;
};

struct Args {
  int64_t M;
  int N, panels, n_tiles, tiles;
  int q_stages;   // 256-K stages of the 4-bit part (0: none)
  int q_groups;   // 128-K scale groups of the 4-bit part
  int h_stages;   // 64-K stages of the bf16 part
  int stages;
  uint32_t y_off, control_off;
  unsigned long long wait_limit_ns;
};

// Tile i: token panel p, column tile t; blocks of RASTER panels, panels fastest.
__device__ __forceinline__ void tile_at(const Args& a, int i, int& p, int& t) {
  const int per = RASTER * a.n_tiles;
  const int block = i / per, r = i - block * per;
  const int rows = min(RASTER, a.panels - block * RASTER);
  t = r / rows;
  p = block * RASTER + (r - t * rows);
}

template <int TN>
__device__ void produce(const CUtensorMap* tm_aq, const CUtensorMap* tm_bq, const CUtensorMap* tm_sa,
                        const CUtensorMap* tm_sb, const CUtensorMap* tm_a, const CUtensorMap* tm_b, const Args& a,
                        Control* ctl, uint32_t smem, uint32_t half, uint32_t cid, uint32_t ncl,
                        volatile int* abort_flag) {
  using C = Cfg<TN>;
  const uint32_t full_local = smem_u32(&ctl->full[0]);
  const uint32_t full0 = mapa_shared(full_local, 0);
  const uint32_t empty0 = smem_u32(&ctl->empty[0]);
  const uint32_t stages = (uint32_t)a.stages;
  uint32_t stage = 0, phase = 0;
  uint64_t fills = 0;
  bool ok = true, waited = false;
  for (int i = (int)cid; ok && i < a.tiles; i += (int)ncl) {
    int p, t;
    tile_at(a, i, p, t);
    const int m0 = (2 * p + (int)half) * BM;
    const int n0 = t * TN + (int)half * (int)C::B_ROWS;
    const int g0 = t * TN / 128;  // first scale group of the tile's columns
    for (int kb = 0; kb < a.q_stages; ++kb) {
      if (!all_waited(wait_limited(empty0 + 8 * stage, phase ^ 1, a.wait_limit_ns, abort_flag))) {
        ok = false;
        break;
      }
      const uint32_t sa = smem + stage * C::STAGE;
      const uint32_t bar = full0 + 8 * stage;
      if (elect_lane()) {
        if (half == 0) mbar_arrive_expect_tx(full_local + 8 * stage, 2 * (A_BYTES + C::B_BYTES + C::SF_BYTES));
        tma_load_2d_pair(sa, tm_aq, bar, kb * 128, m0);
        tma_load_2d_pair(sa + A_BYTES, tm_bq, bar, kb * 128, n0);
        // Each CTA's tensor memory takes its own rows' scales and those of all
        // the tile's columns, two 512-byte groups (four 256-byte rows of the
        // map) at a time; past an odd last group: bytes that no MMA reads.
        const uint32_t sf = sa + A_BYTES + C::B_BYTES;
        tma_load_2d_pair(sf, tm_sa, bar, 0, 2 * ((m0 / BM) * a.q_groups + 2 * kb));
#pragma unroll
        for (int w = 0; w < C::W_GROUPS; ++w)
          tma_load_2d_pair(sf + (1 + w) * 2 * SF_GROUP, tm_sb, bar, 0, 2 * ((g0 + w) * a.q_groups + 2 * kb));
      }
      __syncwarp();
      ++fills;
      advance(stage, phase, stages);
    }
    if (ok && a.h_stages > 0 && !waited) {
      asm volatile("griddepcontrol.wait;" ::: "memory");  // the bf16 operands are there
      waited = true;
    }
    for (int kb = 0; ok && kb < a.h_stages; ++kb) {
      if (!all_waited(wait_limited(empty0 + 8 * stage, phase ^ 1, a.wait_limit_ns, abort_flag))) {
        ok = false;
        break;
      }
      const uint32_t sa = smem + stage * C::STAGE;
      const uint32_t bar = full0 + 8 * stage;
      if (elect_lane()) {
        if (half == 0) mbar_arrive_expect_tx(full_local + 8 * stage, 2 * (A_BYTES + C::B_BYTES));
        tma_load_2d_pair(sa, tm_a, bar, kb * BK, m0);
        tma_load_2d_pair(sa + A_BYTES, tm_b, bar, kb * BK, n0);
      }
      __syncwarp();
      ++fills;
      advance(stage, phase, stages);
    }
  }
  // Also after a wait that ran out: the grid does not end before the one it depends on.
  if (a.h_stages > 0 && !waited) asm volatile("griddepcontrol.wait;" ::: "memory");
  if (half == 0) {
    // The leader's barriers count both CTAs' bytes: every copy has landed.
    for (uint32_t s = 0; s < stages; ++s) {
      const uint64_t fs = fills / stages + (s < fills % stages ? 1 : 0);
      if (fs) wait_teardown(full_local + 8 * s, (uint32_t)((fs - 1) & 1), abort_flag);
    }
  } else if (!ok) {
    // A follower that gave up cannot observe them; its copies in flight land
    // within microseconds.
    const uint64_t t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < 200000ull) {
    }
  }
}

// In both issuing warps all lanes walk the stages and one elected lane issues:
// addresses and descriptors stay warp-uniform values, which TMA and tcgen05
// instructions take from uniform registers.  (From a divergent lane every
// operand is moved there first: a stage's eight loads alone then took 0.53 us,
// twice its MMAs' time at any tile width.)
template <int TN>
__device__ void multiply(const Args& a, Control* ctl, uint32_t smem, uint32_t tmem, uint32_t cid, uint32_t ncl,
                         volatile int* abort_flag) {
  using C = Cfg<TN>;
  const uint32_t stages = (uint32_t)a.stages;
  const uint32_t full0 = smem_u32(&ctl->full[0]);
  const uint32_t empty0 = smem_u32(&ctl->empty[0]);
  constexpr uint32_t idesc = idesc_bf16_f32(2 * BM, TN);
  uint32_t stage = 0, phase = 0, n = 0, sf_buf = 0;
  bool ok = true;
  for (int i = (int)cid; ok && i < a.tiles; i += (int)ncl, ++n) {
    int p, t;
    tile_at(a, i, p, t);
    const uint32_t buf = n % C::ACCS;
    const uint32_t d = tmem + buf * TN;
    // Columns of the tile start at row t TN of W: a multiple of 64, so up to
    // two scale columns (32 rows each) into the first group.
    const uint32_t sb_shift = (uint32_t)(t * TN % 128) / 32;
    if (!all_waited(wait_limited(smem_u32(&ctl->acc_empty[buf]), (n / C::ACCS + 1) & 1, a.wait_limit_ns, abort_flag, true)))
      break;
    tc_fence_after();
    for (int kb = 0; kb < a.q_stages; ++kb) {
      if (!all_waited(wait_limited(full0 + 8 * stage, phase, a.wait_limit_ns, abort_flag))) {
        ok = false;
        break;
      }
      tc_fence_after();
      const uint32_t sa = smem + stage * C::STAGE;
      const uint64_t da = sw128_kmajor_desc(sa), db = sw128_kmajor_desc(sa + A_BYTES);
      const int groups = min(2, a.q_groups - 2 * kb);
      const uint32_t sf0 = tmem + C::SF_COL + C::SF_STAGE_COLS * sf_buf;
      if (elect_lane()) {
        for (int g = 0; g < groups; ++g) {
          const uint32_t src = sa + A_BYTES + C::B_BYTES + (uint32_t)g * SF_GROUP;
#pragma unroll
          for (int w = 0; w < 1 + C::W_GROUPS; ++w)
            tmem_cp_32x128b_x4_pair(sf0 + (uint32_t)g * C::SF_K + 4 * w, plain_rows16_desc(src + 2 * w * SF_GROUP));
        }
        for (int g = 0; g < groups; ++g) {
          const uint32_t sf = sf0 + (uint32_t)g * C::SF_K;
#pragma unroll
          for (int k = 0; k < 2; ++k) {  // K = 64 each, bytes 2 k and 2 k + 1 of the scale words
            umma_mxf4_pair(d, da + 2 * (2 * g + k), db + 2 * (2 * g + k),
                           idesc_mxf4(2 * BM, TN, 2u * (uint32_t)k, 2u * (uint32_t)k), sf, sf + 4 + sb_shift,
                           (kb | g | k) != 0);
          }
        }
        umma_commit_pair_mc(empty0 + 8 * stage, 3);
      }
      __syncwarp();
      if (++sf_buf == C::SF_BUFS) sf_buf = 0;
      advance(stage, phase, stages);
    }
    for (int kb = 0; ok && kb < a.h_stages; ++kb) {
      if (!all_waited(wait_limited(full0 + 8 * stage, phase, a.wait_limit_ns, abort_flag))) {
        ok = false;
        break;
      }
      tc_fence_after();
      const uint32_t sa = smem + stage * C::STAGE;
      const uint64_t da = sw128_kmajor_desc(sa), db = sw128_kmajor_desc(sa + A_BYTES);
      if (elect_lane()) {
#pragma unroll
        for (int k = 0; k < BK / 16; ++k) umma_ss_pair(d, da + 2 * k, db + 2 * k, idesc, (a.q_stages | kb | k) != 0);
        umma_commit_pair_mc(empty0 + 8 * stage, 3);
      }
      __syncwarp();
      advance(stage, phase, stages);
    }
    if (!ok) break;
    if (elect_lane()) umma_commit_pair_mc(smem_u32(&ctl->acc_full[buf]), 3);
    __syncwarp();
  }
  // Every MMA and copy must finish before TMEM is freed or either CTA exits.
  if (elect_lane()) umma_commit_pair_mc(smem_u32(&ctl->drain), 3);
  __syncwarp();
  wait_teardown(smem_u32(&ctl->drain), 0, abort_flag);
}

template <int TN>
__device__ void store_tiles(const CUtensorMap* tm_y, const Args& a, Control* ctl, uint32_t smem, uint32_t tmem,
                            uint32_t half, uint32_t cid, uint32_t ncl, int warp, int lane, volatile int* abort_flag) {
  using C = Cfg<TN>;
  const int q = warp & 3;           // TMEM lane quarter
  const int side = (warp - 2) >> 2;  // half of the tile's columns
  const uint32_t lanes = tmem + ((uint32_t)(32 * q) << 16);
  const uint32_t acc_full0 = smem_u32(&ctl->acc_full[0]);
  const uint32_t acc_empty0 = mapa_shared(smem_u32(&ctl->acc_empty[0]), 0);
  const uint32_t buf_y = smem + a.y_off + (uint32_t)(warp - 2) * Y_WARP_BYTES;
  const uint32_t my = buf_y + (uint32_t)lane * (Y_BOX * 2);
  const uint32_t sw = ((uint32_t)lane >> 1) & 3u;
  const uint64_t pol = l2_policy_evict_first();
  uint32_t n = 0;
  for (int i = (int)cid; i < a.tiles; i += (int)ncl, ++n) {
    int p, t;
    tile_at(a, i, p, t);
    const uint32_t buf = n % C::ACCS;
    if (!__all_sync(0xffffffffu,
                    wait_limited(acc_full0 + 8 * buf, (n / C::ACCS) & 1, a.wait_limit_ns, abort_flag)))
      break;
    tc_fence_after();
    uint32_t v[C::HALF / 32][32];
#pragma unroll
    for (int c = 0; c < C::HALF / 32; ++c) tmem_ld_32x32b_x32(lanes + buf * TN + (uint32_t)(side * C::HALF + 32 * c), v[c]);
    tmem_wait_ld();
    // Hand the accumulator back before converting (nothing is published: relaxed).
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive_remote_relaxed(acc_empty0 + 8 * buf);
    const int row0 = (2 * p + (int)half) * BM + 32 * q;
    const int col0 = t * TN + side * C::HALF;
#pragma unroll
    for (int c = 0; c < C::HALF / 32; ++c) {
      if (col0 + 32 * c >= a.N || row0 >= a.M) break;  // the box lies outside (N is a multiple of 32)
      if (lane == 0) bulk_wait_group_read0();
      __syncwarp();
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t* w = &v[c][8 * k];
        const uint32_t at = my + (((uint32_t)k ^ sw) << 4);
        asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at),
                     "r"(pack_bf16x2(__uint_as_float(w[0]), __uint_as_float(w[1]))),
                     "r"(pack_bf16x2(__uint_as_float(w[2]), __uint_as_float(w[3]))),
                     "r"(pack_bf16x2(__uint_as_float(w[4]), __uint_as_float(w[5]))),
                     "r"(pack_bf16x2(__uint_as_float(w[6]), __uint_as_float(w[7])))
                     : "memory");
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        tma_store_2d_hint(tm_y, buf_y, col0 + 32 * c, row0, pol);
        bulk_commit_group();
      }
    }
  }
  if (lane == 0) bulk_wait_group0();
  __syncwarp();
}

template <int TN>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(THREADS, 1)
    k_mxfp4_tile(const __grid_constant__ CUtensorMap tm_aq, const __grid_constant__ CUtensorMap tm_bq,
                 const __grid_constant__ CUtensorMap tm_sa, const __grid_constant__ CUtensorMap tm_sb,
                 const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b,
                 const __grid_constant__ CUtensorMap tm_y, const Args a) {
  using C = Cfg<TN>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  Control* ctl = reinterpret_cast<Control*>(base + a.control_off);
  const uint32_t smem = smem_u32(base);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const uint32_t half = cluster_ctarank();
  const uint32_t cid = cluster_id_x(), ncl = cluster_count_x();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (threadIdx.x == 0) {
    for (int s = 0; s < a.stages; ++s) {
      mbar_init(smem_u32(&ctl->full[s]), 1);
      mbar_init(smem_u32(&ctl->empty[s]), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(smem_u32(&ctl->acc_full[b]), 1);
      mbar_init(smem_u32(&ctl->acc_empty[b]), 2 * EPI_WARPS);
    }
    mbar_init(smem_u32(&ctl->drain), 1);
    ctl->abort_flag = 0;
    fence_mbarrier_init();
    if (a.q_stages > 0) {
      tma_prefetch_desc(&tm_aq);
      tma_prefetch_desc(&tm_bq);
      tma_prefetch_desc(&tm_sa);
      tma_prefetch_desc(&tm_sb);
    }
    if (a.h_stages > 0) {
      tma_prefetch_desc(&tm_a);
      tma_prefetch_desc(&tm_b);
    }
    tma_prefetch_desc(&tm_y);
  }
  if (warp == 1) {
    tmem_alloc_pair(smem_u32(&ctl->tmem_base), TMEM_COLS);
    tmem_relinquish_pair();
    tc_fence_before();
  }
  cluster_sync_all();
  tc_fence_after();
  const uint32_t tmem = ctl->tmem_base;
  volatile int* abort_flag = &ctl->abort_flag;
  if (warp == 0) {
    produce<TN>(&tm_aq, &tm_bq, &tm_sa, &tm_sb, &tm_a, &tm_b, a, ctl, smem, half, cid, ncl, abort_flag);
  } else if (warp == 1) {
    if (half == 0) multiply<TN>(a, ctl, smem, tmem, cid, ncl, abort_flag);
    __syncwarp();
  } else {
    store_tiles<TN>(&tm_y, a, ctl, smem, tmem, half, cid, ncl, warp, lane, abort_flag);
  }
  tc_fence_before();
  __syncthreads();
  // The leader's MMAs read the follower's shared memory and write its TMEM:
  // the follower waits for the (multicast) drain commit.
  if (half == 1 && warp == 1 && lane == 0)
    wait_teardown(smem_u32(&ctl->drain), 0, abort_flag, a.wait_limit_ns + TEARDOWN_LIMIT_NS);
  cluster_sync_all();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, TMEM_COLS);
  }
  cluster_sync_all();
}

// One product: its operands (null codes: no 4-bit part; bf16_k 0: no bf16 part).
struct Product {
  const void* aq = nullptr;
  const void* sa = nullptr;
  const void* bq = nullptr;
  const void* sb = nullptr;
  int q_k = 0;
  const void* a = nullptr;
  const void* b = nullptr;
  int bf16_k = 0;
  void* y = nullptr;
  int64_t M = 0;
  int N = 0;
  bool dependent = false;  // launched as a programmatic dependent of the kernel before
};

template <int TN>
cudaError_t tile_launch(const Product& p, int pairs, uint64_t wait_limit_ns, cudaStream_t s, bool* driver_failed,
                        PFN_cuTensorMapEncodeTiled_v12000 enc) {
  using C = Cfg<TN>;
  CUtensorMap tm_aq, tm_bq, tm_sa, tm_sb, tm_a, tm_b, tm_y;
  bool ok = make_store_map(enc, &tm_y, p.y, (uint64_t)p.N, (uint64_t)p.M);
  tm_aq = tm_bq = tm_sa = tm_sb = tm_a = tm_b = tm_y;  // the parts a call lacks are never read
  if (p.q_k > 0) {
    const uint64_t groups = (uint64_t)p.q_k / BKQ;
    ok = ok && make_map_codes(enc, &tm_aq, p.aq, (uint64_t)p.q_k / 2, (uint64_t)p.M, BM) &&
         make_map_codes(enc, &tm_bq, p.bq, (uint64_t)p.q_k / 2, (uint64_t)p.N, C::B_ROWS) &&
         make_map_scales(enc, &tm_sa, p.sa, (uint64_t)((p.M + 127) / 128) * groups, 4) &&
         make_map_scales(enc, &tm_sb, p.sb, (uint64_t)((p.N + 127) / 128) * groups, 4);
  }
  if (p.bf16_k > 0) {
    ok = ok && make_map(enc, &tm_a, p.a, (uint64_t)p.bf16_k, (uint64_t)p.M, BM) &&
         make_map(enc, &tm_b, p.b, (uint64_t)p.bf16_k, (uint64_t)p.N, C::B_ROWS);
  }
  if (!ok) {
    *driver_failed = true;
    return cudaErrorInvalidValue;
  }
  Args a;
  a.M = p.M;
  a.N = p.N;
  a.panels = (int)((p.M + 2 * BM - 1) / (2 * BM));
  a.n_tiles = (p.N + TN - 1) / TN;
  a.tiles = a.panels * a.n_tiles;
  a.q_stages = (p.q_k + 255) / 256;
  a.q_groups = p.q_k / BKQ;
  a.h_stages = p.bf16_k / BK;
  constexpr size_t fixed = 1024 + Y_BYTES + sizeof(Control);
  a.stages = (int)((MAX_SMEM - fixed) / C::STAGE);
  if (a.stages > MAX_STAGES) a.stages = MAX_STAGES;
  a.y_off = (uint32_t)a.stages * C::STAGE;
  a.control_off = a.y_off + Y_BYTES;
  a.wait_limit_ns = wait_limit_ns;
  cudaError_t e = allow_shared_memory((const void*)k_mxfp4_tile<TN>, (int)MAX_SMEM);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(2 * (a.tiles < pairs ? a.tiles : pairs)), 1, 1);
  cfg.blockDim = dim3(THREADS, 1, 1);
  cfg.dynamicSmemBytes = fixed + (size_t)a.stages * C::STAGE;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = p.dependent ? 1 : 0;
  g_launched.store(true);
  return cudaLaunchKernelEx(&cfg, k_mxfp4_tile<TN>, tm_aq, tm_bq, tm_sa, tm_sb, tm_a, tm_b, tm_y, a);
}

// Column tile of a product: the fewest rounds of tiles over the SM pairs times a
// tile's time, which is its columns plus what does not shrink with them (the 256
// token rows' share of the operand traffic, the tile's start and end).  h's
// product runs beside the 4-bit part of the main one and need not fill the device:
// the least work by its columns alone (2304 x 7168 -> 7168, rank 576, the whole
// layer: h in 192 columns 95 us, in 128 103, in 64 118; splitting its K over idle
// pairs instead: 105 and up).
int tile_columns(const Product& p, int pairs) {
  const int64_t panels = p.q_k > 0 ? (p.M + 2 * BM - 1) / (2 * BM) : 1;
  int best = 64;
  double least = 1e300;
  for (int tn : {256, 192, 128, 64}) {
    const int64_t tiles = panels * ((p.N + tn - 1) / tn);
    const double cost = (double)(p.q_k > 0 ? (tiles + pairs - 1) / pairs : tiles) * (tn + 64);
    if (cost < least) {
      least = cost;
      best = tn;
    }
  }
  return best;
}

cudaError_t product_launch(const Product& p, int sm_count, uint64_t wait_limit_ns, cudaStream_t s, bool* driver_failed,
                           PFN_cuTensorMapEncodeTiled_v12000 enc) {
  const int pairs = sm_count / 2;
  switch (tile_columns(p, pairs)) {
    case 256: return tile_launch<256>(p, pairs, wait_limit_ns, s, driver_failed, enc);
    case 192: return tile_launch<192>(p, pairs, wait_limit_ns, s, driver_failed, enc);
    case 128: return tile_launch<128>(p, pairs, wait_limit_ns, s, driver_failed, enc);
    default: return tile_launch<64>(p, pairs, wait_limit_ns, s, driver_failed, enc);
  }
}

}  // namespace

cudaError_t take_tile_error(int* value) {
  *value = 0;
  return g_launched.load() ? take_device_error(value) : cudaSuccess;
}

cudaError_t launch_lora_linear_tiles(const LinearLaunch& p, uint16_t* h, int* kernels, cudaStream_t s,
                                     bool* driver_failed) {
  *driver_failed = false;
  *kernels = 0;
  PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
  if (!enc) {
    *driver_failed = true;
    return cudaErrorNotSupported;
  }
  Product y;
  y.aq = p.xq;
  y.sa = p.xsf;
  y.bq = p.wq;
  y.sb = p.wsf;
  y.q_k = p.K;
  y.y = p.y;
  y.M = p.M;
  y.N = p.N;
  if (p.R > 0) {
    Product d;
    d.a = p.x;
    d.b = p.A_bf16;
    d.bf16_k = p.K;
    d.y = h;
    d.M = p.M;
    d.N = p.R;
    d.dependent = true;  // of the factors' copy
    const cudaError_t e = product_launch(d, p.sm_count, p.wait_limit_ns, s, driver_failed, enc);
    if (e != cudaSuccess) return e;
    *kernels += 1;
    y.a = h;
    y.b = p.B_bf16;
    y.bf16_k = p.R;
    y.dependent = true;  // of h
  }
  const cudaError_t e = product_launch(y, p.sm_count, p.wait_limit_ns, s, driver_failed, enc);
  if (e == cudaSuccess) *kernels += 1;
  return e;
}

}  // namespace lg
