// FP8 linear layer, token-major kernel: many tokens (sm_103a).
//
// A pair of CTAs (cta_group::2) computes 256 tokens x 256 weight rows: each CTA holds its own
// 128 tokens and 128 of the 256 weight rows in shared memory, the tensor core reads both
// CTAs' weight tiles, and each CTA's TMEM gets its 128 tokens x 256 outputs.  So a CTA loads
// 32 KB per 128-column k-block where one alone would load 48 KB.  SwiGLU pairs the 128 gate
// rows (first CTA) with the 128 matching up rows (second CTA).
//
// The scales are general fp32 per 128 columns, so every k-block's product is read from TMEM
// and added into registers times xs[m, kb] * ws[rb, kb] (128 KB per CTA and k-block, two
// 256-column slots in turn).  Multiplications and copies alone take 734 cycles per k-block, with
// the reading it is 830, and the end of a tile takes 2,700 (SwiGLU to codes some 5,800, 4,700 of
// them but for the exponentials).  4096 x 7168 x 3584 in 81 us, 8192 x 4096 x 7168 SwiGLU to codes
// in 187 us (2.6 PFLOP/s) in a burst at full clock; 87 and 200 us (2.4) in a run of seconds, which
// the power limit holds at 1.9 GHz.
//
// Persistent: one pair per two SMs, tiles dealt round robin, token tiles fastest (the pairs
// that run together share weight tiles in L2).  Where there are too few tiles for that, two
// pairs form a cluster and share one tile's K; at the end each warp's 32 rows go to the pair
// that finishes them, through distributed shared memory, and are added in rank order (four
// pairs, clusters of 8 CTAs that fill their SMs, were slower at every size).
#include "klt_linear.cuh"

#include "../../include/klt.h"

namespace klt {
namespace {

constexpr int THREADS = 384;  // warps 0 copies, 1 MMA, 2 TMEM, 3 idle, 4-11 epilogue
constexpr int STAGES = 5;
constexpr int STAGE_BYTES = 2 * LIN_TILE_BYTES;
constexpr int RING_BYTES = STAGES * STAGE_BYTES;
constexpr int BOX_BYTES = 32 * 128;        // stored at a time by a warp: 32 rows x 128 bytes
constexpr int BOXES = 2;                   // per epilogue warp
constexpr int OUT_BYTES = 8 * BOXES * BOX_BYTES;
constexpr int PART_BYTES = 32 * 128 * 4;  // a warp's 32 rows x 128 columns, fp32
constexpr int AMAX_BYTES = 2 * 128 * 4;
constexpr int SMEM = 1024 + RING_BYTES + OUT_BYTES + AMAX_BYTES + 256;
static_assert(SMEM <= 232448, "shared memory of a block");

struct Smem {
  uint8_t *ring, *stage;
  float* amax;  // [2][128]
  uint64_t *full, *done, *tempty, *drain, *ended;
  uint32_t *tmem_holder, *copies;
  volatile int* abort_flag;
};

// The output leaves through a warp's two boxes of 32 rows x 128 bytes (codes: one of 64 bytes):
// staged in the output map's swizzle (no bank conflicts) and stored by bulk copies, which cut
// off what lies outside the output and run on while the warp goes on.  Few and large ones: the
// copies queue behind the loads, some 400 cycles each.  Lane b issues the copy of box b.
KLT_DEV void boxes_free() {  // the warp's copies have read their boxes
  tma_store_wait_read<0>();
  __syncwarp();
}
// This thread's BYTES (64 or 128, in w) of row `lane` of a box.
template <int BYTES>
KLT_DEV void fill_box(uint8_t* box, const uint32_t* w) {
  const int lane = lane_id(), x = BYTES == 128 ? lane & 7 : (lane >> 1) & 3;
#pragma unroll
  for (int j = 0; j < BYTES / 16; ++j)
    *reinterpret_cast<uint4*>(box + lane * BYTES + (j ^ x) * 16) =
        make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
}
// Stores the filled boxes to rows m0 .. m0 + 31: lane b holds box b's byte column, or one that
// is past the row's `bytes` (then it issues none: a copy starts inside the output).
KLT_DEV void store_boxes(const uint8_t* boxes, const CUtensorMap* omap, int col, int bytes,
                         int m0) {
  fence_proxy_async_shared();
  __syncwarp();
  if (col < bytes) tma_store_2d(omap, boxes + lane_id() * BOX_BYTES, col, m0);
}
// A warp's 2 x 64 columns (128 apart, from c on) of its 32 rows from m0 on; this thread's row
// in v, two values each.  COUNT = 1: the first 64 only.
template <int COUNT>
KLT_DEV void store_rows(const LinParams& p, const CUtensorMap* omap, uint8_t* boxes, int m0,
                        int c, const unsigned long long (*v)[32]) {
  if (m0 >= p.M) return;
  const int lane = lane_id();
  if (p.out_wide && p.out_dtype == KLT_DT_F32) {
#pragma unroll
    for (int g = 0; g < COUNT; ++g) {
      boxes_free();
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        uint32_t w[32];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          w[2 * i] = static_cast<uint32_t>(v[g][b * 16 + i]);
          w[2 * i + 1] = static_cast<uint32_t>(v[g][b * 16 + i] >> 32);
        }
        fill_box<128>(boxes + b * BOX_BYTES, w);
      }
      store_boxes(boxes, omap, lane < 2 ? (c + g * 128 + lane * 32) * 4 : p.width * 4,
                  p.width * 4, m0);
    }
  } else if (p.out_wide) {
    boxes_free();
#pragma unroll
    for (int b = 0; b < COUNT; ++b) {
      uint32_t w[32];
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        float lo, hi;
        unpack2(v[b][i], lo, hi);
        const __nv_bfloat162 t = __floats2bfloat162_rn(lo, hi);
        w[i] = *reinterpret_cast<const uint32_t*>(&t);
      }
      fill_box<128>(boxes + b * BOX_BYTES, w);
    }
    store_boxes(boxes, omap, lane < COUNT ? (c + lane * 128) * 2 : p.width * 2, p.width * 2, m0);
  } else {
    // rows that are not vectors: 64 columns at a time through the boxes, then row by row,
    // neighbouring lanes neighbouring columns (each thread its own row: 1003 x 777 fp32 spent
    // 20 us here)
    const bool f32 = p.out_dtype == KLT_DT_F32;
    float* t = reinterpret_cast<float*>(boxes);  // [32][64], columns rotated by the row
    const int rows = p.M - m0 < 32 ? p.M - m0 : 32;
#pragma unroll
    for (int g = 0; g < COUNT; ++g) {
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        float lo, hi;
        unpack2(v[g][i], lo, hi);
        t[lane * 64 + ((2 * i + lane) & 63)] = lo;
        t[lane * 64 + ((2 * i + 1 + lane) & 63)] = hi;
      }
      __syncwarp();
      for (int r = 0; r < rows; ++r) {
        const int64_t row = (m0 + r) * p.ld_out;
#pragma unroll
        for (int h = 0; h < 64; h += 32) {
          const int col = c + g * 128 + h + lane;
          const float x = t[r * 64 + ((h + lane + r) & 63)];
          if (col < p.width) {
            if (f32)
              static_cast<float*>(p.out)[row + col] = x;
            else
              static_cast<__nv_bfloat16*>(p.out)[row + col] = __float2bfloat16(x);
          }
        }
      }
      __syncwarp();
    }
  }
}

// grid 2 x pairs, cluster 2; PARTS of K > 1: grid tiles x 2 x PARTS, cluster 2 x PARTS
template <int ACT, int PARTS>
__global__ void __launch_bounds__(THREADS, 1)
    wide_kernel(const __grid_constant__ CUtensorMap tok, const __grid_constant__ CUtensorMap wmap,
                const __grid_constant__ CUtensorMap omap, const LinParams p) {
  extern __shared__ uint8_t smem_raw[];
  Smem sm;
  sm.ring = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  sm.stage = sm.ring + RING_BYTES;
  sm.amax = reinterpret_cast<float*>(sm.stage + OUT_BYTES);
  sm.full = reinterpret_cast<uint64_t*>(sm.stage + OUT_BYTES + AMAX_BYTES);
  sm.done = sm.full + STAGES;
  sm.tempty = sm.done + STAGES;
  sm.drain = sm.tempty + 2;
  sm.ended = sm.drain + 1;
  sm.tmem_holder = reinterpret_cast<uint32_t*>(sm.ended + 1);
  sm.abort_flag = reinterpret_cast<volatile int*>(sm.tmem_holder + 1);
  sm.copies = sm.tmem_holder + 2;
  static_assert((2 * STAGES + 4) * 8 + 12 <= 256, "barrier space");

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // this CTA's half of the pair's tokens and weight rows, the pair's first CTA, its part of K
  const uint32_t crank = cluster_rank(), rank = crank & 1, leader = PARTS > 1 ? crank & ~1u : 0;
  const uint16_t both = static_cast<uint16_t>(3u << leader);
  const int part = PARTS > 1 ? static_cast<int>(crank >> 1) : 0;
  const int k0 = PARTS > 1 ? static_cast<int>(static_cast<int64_t>(p.KB) * part / PARTS) : 0;
  const int k1 =
      PARTS > 1 ? static_cast<int>(static_cast<int64_t>(p.KB) * (part + 1) / PARTS) : p.KB;
  // this pair's tiles: the first one, then steps of the number of pairs
  const int pair = blockIdx.x / (2 * PARTS);
  int tm = pair % p.tiles_m, tn = pair / p.tiles_m;
  auto next_tile = [&]() {
    tm += p.step_m;
    tn += p.step_n;
    if (tm >= p.tiles_m) tm -= p.tiles_m, ++tn;
  };

  if (threadIdx.x == 0) {
    for (int i = 0; i < STAGES; ++i) {
      mbar_init(&sm.full[i], 1);   // first CTA's: bytes of both CTAs
      mbar_init(&sm.done[i], 1);   // each CTA's: the MMAs that read the stage are done, so
                                   // the stage is free and the slot full
    }
    for (int i = 0; i < 2; ++i)
      mbar_init(&sm.tempty[i], 16);  // first CTA's: the epilogue warps of both CTAs
    mbar_init(sm.drain, 1);
    mbar_init(sm.ended, 1);  // first CTA's: the second has issued its last copy
    *sm.abort_flag = 0;
    fence_barrier_init();
    mbar_arrive_expect_tx(sm.ended, 4);
  }
  if (warp == 2) tmem_alloc_pair(sm.tmem_holder, 512);
  tc_fence_before();
  __syncthreads();
  cluster_arrive();  // the other CTA's barriers exist
  cluster_wait();
  tc_fence_after();
  const uint32_t tmem = *sm.tmem_holder;
  pdl_trigger();

  if (warp < 4) {
    regs_dec<56>();
    if (warp == 0 && lane == 0) {
      pdl_wait();
      const uint32_t full0 = map_to_rank(smem_u32(sm.full), leader);
      int it = 0;
      bool ok = true;
      for (; tn < p.tiles_n && ok; next_tile()) {
        const int row0 = tm * 256 + static_cast<int>(rank) * 128;
        const int rb = ACT ? tn + static_cast<int>(rank) * p.up : tn * 2 + static_cast<int>(rank);
        for (int kb = k0; kb < k1; ++kb, ++it) {
          if (p.stall > 0 && it >= p.stall) {
            ok = false;
            break;
          }
          const int st = it % STAGES;
          if (!mbar_wait_spin(&sm.done[st], ((it / STAGES) & 1) ^ 1, sm.abort_flag, p.err,
                              p.timeout)) {
            ok = false;
            break;
          }
          if (rank == 0) mbar_arrive_expect_tx(&sm.full[st], 2 * STAGE_BYTES);
          uint8_t* dst = sm.ring + st * STAGE_BYTES;
          tma_load_2d_pair(dst, &tok, full0 + st * 8, kb * 128, row0);
          tma_load_2d_pair(dst + LIN_TILE_BYTES, &wmap, full0 + st * 8, 0,
                           (rb * p.KB + kb) * LIN_TILE);
        }
      }
      // No copy of the pair is in flight past this point: both CTAs' complete here.  After a wait
      // that ran out the second CTA may have issued up to STAGES that the first has not expected.
      if (rank == 0) {
        int none = 0;
        for (int j = it > STAGES ? it - STAGES : 0; j < it; ++j)
          mbar_wait(&sm.full[j % STAGES], (j / STAGES) & 1, &none, p.err, p.timeout);
        // its waits are bounded and began before this CTA's last ones ended
        if (mbar_wait(sm.ended, 0, &none, p.err, 3 * p.timeout)) {
          const int last = static_cast<int>(*static_cast<volatile uint32_t*>(sm.copies));
          for (; it < last; ++it) {
            mbar_arrive_expect_tx(&sm.full[it % STAGES], STAGE_BYTES);
            mbar_wait(&sm.full[it % STAGES], (it / STAGES) & 1, &none, p.err, p.timeout);
          }
        }
      } else {
        st_async_u32(map_to_rank(smem_u32(sm.copies), leader), it,
                     map_to_rank(smem_u32(sm.ended), leader));
      }
    } else if (warp == 1 && lane == 0 && rank == 0) {
      pdl_wait();  // the bounds of the waits below begin when the tokens are there
      constexpr uint32_t idesc = idesc_make(0, 256, 256);
      int it = 0;
      bool ok = true;
      for (; tn < p.tiles_n && ok; next_tile())
        for (int kb = k0; kb < k1; ++kb, ++it) {
          const int st = it % STAGES, slot = it & 1;
          ok = mbar_wait_spin(&sm.full[st], (it / STAGES) & 1, sm.abort_flag, p.err, p.timeout) &&
               mbar_wait_spin(&sm.tempty[slot], ((it >> 1) & 1) ^ 1, sm.abort_flag, p.err,
                              p.timeout);
          if (!ok) break;
          tc_fence_after();
          const uint32_t base = smem_u32(sm.ring + st * STAGE_BYTES);
          mma4_fp8_pair(tmem + slot * 256, sdesc_sw128(base), sdesc_sw128(base + LIN_TILE_BYTES),
                        idesc);
          tc_commit_pair(&sm.done[st], both);
        }
      tc_commit_pair(sm.drain, both);  // no MMA of the pair runs past this point
      int none = 0;
      mbar_wait(sm.drain, 0, &none, p.err, p.timeout);
    }
    __syncwarp();
    for (int i = 0; PARTS > 1 && i < 2; ++i) {  // the epilogue's two
      cluster_arrive();
      cluster_wait();
    }
  } else {
    regs_inc<224>();
    pdl_wait();
    const int quad = warp & 3, half = (warp - 4) >> 2;
    const int row = quad * 32 + lane;
    uint8_t* boxes = sm.stage + (warp - 4) * BOXES * BOX_BYTES;
    const uint32_t tempty0 = map_to_rank(smem_u32(sm.tempty), leader);
    // this thread's columns of a slot: 64 of the first CTA's weight rows (SwiGLU: gate), 64 of
    // the second's (the matching up rows)
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    const int c0 = half * 64, c1 = 128 + half * 64;
    int it = 0;
    bool ok = true;  // of the whole warp; a warp that gave up still meets the others' barriers
    // the scales of this thread's row and of the two weight tiles, loaded one k-block (at the
    // end of a tile: one tile) ahead
    int xo, wo;
    float x, w0, w1;
    auto first_scales = [&]() {
      const int m = tm * 256 + static_cast<int>(rank) * 128 + row;
      xo = (m < p.M ? m : 0) * p.KB + k0;
      wo = (ACT ? tn : tn * 2) * p.KB + k0;
      x = p.xs[xo];
      w0 = p.ws[wo];
      w1 = p.ws[wo + p.step_ws];
    };
    first_scales();
    while (tn < p.tiles_n) {
      unsigned long long acc[2][32];
#pragma unroll
      for (int i = 0; i < 32; ++i) acc[0][i] = acc[1][i] = 0ull;
      for (int kb = 0; kb < k1 - k0; ++kb, ++it) {
        const int slot = it & 1;
        const float f0 = x * w0, f1 = x * w1;
        const unsigned long long s0 = pack2(f0, f0), s1 = pack2(f1, f1);
        if (kb + 1 < k1 - k0) {
          x = p.xs[xo + kb + 1];
          w0 = p.ws[wo + kb + 1];
          w1 = p.ws[wo + kb + 1 + p.step_ws];
        }
        ok = ok && mbar_wait_spin(&sm.done[it % STAGES], (it / STAGES) & 1, sm.abort_flag, p.err,
                                  p.timeout);
        ok = __all_sync(0xFFFFFFFFu, ok);
        if (!ok) break;
        tc_fence_after();
        // four loads of 32 columns, each started before the products of the one before it;
        // the slot is handed back before the last products
        const uint32_t ta = lane_base + slot * 256;
        uint32_t v[2][32];
        tmem_start_ld32(ta + c0, v[0]);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t* r = v[c & 1];
          tmem_wait_ld32(r);
          if (c < 3) {
            tmem_start_ld32(ta + (c < 1 ? c0 : c1) + (c + 1) % 2 * 32, v[(c + 1) & 1]);
          } else {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(tempty0 + slot * 8);
          }
#pragma unroll
          for (int i = 0; i < 16; ++i)
            fma2(acc[c >> 1][(c & 1) * 16 + i],
                 pack2(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1])),
                 c < 2 ? s0 : s1);
        }
      }
      const int m0 = tm * 256 + static_cast<int>(rank) * 128 + quad * 32, m = m0 + lane, tn0 = tn;
      next_tile();
      if (tn < p.tiles_n) first_scales();
      bool finish = ok;
      if (PARTS > 1) {
        // Every product of the cluster's pairs is in registers once all have arrived, and their
        // stages are free: each warp's rows go to the pair that finishes them (quadrant q: pair
        // q * PARTS / 4), as 32 pieces of 4 columns x 32 rows, and are added in rank order.
        cluster_arrive();
        cluster_wait();
        constexpr int OWNED = 4 / PARTS;
        const int owner = quad / OWNED;
        // where `owner` keeps these rows of part `from` (its own: any)
        auto piece = [&](int from) {
          const int slot = ((from - (from > owner)) * OWNED + quad % OWNED) * 2 + half;
          return smem_u32(sm.ring) + (from == owner ? 0 : slot) * PART_BYTES + lane * 16;
        };
        if (owner != part) {
          const uint32_t dst = map_to_rank(piece(part), owner * 2 + rank);
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            float a, b, c, e;
            unpack2(acc[i >> 4][(i & 15) * 2], a, b);
            unpack2(acc[i >> 4][(i & 15) * 2 + 1], c, e);
            st_cluster_f4(dst + i * 512, a, b, c, e);
          }
          finish = false;
        }
        cluster_arrive();  // the rows are where they are finished
        cluster_wait();
        // (the other warps add up what they find and store nothing)
        uint32_t src[PARTS];
#pragma unroll
        for (int r = 0; r < PARTS; ++r) src[r] = piece(r);
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          unsigned long long* a = &acc[i >> 4][(i & 15) * 2];
          unsigned long long s0 = 0, s1 = 0;
#pragma unroll
          for (int r = 0; r < PARTS; ++r) {
            ulonglong2 v = ld_shared_u64x2(src[r] + i * 512);
            if (r == part) v = make_ulonglong2(a[0], a[1]);
            if (r == 0)
              s0 = v.x, s1 = v.y;
            else
              add2(s0, v.x), add2(s1, v.y);
          }
          a[0] = s0;
          a[1] = s1;
        }
      }
      if (ACT) {
        float big = 0.f;
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          float g0, g1, u0, u1;
          unpack2(acc[0][i], g0, g1);
          unpack2(acc[1][i], u0, u1);
          const float a0 = silu(g0) * u0, a1 = silu(g1) * u1;
          big = max_nan(big, a0, a1);
          acc[0][i] = pack2(a0, a1);
        }
        if (p.out_dtype == KLT_DT_E4M3) {
          // the group's other 64 columns are in the thread of the other half
          sm.amax[half * 128 + row] = big;
          named_bar_sync(1, 256);
          big = max_nan(big, sm.amax[(half ^ 1) * 128 + row]);
          named_bar_sync(1, 256);  // amax is free for the next tile
          float s = group_scale(big);
          if (finish && half == 0 && m < p.M)
            p.out_s[static_cast<int64_t>(m) * (p.width / 128) + tn0] = s;
          const float k = rescale(s), inv = __frcp_rn(s);
          if (k != 1.0f) {
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              float q0, q1;
              unpack2(acc[0][i], q0, q1);
              acc[0][i] = pack2(q0 * k, q1 * k);
            }
          }
          // negated codes: two quotients at a time
          const unsigned long long s2 = pack2(s, s), ninv2 = pack2(-inv, -inv);
          uint32_t w[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            float q[4];
            unpack2(neg_quot_group2(acc[0][2 * j], s2, ninv2), q[0], q[1]);
            unpack2(neg_quot_group2(acc[0][2 * j + 1], s2, ninv2), q[2], q[3]);
            w[j] = (f32x2_to_e4m3x2(q[0], q[1]) | (f32x2_to_e4m3x2(q[2], q[3]) << 16)) ^
                   0x80808080u;
          }
          if (finish && m0 < p.M) {
            const int c = tn0 * 128 + half * 64;
            if (p.out_wide) {
              boxes_free();
              fill_box<64>(boxes, w);
              store_boxes(boxes, &omap, lane == 0 ? c : p.width, p.width, m0);
            } else if (m < p.M) {
              uint8_t* o = static_cast<uint8_t*>(p.out) + static_cast<int64_t>(m) * p.ld_out + c;
#pragma unroll
              for (int j = 0; j < 64; ++j) o[j] = static_cast<uint8_t>(w[j / 4] >> (8 * (j % 4)));
            }
          }
        } else if (finish) {
          store_rows<1>(p, &omap, boxes, m0, tn0 * 128 + half * 64, acc);
        }
      } else if (finish) {
        store_rows<2>(p, &omap, boxes, m0, tn0 * 256 + half * 64, acc);
      }
    }
    tma_store_wait();
    tc_fence_before();
    __syncwarp();
  }
  __syncthreads();
  cluster_arrive();  // nothing of the pair still reads across, and no MMA of it runs
  cluster_wait();
  if (threadIdx.x == 0) {  // nor is a signal of its MMAs to this CTA on its way
    int none = 0;
    mbar_wait(sm.drain, 0, &none, p.err, p.timeout);
  }
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

void config(cudaLaunchConfig_t* cfg, cudaLaunchAttribute attr[2], int clusters, int parts,
            cudaStream_t s) {
  cfg->gridDim = dim3(2 * parts * clusters);
  cfg->blockDim = dim3(THREADS);
  cfg->dynamicSmemBytes = SMEM;
  cfg->stream = s;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2 * parts;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg->attrs = attr;
  cfg->numAttrs = 2;
}

template <int ACT>
cudaError_t launch(const CUtensorMap& tok, const CUtensorMap& wmap, const CUtensorMap& omap,
                   LinParams p, int parts, int num_sms, cudaStream_t s) {
  p.tiles_m = (p.M + 255) / 256;
  p.tiles_n = ACT ? p.width / 128 : (p.NB + 1) / 2;
  p.step_ws = ACT ? p.up * p.KB : p.KB;
  const int64_t tiles = static_cast<int64_t>(p.tiles_m) * p.tiles_n;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  if (parts > 1) {  // one tile per cluster
    if (tiles > 0x7FFFFFF) return cudaErrorInvalidValue;
    p.step_m = 0;
    p.step_n = p.tiles_n;
    config(&cfg, attr, static_cast<int>(tiles), parts, s);
    return cudaLaunchKernelEx(&cfg, wide_kernel<ACT, 2>, tok, wmap, omap, p);
  }
  const int pairs = tiles < num_sms / 2 ? static_cast<int>(tiles) : num_sms / 2;
  p.step_m = pairs % p.tiles_m;
  p.step_n = pairs / p.tiles_m;
  config(&cfg, attr, pairs, 1, s);
  return cudaLaunchKernelEx(&cfg, wide_kernel<ACT, 1>, tok, wmap, omap, p);
}

// max_tiles: lowered to the clusters of PARTS pairs that run at once.
template <int ACT, int PARTS>
bool prepare(int* max_tiles) {
  // setmaxnreg moves registers between the warpgroups: 56 + 2 x 224 = 3 x 168 at launch
  auto k = wide_kernel<ACT, PARTS>;
  cudaFuncAttributes a;
  if (cudaFuncGetAttributes(&a, k) != cudaSuccess || a.numRegs < 168 ||
      cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM) != cudaSuccess)
    return false;
  if (PARTS == 1) return true;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  config(&cfg, attr, 1, PARTS, 0);
  cfg.numAttrs = 1;  // the cluster alone
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, k, &cfg) != cudaSuccess) return false;
  if (n < *max_tiles) *max_tiles = n;
  return true;
}

}  // namespace

bool prepare_linear_wide(int* max_tiles) {
  *max_tiles = 1 << 20;
  return prepare<0, 1>(nullptr) && prepare<1, 1>(nullptr) && prepare<0, 2>(max_tiles) &&
         prepare<1, 2>(max_tiles);
}

cudaError_t launch_linear_wide(const CUtensorMap& tok, const CUtensorMap& wmap,
                               const CUtensorMap& omap, const LinParams& p, bool swiglu,
                               int parts, int num_sms, cudaStream_t s) {
  return swiglu ? launch<1>(tok, wmap, omap, p, parts, num_sms, s)
                : launch<0>(tok, wmap, omap, p, parts, num_sms, s);
}

}  // namespace klt
