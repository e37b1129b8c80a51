// FP8 linear layer, token-major kernel: many tokens (sm_103a).
//
// A pair of CTAs (cta_group::2) computes 256 tokens x 256 weight rows: each CTA holds its own
// 128 tokens and 128 of the 256 weight rows in shared memory, the tensor core reads both
// CTAs' weight tiles, and each CTA's TMEM gets its 128 tokens x 256 outputs.  So a CTA loads
// 32 KB per 128-column k-block where one alone would load 48 KB.  SwiGLU pairs the 128 gate
// rows (first CTA) with the 128 matching up rows (second CTA).
//
// The scales are general fp32 per 128 columns, so every k-block's product is read from TMEM
// and added into registers times xs[m, kb] * ws[rb, kb]: that reading (128 KB per CTA and
// k-block, two 256-column slots in turn), not the multiplication, bounds the kernel.
//
// Persistent: one pair per two SMs, tiles dealt round robin, token tiles fastest (the pairs
// that run together share weight tiles in L2).
#include "klt_linear.cuh"

#include "../../include/klt.h"

namespace klt {
namespace {

constexpr int THREADS = 384;  // warps 0 copies, 1 MMA, 2 TMEM, 3 idle, 4-11 epilogue
constexpr int STAGES = 6;
constexpr int STAGE_BYTES = 2 * LIN_TILE_BYTES;
constexpr int RING_BYTES = STAGES * STAGE_BYTES;
constexpr int SMEM = 1024 + RING_BYTES + 1024 + 256;

struct Smem {
  uint8_t* ring;
  float* amax;  // [2][128]
  uint64_t *full, *empty, *tfull, *tempty, *drain;
  uint32_t* tmem_holder;
  volatile int* abort_flag;
};

// 32 consecutive fp32 columns of this thread's TMEM lane, waited for.
KLT_DEV void tmem_ld32(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
        "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]),
        "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]),
        "=r"(r[31])
      : "r"(taddr)
      : "memory");
}

// Stores 64 consecutive outputs (columns c .. c + 63) of row m.
KLT_DEV void store_row64(const LinParams& p, int64_t m, int c, const float* v) {
  if (p.out_dtype == KLT_DT_F32) {
    float* o = static_cast<float*>(p.out) + m * p.ld_out + c;
    if (p.out_wide && c + 64 <= p.width) {
#pragma unroll
      for (int i = 0; i < 16; ++i)
        reinterpret_cast<float4*>(o)[i] =
            make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
    } else {
#pragma unroll
      for (int i = 0; i < 64; ++i)
        if (c + i < p.width) o[i] = v[i];
    }
  } else {
    __nv_bfloat16* o = static_cast<__nv_bfloat16*>(p.out) + m * p.ld_out + c;
    if (p.out_wide && c + 64 <= p.width) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const __nv_bfloat162 b = __floats2bfloat162_rn(v[8 * i + 2 * j], v[8 * i + 2 * j + 1]);
          w[j] = *reinterpret_cast<const uint32_t*>(&b);
        }
        reinterpret_cast<uint4*>(o)[i] = make_uint4(w[0], w[1], w[2], w[3]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 64; ++i)
        if (c + i < p.width) o[i] = __float2bfloat16(v[i]);
    }
  }
}

// grid 2 x pairs, cluster 2
template <int ACT>
__global__ void __launch_bounds__(THREADS, 1)
    wide_kernel(const __grid_constant__ CUtensorMap tok, const __grid_constant__ CUtensorMap wmap,
                const LinParams p, int tiles_m, int tiles) {
  extern __shared__ uint8_t smem_raw[];
  Smem sm;
  sm.ring = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  sm.amax = reinterpret_cast<float*>(sm.ring + RING_BYTES);
  sm.full = reinterpret_cast<uint64_t*>(sm.ring + RING_BYTES + 1024);
  sm.empty = sm.full + STAGES;
  sm.tfull = sm.empty + STAGES;
  sm.tempty = sm.tfull + 2;
  sm.drain = sm.tempty + 2;
  sm.tmem_holder = reinterpret_cast<uint32_t*>(sm.drain + 1);
  sm.abort_flag = reinterpret_cast<volatile int*>(sm.tmem_holder + 1);
  static_assert((2 * STAGES + 5) * 8 + 8 <= 256, "barrier space");

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;

  if (threadIdx.x == 0) {
    for (int i = 0; i < STAGES; ++i) {
      mbar_init(&sm.full[i], 1);   // first CTA's: bytes of both CTAs
      mbar_init(&sm.empty[i], 1);  // each CTA's: the MMAs that read the stage are done
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.tfull[i], 1);
      mbar_init(&sm.tempty[i], 16);  // first CTA's: the epilogue warps of both CTAs
    }
    mbar_init(sm.drain, 1);
    *sm.abort_flag = 0;
    fence_barrier_init();
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
    regs_dec<72>();
    if (warp == 0 && lane == 0) {
      pdl_wait();
      const uint32_t full0 = map_to_rank(smem_u32(sm.full), 0);
      int it = 0;
      bool ok = true;
      for (int tile = pair; tile < tiles && ok; tile += pairs) {
        const int tm = tile % tiles_m, tn = tile / tiles_m;
        const int row0 = tm * 256 + static_cast<int>(rank) * 128;
        const int rb = ACT ? tn + static_cast<int>(rank) * p.up : tn * 2 + static_cast<int>(rank);
        for (int kb = 0; kb < p.KB; ++kb, ++it) {
          if (p.stall > 0 && it >= p.stall) {
            ok = false;
            break;
          }
          const int st = it % STAGES;
          if (!mbar_wait_spin(&sm.empty[st], ((it / STAGES) & 1) ^ 1, sm.abort_flag, p.err,
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
      // no copy of the pair is in flight past this point (both CTAs' complete here)
      if (rank == 0) {
        int none = 0;
        for (int j = it > STAGES ? it - STAGES : 0; j < it; ++j)
          mbar_wait(&sm.full[j % STAGES], (j / STAGES) & 1, &none, p.err, p.timeout);
      }
    } else if (warp == 1 && lane == 0 && rank == 0) {
      constexpr uint32_t idesc = idesc_make(0, 256, 256);
      int it = 0;
      bool ok = true;
      for (int tile = pair; tile < tiles && ok; tile += pairs) {
        for (int kb = 0; kb < p.KB; ++kb, ++it) {
          const int st = it % STAGES, slot = it & 1;
          if (!mbar_wait_spin(&sm.tempty[slot], ((it >> 1) & 1) ^ 1, sm.abort_flag, p.err,
                              p.timeout) ||
              !mbar_wait_spin(&sm.full[st], (it / STAGES) & 1, sm.abort_flag, p.err,
                              p.timeout)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t base = smem_u32(sm.ring + st * STAGE_BYTES);
          mma4_fp8_pair(tmem + slot * 256, sdesc_sw128(base), sdesc_sw128(base + LIN_TILE_BYTES),
                        idesc);
          tc_commit_pair(&sm.empty[st]);
          tc_commit_pair(&sm.tfull[slot]);
        }
      }
      tc_commit_pair(sm.drain);  // no MMA of the pair runs past this point
      int none = 0;
      mbar_wait(sm.drain, 0, &none, p.err, p.timeout);
    }
    __syncwarp();
  } else {
    regs_inc<216>();
    pdl_wait();
    const int quad = warp & 3, half = (warp - 4) >> 2;
    const int row = quad * 32 + lane;
    const uint32_t tempty0 = map_to_rank(smem_u32(sm.tempty), 0);
    // this thread's columns of a slot: 128 neighbouring ones, or 64 gate and the 64 matching
    // up columns
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    const int c0 = ACT ? half * 64 : half * 128;
    const int c1 = ACT ? 128 + half * 64 : half * 128 + 64;
    int it = 0;
    bool ok = true;  // of the whole warp; a warp that gave up still meets the others' barriers
    for (int tile = pair; tile < tiles; tile += pairs) {
      const int tm = tile % tiles_m, tn = tile / tiles_m;
      const int64_t m = static_cast<int64_t>(tm) * 256 + rank * 128 + row;
      const float* xs = p.xs + (m < p.M ? m : 0) * p.KB;
      const int rb0 = ACT ? tn : tn * 2 + half, rb1 = ACT ? tn + p.up : rb0;
      const float* ws0 = p.ws + static_cast<int64_t>(rb0 < p.NB ? rb0 : 0) * p.KB;
      const float* ws1 = p.ws + static_cast<int64_t>(rb1 < p.NB ? rb1 : 0) * p.KB;
      unsigned long long acc[2][32];
#pragma unroll
      for (int i = 0; i < 32; ++i) acc[0][i] = acc[1][i] = 0ull;
      float x = xs[0], w0 = ws0[0], w1 = ws1[0];
      for (int kb = 0; kb < p.KB; ++kb, ++it) {
        const int slot = it & 1;
        const float f0 = x * w0, f1 = x * w1;
        const unsigned long long s0 = pack2(f0, f0), s1 = pack2(f1, f1);
        if (kb + 1 < p.KB) {
          x = xs[kb + 1];
          w0 = ws0[kb + 1];
          w1 = ws1[kb + 1];
        }
        ok = ok && mbar_wait_spin(&sm.tfull[slot], (it >> 1) & 1, sm.abort_flag, p.err, p.timeout);
        ok = __all_sync(0xFFFFFFFFu, ok);
        if (!ok) break;
        tc_fence_after();
        const uint32_t ta = lane_base + slot * 256;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int c = 0; c < 64; c += 32) {
            uint32_t v[32];
            tmem_ld32(ta + (h ? c1 : c0) + c, v);
#pragma unroll
            for (int j = 0; j < 16; ++j)
              fma2(acc[h][c / 2 + j], pack2(__uint_as_float(v[2 * j]), __uint_as_float(v[2 * j + 1])),
                   h ? s1 : s0);
          }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(tempty0 + slot * 8);
      }
      if (ACT) {
        float v[64];
        uint32_t big = 0;
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          float g0, g1, u0, u1;
          unpack2(acc[0][i], g0, g1);
          unpack2(acc[1][i], u0, u1);
          v[2 * i] = silu_fast(g0) * u0;
          v[2 * i + 1] = silu_fast(g1) * u1;
          big = max(big, max(__float_as_uint(v[2 * i]) & 0x7FFFFFFFu,
                             __float_as_uint(v[2 * i + 1]) & 0x7FFFFFFFu));
        }
        if (p.out_dtype == KLT_DT_E4M3) {
          // the group's other 64 columns are in the thread of the other half
          sm.amax[half * 128 + row] = __uint_as_float(big);
          named_bar_sync(1, 256);
          big = max(big, __float_as_uint(sm.amax[(half ^ 1) * 128 + row]));
          const float s = group_scale(big);
          const float inv = 1.0f / s;
          const bool fast = quot_fast(s);
          if (ok && m < p.M) {
            uint8_t* o = static_cast<uint8_t*>(p.out) + m * p.ld_out + tn * 128 + half * 64;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint32_t w[4];
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                float q[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) q[e] = quot_group(v[16 * i + 4 * j + e], s, inv, fast);
                w[j] = f32x2_to_e4m3x2(q[0], q[1]) | (f32x2_to_e4m3x2(q[2], q[3]) << 16);
              }
              if (p.out_wide) {
                reinterpret_cast<uint4*>(o)[i] = make_uint4(w[0], w[1], w[2], w[3]);
              } else {
#pragma unroll
                for (int j = 0; j < 16; ++j)
                  o[16 * i + j] = static_cast<uint8_t>(w[j / 4] >> (8 * (j % 4)));
              }
            }
            if (half == 0) p.out_s[m * (p.width / 128) + tn] = s;
          }
          named_bar_sync(1, 256);  // amax is free for the next tile
        } else if (ok && m < p.M) {
          store_row64(p, m, tn * 128 + half * 64, v);
        }
      } else if (ok && m < p.M) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float v[64];
#pragma unroll
          for (int i = 0; i < 32; ++i) unpack2(acc[h][i], v[2 * i], v[2 * i + 1]);
          store_row64(p, m, tn * 256 + half * 128 + h * 64, v);
        }
      }
    }
    tc_fence_before();
    __syncwarp();
  }
  __syncthreads();
  cluster_arrive();  // nothing of the pair still reads or signals across
  cluster_wait();
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

template <int ACT>
cudaError_t launch(const CUtensorMap& tok, const CUtensorMap& wmap, const LinParams& p,
                   int num_sms, cudaStream_t s) {
  cudaError_t e = cudaFuncSetAttribute(wide_kernel<ACT>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
  if (e != cudaSuccess) return e;
  const int tiles_m = (p.M + 255) / 256;
  const int tiles = tiles_m * (ACT ? p.width / 128 : (p.NB + 1) / 2);
  const int pairs = tiles < num_sms / 2 ? tiles : num_sms / 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * pairs);
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = SMEM;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 2;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, wide_kernel<ACT>, tok, wmap, p, tiles_m, tiles);
}

}  // namespace

bool linear_wide_regs_ok() {
  // setmaxnreg moves registers between the warpgroups: 72 + 2 x 216 = 3 x 168 at launch
  cudaFuncAttributes a;
  return cudaFuncGetAttributes(&a, wide_kernel<0>) == cudaSuccess && a.numRegs >= 168 &&
         cudaFuncGetAttributes(&a, wide_kernel<1>) == cudaSuccess && a.numRegs >= 168;
}

cudaError_t launch_linear_wide(const CUtensorMap& tok, const CUtensorMap& wmap,
                               const LinParams& p, bool swiglu, int num_sms, cudaStream_t s) {
  return swiglu ? launch<1>(tok, wmap, p, num_sms, s) : launch<0>(tok, wmap, p, num_sms, s);
}

}  // namespace klt
