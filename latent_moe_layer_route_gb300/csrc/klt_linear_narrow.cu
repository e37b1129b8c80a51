// FP8 linear layer, feature-major kernel: few tokens (sm_103a).
//
// A CTA multiplies 128 weight rows (SwiGLU: 128 gate and the 128 matching up rows) by one
// tile of BN tokens over a part of K; the CTAs of a cluster share K and add their parts
// through distributed shared memory in rank order, so there is no workspace, no atomic and
// the result does not depend on timing.  At these sizes the weight stream is the cost: the
// weights are the MMA's M side (128 rows per instruction however few the tokens are), every
// tile is one contiguous bulk copy, and the copies of the first stages start before the
// wait for the kernel that writes the activations.
//
// The scales are general fp32 per 128 columns, so each k-block's product is read from TMEM
// and added into registers times xs[t, kb] * ws[rb, kb] (staged in shared memory).
#include "klt_linear.cuh"

#include "../../include/klt.h"

namespace klt {
namespace {

constexpr int THREADS = 192;  // warps 0-3 epilogue (one per TMEM quadrant), 4 copies, 5 MMA
constexpr int SCALE_KB = 16;  // k-blocks whose scales are staged at once

template <int BN, int ACT>
struct Narrow {
  static constexpr int AT = ACT ? 2 : 1;  // weight tiles per k-block
  static constexpr int STAGE_BYTES = AT * LIN_TILE_BYTES + BN * 128;
  // the ring also holds the CTA's fp32 partial result once the products are done
  static constexpr int PART_BYTES = AT * BN * 128 * 4;
  static constexpr int STAGES = ACT && BN < 64 ? 3 : 4;
  static constexpr int RING_BYTES =
      STAGES * STAGE_BYTES > PART_BYTES ? STAGES * STAGE_BYTES : PART_BYTES;
  static constexpr int SLOTS = BN >= 128 ? 2 : 4;
  static constexpr int SLOT_COLS = AT * BN;
  static constexpr int TMEM_COLS = SLOTS * SLOT_COLS;  // a power of two, 64 .. 512
  static constexpr int SCALE_BYTES = AT * SCALE_KB * BN * 4;
  static constexpr int SMEM = 1024 + RING_BYTES + SCALE_BYTES + 256;
};

// Writes four neighbouring outputs (columns c .. c+3) of row m.
KLT_DEV void store4(const LinParams& p, int64_t m, int c, float4 v) {
  if (p.out_dtype == KLT_DT_F32) {
    float* o = static_cast<float*>(p.out) + m * p.ld_out + c;
    if (p.out_wide && c + 4 <= p.width) {
      *reinterpret_cast<float4*>(o) = v;
    } else {
      if (c < p.width) o[0] = v.x;
      if (c + 1 < p.width) o[1] = v.y;
      if (c + 2 < p.width) o[2] = v.z;
      if (c + 3 < p.width) o[3] = v.w;
    }
  } else {
    __nv_bfloat16* o = static_cast<__nv_bfloat16*>(p.out) + m * p.ld_out + c;
    if (p.out_wide && c + 4 <= p.width) {
      const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y);
      const __nv_bfloat162 b = __floats2bfloat162_rn(v.z, v.w);
      *reinterpret_cast<uint2*>(o) = make_uint2(*reinterpret_cast<const uint32_t*>(&a),
                                                *reinterpret_cast<const uint32_t*>(&b));
    } else {
      if (c < p.width) o[0] = __float2bfloat16(v.x);
      if (c + 1 < p.width) o[1] = __float2bfloat16(v.y);
      if (c + 2 < p.width) o[2] = __float2bfloat16(v.z);
      if (c + 3 < p.width) o[3] = __float2bfloat16(v.w);
    }
  }
}

// grid (split, token tiles, row blocks), cluster (split, 1, 1)
template <int BN, int ACT>
__global__ void __launch_bounds__(THREADS)
    narrow_kernel(const __grid_constant__ CUtensorMap tok, const LinParams p) {
  using C = Narrow<BN, ACT>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  float* scales = reinterpret_cast<float*>(ring + C::RING_BYTES);  // [AT][SCALE_KB][BN]
  uint64_t* bars = reinterpret_cast<uint64_t*>(ring + C::RING_BYTES + C::SCALE_BYTES);
  uint64_t* full = bars;
  uint64_t* empty = full + C::STAGES;
  uint64_t* tfull = empty + C::STAGES;
  uint64_t* tempty = tfull + C::SLOTS;
  uint64_t* drain = tempty + C::SLOTS;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
  static_assert((2 * C::STAGES + 2 * C::SLOTS + 1) * 8 + 8 <= 256, "barrier space");

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int split = gridDim.x, rank = blockIdx.x;
  const int t0 = blockIdx.y * BN, rb = blockIdx.z;
  const int k0 = static_cast<int>(static_cast<int64_t>(p.KB) * rank / split);
  const int nk = static_cast<int>(static_cast<int64_t>(p.KB) * (rank + 1) / split) - k0;

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::STAGES; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < C::SLOTS; ++i) {
      mbar_init(&tfull[i], 1);
      mbar_init(&tempty[i], 4);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 5) {
    tmem_alloc(tmem_holder, C::TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  pdl_trigger();  // this CTA holds its TMEM: a dependent's CTAs cannot take it away

  float acc[C::AT][BN];
#pragma unroll
  for (int a = 0; a < C::AT; ++a)
#pragma unroll
    for (int t = 0; t < BN; ++t) acc[a][t] = 0.f;

  if (warp == 4) {
    if (lane == 0) {
      const uint64_t pol = gridDim.y > 1 ? policy_evict_normal() : policy_evict_first();
      const uint64_t keep = policy_evict_normal();
      const int n = p.stall > 0 && p.stall < nk ? p.stall : nk;
      auto weights = [&](int i, int st) {
        mbar_arrive_expect_tx(&full[st], C::STAGE_BYTES);
#pragma unroll
        for (int a = 0; a < C::AT; ++a)
          bulk_load(ring + st * C::STAGE_BYTES + a * LIN_TILE_BYTES,
                    p.w + (static_cast<int64_t>(rb + a * p.up) * p.KB + k0 + i) * LIN_TILE_BYTES,
                    LIN_TILE_BYTES, &full[st], pol);
      };
      auto tokens = [&](int i, int st) {
        tma_load_2d(ring + st * C::STAGE_BYTES + C::AT * LIN_TILE_BYTES, &tok, &full[st],
                    (k0 + i) * 128, t0, keep);
      };
      // the weights are nobody's output: their first copies do not wait for the launch before
      const int pre = n < C::STAGES ? n : C::STAGES;
      for (int i = 0; i < pre; ++i) weights(i, i);
      pdl_wait();
      for (int i = 0; i < pre; ++i) tokens(i, i);
      int st = pre % C::STAGES, ph = pre / C::STAGES, i = pre;
      for (; i < n; ++i) {
        if (!mbar_wait_spin(&empty[st], (ph & 1) ^ 1, abort_flag, p.err, p.timeout)) break;
        weights(i, st);
        tokens(i, st);
        if (++st == C::STAGES) st = 0, ++ph;
      }
      // no copy of this CTA is in flight past this point
      int none = 0;
      for (int j = i > C::STAGES ? i - C::STAGES : 0; j < i; ++j)
        mbar_wait(&full[j % C::STAGES], (j / C::STAGES) & 1, &none, p.err, p.timeout);
    }
    __syncwarp();
  } else if (warp == 5) {
    if (lane == 0) {
      constexpr uint32_t idesc = idesc_make(0, 128, BN);
      int i = 0;
      for (; i < nk; ++i) {
        const int st = i % C::STAGES, slot = i % C::SLOTS;
        if (!mbar_wait_spin(&tempty[slot], ((i / C::SLOTS) & 1) ^ 1, abort_flag, p.err,
                            p.timeout) ||
            !mbar_wait_spin(&full[st], (i / C::STAGES) & 1, abort_flag, p.err, p.timeout))
          break;
        tc_fence_after();
        const uint32_t base = smem_u32(ring + st * C::STAGE_BYTES);
        const uint64_t db = sdesc_sw128(base + C::AT * LIN_TILE_BYTES);
#pragma unroll
        for (int a = 0; a < C::AT; ++a)
          mma4_fp8(tmem + slot * C::SLOT_COLS + a * BN, sdesc_sw128(base + a * LIN_TILE_BYTES),
                   db, idesc, 0);
        tc_commit(&empty[st]);
        tc_commit(&tfull[slot]);
      }
      tc_commit(drain);  // no MMA of this CTA runs past this point
      int none = 0;
      mbar_wait(drain, 0, &none, p.err, p.timeout);
    }
    __syncwarp();
  } else {
    pdl_wait();
    const int row = warp * 32 + lane;
    bool ok = true;  // of the whole warp; a warp that gave up still meets the others' barriers
    for (int i = 0; i < nk; ++i) {
      if (i % SCALE_KB == 0) {
        // xs[t, kb] * ws[rb, kb] of the next k-blocks, once per CTA
        const int cnt = nk - i < SCALE_KB ? nk - i : SCALE_KB;
        named_bar_sync(1, 128);
        for (int e = row; e < BN * SCALE_KB; e += 128) {
          const int t = e / SCALE_KB, kb = e % SCALE_KB;
          if (kb < cnt) {
            const int64_t m = t0 + t;
            const float x = m < p.M ? p.xs[m * p.KB + k0 + i + kb] : 0.f;
#pragma unroll
            for (int a = 0; a < C::AT; ++a)
              scales[(a * SCALE_KB + kb) * BN + t] =
                  x * p.ws[static_cast<int64_t>(rb + a * p.up) * p.KB + k0 + i + kb];
          }
        }
        named_bar_sync(1, 128);
      }
      const int slot = i % C::SLOTS;
      ok = ok && mbar_wait_spin(&tfull[slot], (i / C::SLOTS) & 1, abort_flag, p.err, p.timeout);
      ok = __all_sync(0xFFFFFFFFu, ok);
      if (!ok) continue;
      tc_fence_after();
      const uint32_t ta = tmem + (static_cast<uint32_t>(warp * 32) << 16) + slot * C::SLOT_COLS;
      const float* sc = scales + (i % SCALE_KB) * BN;
#pragma unroll
      for (int a = 0; a < C::AT; ++a)
#pragma unroll
        for (int c = 0; c < BN; c += 16) {
          float v[16];
          tmem_ld16(ta + a * BN + c, v);
#pragma unroll
          for (int j = 0; j < 16; ++j)
            acc[a][c + j] = fmaf(v[j], sc[a * SCALE_KB * BN + c + j], acc[a][c + j]);
        }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&tempty[slot]);
    }
    // every product of this CTA is in registers (the last slot's barrier follows all MMAs),
    // so the ring is free for the partial result, [a][token][row]
    if (ok) {
      float* part = reinterpret_cast<float*>(ring);
#pragma unroll
      for (int a = 0; a < C::AT; ++a)
#pragma unroll
        for (int t = 0; t < BN; ++t)
          if (t0 + t < p.M) part[(a * BN + t) * 128 + row] = acc[a][t];
    }
  }

  if (split > 1) {
    cluster_arrive();
    cluster_wait();
  } else {
    __syncthreads();
  }
  if (warp < 4 && !*abort_flag) {
    // tokens rank, rank + split, ... of the tile are this CTA's to finish: one warp per
    // token, four rows per lane, the parts added in rank order
    const int tokens = p.M - t0 < BN ? p.M - t0 : BN;
    const uint32_t part = smem_u32(ring) + lane * 16;
    for (int t = rank + warp * split; t < tokens; t += 4 * split) {
      float4 sum[C::AT];
#pragma unroll
      for (int a = 0; a < C::AT; ++a) {
        float4 v[8];
#pragma unroll
        for (int r = 0; r < 8; ++r)
          if (r < split) v[r] = ld_cluster_f4(map_to_rank(part + (a * BN + t) * 512, r));
        sum[a] = v[0];
#pragma unroll
        for (int r = 1; r < 8; ++r)
          if (r < split) {
            sum[a].x += v[r].x;
            sum[a].y += v[r].y;
            sum[a].z += v[r].z;
            sum[a].w += v[r].w;
          }
      }
      const int64_t m = t0 + t;
      const int c = rb * 128 + lane * 4;
      if (ACT) {
        const float4 g = sum[0], u = sum[C::AT - 1];
        const float4 v = make_float4(silu_fast(g.x) * u.x, silu_fast(g.y) * u.y,
                                     silu_fast(g.z) * u.z, silu_fast(g.w) * u.w);
        if (p.out_dtype == KLT_DT_E4M3) {
          // the warp holds one group of 128 columns
          float amax = max_nan(max_nan(v.x, v.y), max_nan(v.z, v.w));
#pragma unroll
          for (int o = 16; o; o >>= 1)
            amax = max_nan(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
          float s = group_scale(amax);
          if (lane == 0) p.out_s[m * (p.width / 128) + rb] = s;
          const float k = rescale(s), inv = __frcp_rn(s);
          const float q0 = quot_group(v.x * k, s, inv), q1 = quot_group(v.y * k, s, inv);
          const float q2 = quot_group(v.z * k, s, inv), q3 = quot_group(v.w * k, s, inv);
          const uint32_t codes = f32x2_to_e4m3x2(q0, q1) | (f32x2_to_e4m3x2(q2, q3) << 16);
          uint8_t* o = static_cast<uint8_t*>(p.out) + m * p.ld_out + c;
          if (p.out_wide) {
            *reinterpret_cast<uint32_t*>(o) = codes;
          } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) o[j] = static_cast<uint8_t>(codes >> (8 * j));
          }
        } else {
          store4(p, m, c, v);
        }
      } else {
        store4(p, m, c, sum[0]);
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  if (split > 1) {  // the other CTAs have read this one's part
    cluster_arrive();
    cluster_wait();
  } else {
    __syncthreads();
  }
  if (warp == 5) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

template <int BN, int ACT>
bool prepare() {
  using C = Narrow<BN, ACT>;
  static_assert(C::SMEM <= 232448, "shared memory of a block");
  return cudaFuncSetAttribute(narrow_kernel<BN, ACT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              C::SMEM) == cudaSuccess;
}

template <int BN, int ACT>
cudaError_t launch(const CUtensorMap& tok, const LinParams& p, int split, cudaStream_t s) {
  using C = Narrow<BN, ACT>;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(split, (p.M + BN - 1) / BN, ACT ? p.width / 128 : p.NB);
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = split;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, narrow_kernel<BN, ACT>, tok, p);
}

}  // namespace

bool prepare_linear_narrow() {
  return prepare<16, 0>() && prepare<32, 0>() && prepare<64, 0>() && prepare<128, 0>() &&
         prepare<16, 1>() && prepare<32, 1>() && prepare<64, 1>();
}

cudaError_t launch_linear_narrow(const CUtensorMap& tok, const LinParams& p, int bn, int split,
                                 bool swiglu, cudaStream_t s) {
  switch (bn) {
    case 16: return swiglu ? launch<16, 1>(tok, p, split, s) : launch<16, 0>(tok, p, split, s);
    case 32: return swiglu ? launch<32, 1>(tok, p, split, s) : launch<32, 0>(tok, p, split, s);
    case 64: return swiglu ? launch<64, 1>(tok, p, split, s) : launch<64, 0>(tok, p, split, s);
    case 128:  // SwiGLU would need 256 sums per thread
      return swiglu ? cudaErrorInvalidValue : launch<128, 0>(tok, p, split, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace klt
