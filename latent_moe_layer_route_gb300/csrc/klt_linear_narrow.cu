// FP8 linear layer, feature-major kernel: few tokens (sm_103a).
//
// A CTA multiplies 128 weight rows (SwiGLU: 128 gate and the 128 matching up rows) by one
// tile of BN tokens over a part of K; the CTAs of a cluster share K, store their parts into the
// shared memory of the CTA that finishes a token (asynchronous stores that complete on its
// barrier), and that one adds them in rank order, so there is no workspace, no atomic and the
// result does not depend on timing.  At these sizes the weight stream is the cost: the
// weights are the MMA's M side (128 rows per instruction however few the tokens are), every
// tile is one contiguous bulk copy, and the copies of the first stages start before the
// wait for the kernel that writes the activations.
//
// The scales are general fp32 per 128 columns, so each k-block's product is read from TMEM
// and added into registers times xs[t, kb] * ws[rb, kb] (staged in shared memory).  Eight warps
// do so from 32 columns on: with four, 128 columns took 1600 cycles per k-block, six times
// their multiplication.
//
// Few tokens are bound by latency: the hand-off between launches, the first copies, the joining of
// the parts, and multiplications that take 93 cycles each however few the tokens are.  1 x 7168 x
// 2048 4.8 us (16 of them in turn, 0.8 us), 16 x 4096 x 7168 SwiGLU to codes 7.3 us (56 in turn, 2.6
// us; 4.0 TB/s), 128 x 7168 x 7168 16.3 us (112 of the SMs, each with the token tile of its own).
#include "klt_linear.cuh"

#include "../../include/klt.h"

namespace klt {
namespace {

template <int BN, int ACT>
struct Narrow {
  static constexpr int AT = ACT ? 2 : 1;  // weight tiles per k-block
  static constexpr int STAGE_BYTES = AT * LIN_TILE_BYTES + BN * 128;
  static constexpr int SLOTS = 4;  // products on their way from the MMA to the registers
  static constexpr int COLS = AT * BN;  // columns of a slot: token t of tile a at a * BN + t
  static constexpr int TMEM_COLS = SLOTS * COLS;  // a power of two, 64 .. 512
  // warps: epilogue (two per TMEM quadrant, half of the columns each, from 32 columns on),
  // then copies, then MMA
  static constexpr int EPI = COLS >= 32 ? 8 : 4;
  static constexpr bool ALONE = COLS == 128 && BN >= 64;  // one CTA per SM
  static constexpr int THREADS = (EPI + 2) * 32;
  static constexpr int WC = COLS * 4 / EPI;         // columns of a warp
  static constexpr int CHUNK = WC >= 32 ? 32 : 16;  // loaded at a time
  // as many stages as leave room for two CTAs per SM, so that the next launch's CTAs are
  // resident and copy weights while this one's finish; the largest tiles run alone
  static constexpr int STAGES = ACT ? (BN < 64 ? 2 : 3) : (BN == 64 ? 3 : 4);
  static constexpr int RING_BYTES = STAGES * STAGE_BYTES;
  static constexpr int PART_BYTES = COLS * 128 * 4;  // all parts of the tokens finished here
  static constexpr int SCALE_KB = BN == 128 ? 32 : 16;  // k-blocks of scales staged at once
  static constexpr int SCALE_LD = COLS + 4;             // floats per k-block of scales
  static constexpr int SCALE_BYTES = SCALE_KB * SCALE_LD * 4;
  static constexpr int SMEM = 1024 + RING_BYTES + PART_BYTES + SCALE_BYTES + 256;
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
__global__ void __launch_bounds__(Narrow<BN, ACT>::THREADS)
    narrow_kernel(const __grid_constant__ CUtensorMap tok, const LinParams p) {
  using C = Narrow<BN, ACT>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  // [tokens finished here][weight tile][rank][128 rows]
  float* parts = reinterpret_cast<float*>(ring + C::RING_BYTES);
  float* scales = reinterpret_cast<float*>(ring + C::RING_BYTES + C::PART_BYTES);
  uint64_t* bars =
      reinterpret_cast<uint64_t*>(ring + C::RING_BYTES + C::PART_BYTES + C::SCALE_BYTES);
  uint64_t* full = bars;
  uint64_t* empty = full + C::STAGES;
  uint64_t* tfull = empty + C::STAGES;
  uint64_t* tempty = tfull + C::SLOTS;
  uint64_t* drain = tempty + C::SLOTS;
  uint64_t* got = drain + 1;  // the other CTAs' parts have arrived
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(got + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
  static_assert((2 * C::STAGES + 2 * C::SLOTS + 2) * 8 + 8 <= 256, "barrier space");

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int split = gridDim.x, rank = blockIdx.x;
  const int t0 = blockIdx.y * BN, rb = blockIdx.z;
  const int k0 = static_cast<int>(static_cast<int64_t>(p.KB) * rank / split);
  const int nk = static_cast<int>(static_cast<int64_t>(p.KB) * (rank + 1) / split) - k0;
  // tokens rank, rank + split, ... of the tile are this CTA's to finish
  const int tokens = p.M - t0 < BN ? p.M - t0 : BN;
  const int log_split = __ffs(split) - 1;
  const int mine = (tokens - rank + split - 1) >> log_split;

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::STAGES; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < C::SLOTS; ++i) {
      mbar_init(&tfull[i], 1);
      mbar_init(&tempty[i], C::EPI);
    }
    mbar_init(drain, 1);
    mbar_init(got, 1);
    *abort_flag = 0;
    fence_barrier_init();
    mbar_arrive_expect_tx(got, mine * C::AT * (split - 1) * 512);
  }
  if (warp == C::EPI + 1) {
    tmem_alloc(tmem_holder, C::TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  cluster_arrive_relaxed();  // this CTA's barriers exist: waited for before storing to another
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  pdl_trigger();  // this CTA holds its TMEM: a dependent's CTAs cannot take it away

  if (warp == C::EPI) {
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
      // The weights are nobody's output: their first copies do not wait for the launch before,
      // and where that one's CTAs leave room for these, the others are already on their way to
      // L2 (16 x 4096 x 7168 SwiGLU 8.4 -> 7.2 us).
      const int pre = n < C::STAGES ? n : C::STAGES;
      for (int i = 0; i < pre; ++i) weights(i, i);
      const int ahead = n - pre < 32 ? n - pre : 32;
      if (!C::ALONE && blockIdx.y == 0 && ahead > 0)
        for (int a = 0; a < C::AT; ++a)
          bulk_prefetch_l2(
              p.w + (static_cast<int64_t>(rb + a * p.up) * p.KB + k0 + pre) * LIN_TILE_BYTES,
              ahead * LIN_TILE_BYTES);
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
  } else if (warp == C::EPI + 1) {
    if (lane == 0) {
      pdl_wait();  // the bounds of the waits below begin when the tokens are there
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
          mma4_fp8(tmem + slot * C::COLS + a * BN, sdesc_sw128(base + a * LIN_TILE_BYTES),
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
    const int row = (warp & 3) * 32 + lane, col = (warp >> 2) * C::WC;
    // scales of the k-blocks from i on: neighbouring lanes = k-blocks.  Those of the weights
    // are nobody's output and do not wait for the launch before
    constexpr int TW = 32 / C::SCALE_KB;  // tokens of a warp at a time
    const int skb = lane % C::SCALE_KB, st0 = warp * TW + lane / C::SCALE_KB;
    float w[C::AT];
    auto weight_scales = [&](int i) {
#pragma unroll
      for (int a = 0; a < C::AT; ++a)
        w[a] = i + skb < nk ? p.ws[static_cast<int64_t>(rb + a * p.up) * p.KB + k0 + i + skb]
                            : 0.f;
    };
    auto stage_scales = [&](int i) {
      constexpr int STEP = C::EPI * TW;
      float x[BN / STEP];
#pragma unroll
      for (int j = 0; j < BN / STEP; ++j) {
        const int t = st0 + j * STEP;
        x[j] = i + skb < nk && t < tokens
                   ? p.xs[static_cast<int64_t>(t0 + t) * p.KB + k0 + i + skb]
                   : 0.f;
      }
#pragma unroll
      for (int j = 0; j < BN / STEP; ++j)
#pragma unroll
        for (int a = 0; a < C::AT; ++a)
          scales[skb * C::SCALE_LD + a * BN + st0 + j * STEP] = x[j] * w[a];
    };
    weight_scales(0);
    pdl_wait();
    stage_scales(0);
    named_bar_sync(1, C::EPI * 32);
    unsigned long long acc[C::WC / 2];
#pragma unroll
    for (int i = 0; i < C::WC / 2; ++i) acc[i] = 0ull;
    bool ok = true;  // of the whole warp; a warp that gave up still meets the others' barriers
    for (int i = 0; i < nk; ++i) {
      if (i > 0 && i % C::SCALE_KB == 0) {
        weight_scales(i);
        named_bar_sync(1, C::EPI * 32);
        stage_scales(i);
        named_bar_sync(1, C::EPI * 32);
      }
      const int slot = i % C::SLOTS;
      ok = ok && mbar_wait_spin(&tfull[slot], (i / C::SLOTS) & 1, abort_flag, p.err, p.timeout);
      ok = __all_sync(0xFFFFFFFFu, ok);
      if (!ok) continue;
      tc_fence_after();
      const uint32_t ta =
          tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + slot * C::COLS + col;
      const ulonglong2* sc =
          reinterpret_cast<const ulonglong2*>(scales + (i % C::SCALE_KB) * C::SCALE_LD + col);
      // each load is started before the products of the one before it
      uint32_t v[2][C::CHUNK];
      auto start = [&](int c) {
        if (C::CHUNK == 32)
          tmem_start_ld32(ta + c * 32, v[c & 1]);
        else
          tmem_start_ld16(ta + c * 16, v[c & 1]);
      };
      start(0);
#pragma unroll
      for (int c = 0; c < C::WC / C::CHUNK; ++c) {
        uint32_t* r = v[c & 1];
        if (C::CHUNK == 32)
          tmem_wait_ld32(r);
        else
          tmem_wait_ld16(r);
        if (c + 1 < C::WC / C::CHUNK) {
          start(c + 1);
        } else {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&tempty[slot]);
        }
#pragma unroll
        for (int e = 0; e < C::CHUNK / 4; ++e) {
          const ulonglong2 f = sc[c * (C::CHUNK / 4) + e];
          unsigned long long* a = acc + c * (C::CHUNK / 2) + 2 * e;
          fma2(a[0], pack2(__uint_as_float(r[4 * e]), __uint_as_float(r[4 * e + 1])), f.x);
          fma2(a[1], pack2(__uint_as_float(r[4 * e + 2]), __uint_as_float(r[4 * e + 3])), f.y);
        }
      }
    }
    // This CTA's part to the CTAs that finish its tokens (after a wait that ran out too: they
    // count on it).  Four columns of four neighbouring lanes are transposed, so that a lane
    // stores four neighbouring rows of one token.
    cluster_wait();
    const uint32_t bar = smem_u32(got);
    const bool odd = lane & 1, high = lane & 2;
#pragma unroll
    for (int i = 0; i < C::WC; i += 4) {
      float v0, v1, v2, v3;
      unpack2(acc[i / 2], v0, v1);
      unpack2(acc[i / 2 + 1], v2, v3);
      const float a = __shfl_xor_sync(0xFFFFFFFFu, odd ? v0 : v1, 1);
      const float b = __shfl_xor_sync(0xFFFFFFFFu, odd ? v2 : v3, 1);
      (odd ? v0 : v1) = a;
      (odd ? v2 : v3) = b;
      const float c = __shfl_xor_sync(0xFFFFFFFFu, high ? v0 : v2, 2);
      const float e = __shfl_xor_sync(0xFFFFFFFFu, high ? v1 : v3, 2);
      (high ? v0 : v2) = c;
      (high ? v1 : v3) = e;
      const int t = (col + i) % BN + (lane & 3), tile = (col + i) / BN;
      if (t < tokens) {
        const int owner = t & (split - 1);
        const int part = (((t >> log_split) * C::AT + tile) << log_split) + rank;
        float* dst = parts + part * 128 + (row & ~31) + (lane >> 2) * 4;
        if (owner == rank)
          *reinterpret_cast<float4*>(dst) = make_float4(v0, v1, v2, v3);
        else
          st_async_f4(map_to_rank(smem_u32(dst), owner), v0, v1, v2, v3,
                      map_to_rank(bar, owner));
      }
    }
    cluster_arrive();  // no store of this CTA to another's memory is still to come
    named_bar_sync(1, C::EPI * 32);
    ok = ok && mbar_wait_spin(got, 0, abort_flag, p.err, p.timeout);
    ok = __all_sync(0xFFFFFFFFu, ok);
    // one warp per token, four rows per lane, the parts added in rank order
    for (int i = warp; ok && i < mine; i += C::EPI) {
      const int t = rank + i * split;
      float4 sum[C::AT];
#pragma unroll
      for (int a = 0; a < C::AT; ++a) {
        const float4* v =
            reinterpret_cast<const float4*>(parts + (i * C::AT + a) * split * 128) + lane;
        sum[a] = v[0];
        for (int r = 1; r < split; ++r) {
          sum[a].x += v[r * 32].x;
          sum[a].y += v[r * 32].y;
          sum[a].z += v[r * 32].z;
          sum[a].w += v[r * 32].w;
        }
      }
      const int64_t m = t0 + t;
      const int c = rb * 128 + lane * 4;
      if (ACT) {
        const float4 g = sum[0], u = sum[C::AT - 1];
        const float4 v = make_float4(silu(g.x) * u.x, silu(g.y) * u.y,
                                     silu(g.z) * u.z, silu(g.w) * u.w);
        if (p.out_dtype == KLT_DT_E4M3) {
          // the warp holds one group of 128 columns
          float amax = max_nan(max_nan(v.x, v.y, v.z), v.w);
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
  if (warp >= C::EPI) {
    cluster_wait();
    cluster_arrive();
  }
  tc_fence_before();
  __syncwarp();
  cluster_wait();  // every store into this CTA's memory has been issued, its TMEM has been read
  // An asynchronous store is complete on its barrier alone, which a CTA whose waits ran out has not
  // seen: its memory is the next CTA's only once they have all arrived.
  if (threadIdx.x == 0) {
    int none = 0;
    mbar_wait(got, 0, &none, p.err, p.timeout);
  }
  if (warp == C::EPI + 1) {
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
  cfg.blockDim = dim3(C::THREADS);
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

bool prepare_linear_narrow(int clusters[4]) {
  if (!prepare<16, 0>() || !prepare<32, 0>() || !prepare<64, 0>() || !prepare<128, 0>() ||
      !prepare<16, 1>() || !prepare<32, 1>() || !prepare<64, 1>())
    return false;
  for (int i = 0; i < 4; ++i) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(1 << i, 1, 1);
    cfg.blockDim = dim3(Narrow<128, 0>::THREADS);
    cfg.dynamicSmemBytes = Narrow<128, 0>::SMEM;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 1 << i;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&clusters[i], narrow_kernel<128, 0>, &cfg) != cudaSuccess)
      return false;
    if (clusters[i] < 1) clusters[i] = 1;
  }
  return true;
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
