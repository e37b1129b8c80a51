// Latent attention in expanded form over packed sequences (sm_103a).
//
// A CTA takes 256 queries of one head as two tiles of 128 and goes over the keys 128 at a time:
// S = Q K^T (M = N = 128, K = nope + rope), softmax with a row per thread, P as bf16 back into
// TMEM over S, O += P V with its first operand from TMEM.  The two tiles take turns: while the
// threads of one do its softmax, the tensor core works on the other, so its time is the sum of
// the products, (nope + rope + value) / 16 x 64 cycles per tile and 128 keys.
//
// Roles: warp 0 copies (keys' and values' boxes of 128 rows x 64 columns through a ring of eight),
// warp 1 issues products, warps 4 to 7 and 8 to 11 do the tiles' softmax.  O is rescaled only when a
// row's maximum has grown by 2^8 (by the row's own thread, which knows that no product runs on it).
#include "klt_latent.cuh"

#include "../../include/klt.h"

namespace klt {
namespace {

constexpr int ROWS = 128, KEYS = 128;
constexpr int BOX = 128 * 128;  // 128 rows x 128 bytes
constexpr int Q_BOXES = 3, SLOTS = 8;
constexpr int THREADS = 384;
constexpr int SMEM = 1024 + (2 * Q_BOXES + SLOTS) * BOX;
static_assert(2 * ROWS == PREFILL_ROWS, "");

struct Bars {
  uint64_t full[SLOTS], empty[SLOTS];
  uint64_t q_full[2], s_full[2], p_full[2], pv_done[2];
  uint64_t cleared, drain;
};

__global__ void __launch_bounds__(THREADS, 1)
    prefill_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                   const __grid_constant__ CUtensorMap vmap,
                   const __grid_constant__ CUtensorMap rmap, const PrefillParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* qs = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  uint8_t* ring = qs + 2 * Q_BOXES * BOX;
  __shared__ Bars bars;
  __shared__ uint32_t tmem_holder;
  __shared__ int abort_flag;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < SLOTS; ++i) {
      mbar_init(&bars.full[i], 1);
      mbar_init(&bars.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars.q_full[i], 1);
      mbar_init(&bars.s_full[i], 1);
      mbar_init(&bars.p_full[i], 4);
      mbar_init(&bars.pv_done[i], 1);
    }
    mbar_init(&bars.cleared, 4);
    mbar_init(&bars.drain, 1);
    abort_flag = 0;
    fence_barrier_init();
    tma_prefetch_desc(&qmap);
    tma_prefetch_desc(&kmap);
    tma_prefetch_desc(&vmap);
    tma_prefetch_desc(&rmap);
  }
  if (warp == 1) {
    tmem_alloc(&tmem_holder, 512);
    tmem_relinquish();
  }
  pdl_trigger();
  pdl_wait();

  // this tile's sequence, 32 sequences at a time; a sequence's last tiles, which see most keys, first
  int tile = blockIdx.x, q0 = 0, q1 = 0, k0 = 0, k1 = 0;
  bool found = false;
  for (int b0 = 0; b0 < p.B && !found; b0 += 32) {
    int lo = 0, hi = 0, n = 0;
    if (b0 + lane < p.B) {
      range_of(p.cu_q, b0 + lane, p.T, lo, hi);
      n = (hi - lo + PREFILL_ROWS - 1) / PREFILL_ROWS;
    }
    int in = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xFFFFFFFFu, in, o);
      if (lane >= o) in += v;
    }
    const uint32_t past = __ballot_sync(0xFFFFFFFFu, tile < in);
    if (past) {
      const int src = __ffs(past) - 1;
      found = true;
      tile = __shfl_sync(0xFFFFFFFFu, in, src) - 1 - tile;
      q0 = __shfl_sync(0xFFFFFFFFu, lo, src);
      q1 = __shfl_sync(0xFFFFFFFFu, hi, src);
      range_of(p.cu_k, b0 + src, p.S, k0, k1);
    } else {
      tile -= __shfl_sync(0xFFFFFFFFu, in, 31);
    }
  }
  const int h = blockIdx.y;
  const int n = q1 - q0, len = k1 - k0, r0 = tile * PREFILL_ROWS;
  const int nb = p.nope / 64, vb = p.value / 64;
  // tiles of keys that the last query of each tile of queries sees
  int tiles[2];
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    const int last = min(r0 + (w + 1) * ROWS, n) - 1;
    const int seen = !found || last < r0 + w * ROWS ? 0 : p.causal ? len - (n - 1 - last) : len;
    tiles[w] = max(0, (seen + KEYS - 1) / KEYS);
  }
  const int nt = max(tiles[0], tiles[1]);
  const bool ragged = nt * KEYS > len;  // the last tile of keys ends behind the sequence
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_holder;
  volatile int* stop = &abort_flag;
  auto wait = [&](uint64_t* bar, int phase) {
    return mbar_wait(bar, phase & 1, stop, p.err, p.timeout);
  };

  if (warp < 4) {
    regs_dec<72>();
    if (warp == 0 && elect_one()) {
      // ---------------------------------------------- copies
      for (int w = 0; w < 2; ++w)
        if (tiles[w] > 0) {
          mbar_arrive_expect_tx(&bars.q_full[w], (nb + 1) * BOX);
          for (int i = 0; i <= nb; ++i)
            tma_load_3d(qs + (w * Q_BOXES + i) * BOX, &qmap, &bars.q_full[w], i * 64, h,
                        q0 + r0 + w * ROWS);
        }
      int it = 0;  // boxes
      bool ok = true;
      for (int t = 0; t < nt && ok; ++t) {
        if (p.stall > 0 && t >= p.stall) break;
        const int row = k0 + t * KEYS;
        for (int i = 0; i < nb + 1 + vb; ++i, ++it) {
          const int slot = it % SLOTS;
          ok = wait(&bars.empty[slot], it / SLOTS + 1);
          if (!ok) break;
          mbar_arrive_expect_tx(&bars.full[slot], BOX);
          uint8_t* dst = ring + slot * BOX;
          if (i < nb)
            tma_load_3d(dst, &kmap, &bars.full[slot], i * 64, h, row);
          else if (i == nb)
            tma_load_3d(dst, &rmap, &bars.full[slot], 0, 0, row);
          else
            tma_load_3d(dst, &vmap, &bars.full[slot], (i - nb - 1) * 64, h, row);
        }
      }
      // no copy of this CTA is in flight past this point
      int none = 0;
      for (int w = 0; w < 2; ++w)
        if (tiles[w] > 0) mbar_wait(&bars.q_full[w], 0, &none, p.err, p.timeout);
      for (int j = it > SLOTS ? it - SLOTS : 0; j < it; ++j)
        mbar_wait(&bars.full[j % SLOTS], (j / SLOTS) & 1, &none, p.err, p.timeout);
    } else if (warp == 1 && elect_one()) {
      // ---------------------------------------------- products
      const int per = nb + 1 + vb;
      bool ok = true;
      // scores of tile t of keys for tile w of queries; the last user hands the boxes back
      auto scores = [&](int w, int t, bool last) {
        const uint32_t qa = smem_u32(qs + w * Q_BOXES * BOX);
        for (int i = 0; i <= nb && ok; ++i) {
          const int it = t * per + i, slot = it % SLOTS;
          ok = wait(&bars.full[slot], it / SLOTS);
          if (!ok) return;
          tc_fence_after();
          const uint32_t ka = smem_u32(ring + slot * BOX);
          if (i < nb)
            mma4_bf16(tmem + w * 128, sdesc_sw128(qa + i * BOX), sdesc_sw128(ka),
                      idesc_make(1, 128, 128), i);
          else
            for (int s = 0; s < p.rope / 16; ++s)
              mma_bf16(tmem + w * 128, sdesc_sw128(qa + i * BOX) + 2 * s, sdesc_sw128(ka) + 2 * s,
                       idesc_make(1, 128, 128), 1);
          if (last) tc_commit(&bars.empty[slot]);
        }
        tc_commit(&bars.s_full[w]);
      };
      auto values = [&](int w, int t, bool last) {
        ok = wait(&bars.p_full[w], t) && (!ragged || t < nt - 1 || wait(&bars.cleared, 0));
        for (int i = 0; i < vb && ok; ++i) {
          const int it = t * per + nb + 1 + i, slot = it % SLOTS;
          ok = wait(&bars.full[slot], it / SLOTS);
          if (!ok) return;
          tc_fence_after();
          const uint32_t va = smem_u32(ring + slot * BOX);
#pragma unroll
          for (int s = 0; s < 8; ++s)
            mma_bf16_ta(tmem + 256 + w * 128 + i * 64, tmem + w * 128 + 8 * s,
                        sdesc_sw128_mn(va + s * 2048, BOX), idesc_make(1, 128, 64) | IDESC_B_MN,
                        t | s);
          if (last) tc_commit(&bars.empty[slot]);
        }
        if (ok) tc_commit(&bars.pv_done[w]);
      };
      for (int w = 0; w < 2; ++w)
        if (tiles[w] > 0 && ok) {
          ok = wait(&bars.q_full[w], 0);
          if (ok) scores(w, 0, w == 1 || tiles[1] <= 0);
        }
      for (int t = 0; t < nt && ok; ++t)
        for (int w = 0; w < 2 && ok; ++w) {
          if (t < tiles[w]) values(w, t, w == 1 || tiles[1] <= t);
          if (ok && t + 1 < tiles[w]) scores(w, t + 1, w == 1 || tiles[1] <= t + 1);
        }
      tc_commit(&bars.drain);  // no product runs past this point
      int none = 0;
      mbar_wait(&bars.drain, 0, &none, p.err, p.timeout);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------ softmax: a row per thread
    regs_inc<216>();
    const int w = (warp - 4) >> 2, quad = warp & 3;
    const int row = r0 + w * ROWS + quad * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>(quad * 32) << 16;
    const uint32_t S = tmem + w * 128 + lanes, O = tmem + 256 + w * 128 + lanes;
    const int limit = row >= n ? 0 : p.causal ? len - (n - 1 - row) : len;
    float m = -INFINITY, l = 0.f;
    bool ok = true;
    const int mine = tiles[w];
    for (int t = 0; t < mine; ++t) {
      ok = wait(&bars.s_full[w], t);
      ok = __all_sync(0xFFFFFFFFu, ok);
      if (!ok) break;
      tc_fence_after();
      uint32_t v[4][32];
#pragma unroll
      for (int c = 0; c < 4; ++c) tmem_start_ld32(S + c * 32, v[c]);
#pragma unroll
      for (int c = 0; c < 4; ++c) tmem_wait_ld32(v[c]);
      if (ragged && t == nt - 1 && (w == 1 || tiles[1] < nt)) {
        // what the values' boxes hold behind the sequence is cleared: it may not be finite.  The
        // copy before in the same slot was read by the scores of the tile before, so these waits
        // are not a round late.
        for (int i = 0; i < vb; ++i) {
          const int it = t * (nb + 1 + vb) + nb + 1 + i, slot = it % SLOTS;
          ok = ok && wait(&bars.full[slot], it / SLOTS);
          if (ok)
            for (int c = (len - t * KEYS) * 8 + quad * 32 + lane; c < KEYS * 8; c += 128)
              *reinterpret_cast<uint4*>(ring + slot * BOX + c * 16) = make_uint4(0, 0, 0, 0);
        }
        ok = __all_sync(0xFFFFFFFFu, ok);
        if (!ok) break;
        fence_proxy_async_shared();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.cleared);
      }
      if ((t + 1) * KEYS > limit) {
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (t * KEYS + c * 32 + i >= limit) v[c][i] = 0xFF800000u;  // -inf
      }
      float top4[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        top4[c] = __uint_as_float(v[c][0]);
#pragma unroll
        for (int i = 1; i < 31; i += 2)
          top4[c] = fmaxf(fmaxf(top4[c], __uint_as_float(v[c][i])), __uint_as_float(v[c][i + 1]));
        top4[c] = fmaxf(top4[c], __uint_as_float(v[c][31]));
      }
      const float top = fmaxf(fmaxf(top4[0], top4[1]), fmaxf(top4[2], top4[3])) * p.scale;
      // the maximum in use may lag by 8: weights stay below 2^8
      if (__any_sync(0xFFFFFFFFu, top > m + 8.f)) {
        const float now = fmaxf(m, top);
        const float f = now == -INFINITY ? 1.f : exp2_fast(m - now);
        m = now;
        l *= f;
        if (t > 0) {  // the row's last product has to be done
          ok = wait(&bars.pv_done[w], t - 1);
          ok = __all_sync(0xFFFFFFFFu, ok);
          if (!ok) break;
          tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < p.value; c += 16) {
            float o[16];
            tmem_ld16(O + c, o);
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] *= f;
            tmem_st16(O + c, o);
          }
        }
      }
      const float base = m == -INFINITY ? 0.f : m;
      const unsigned long long s2 = pack2(p.scale, p.scale), b2 = pack2(-base, -base);
      unsigned long long sum[2] = {0ull, 0ull};
#pragma unroll
      for (int c = 0; c < 4; c += 2) {
        uint32_t pk[32];
#pragma unroll
        for (int g = 0; g < 2; ++g)
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            float a, b;
            unpack2(fmaf2(pack2(__uint_as_float(v[c + g][i]), __uint_as_float(v[c + g][i + 1])),
                          s2, b2),
                    a, b);
            a = exp2_fast(a);
            b = exp2_fast(b);
            add2(sum[g], pack2(a, b));
            pk[g * 16 + i / 2] = pack_bf16(a, b);
          }
        tmem_st32(S + c * 16, pk);
      }
      add2(sum[0], sum[1]);
      float a, b;
      unpack2(sum[0], a, b);
      l += a + b;
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars.p_full[w]);
    }
    if (ok && mine > 0) ok = wait(&bars.pv_done[w], mine - 1);
    ok = __all_sync(0xFFFFFFFFu, ok);
    if (ok && r0 + w * ROWS < n) {
      tc_fence_after();
      const float f = l != 0.f ? 1.0f / l : 0.f;
      if (p.lse && row < n)
        p.lse[static_cast<int64_t>(q0 + row) * p.H + h] =
            l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
      // through this warp's part of the queries' memory, which no product reads any more, so that
      // whole rows are stored: 16 bytes at chunk c ^ row of a row
      const int chunks = p.value / 8;
      uint8_t* stage = qs + (w * Q_BOXES * BOX) + quad * 32 * 256;
#pragma unroll 1
      for (int c = 0; c < p.value; c += 32) {
        uint32_t o[32];
        if (mine > 0) {
          tmem_start_ld32(O + c, o);
          tmem_wait_ld32(o);
        }
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if (mine == 0 || f == 0.f) o[i] = 0;
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          uint32_t x[4];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            x[i] = pack_bf16(__uint_as_float(o[8 * g + 2 * i]) * f,
                             __uint_as_float(o[8 * g + 2 * i + 1]) * f);
          *reinterpret_cast<uint4*>(stage + lane * 256 + (((c / 8 + g) ^ (lane & 7)) << 4)) =
              make_uint4(x[0], x[1], x[2], x[3]);
        }
      }
      __syncwarp();
      const int first = r0 + w * ROWS + quad * 32;
      for (int i = lane; i < 32 * chunks; i += 32) {
        const int r = i / chunks, c = i % chunks;
        if (first + r < n)
          *reinterpret_cast<uint4*>(p.out + static_cast<int64_t>(q0 + first + r) * p.out_token +
                                    h * p.out_head + c * 8) =
              *reinterpret_cast<const uint4*>(stage + r * 256 + ((c ^ (r & 7)) << 4));
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

}  // namespace

bool prepare_prefill() {
  cudaFuncAttributes a;
  // the register split needs the launch's 168 a thread
  return cudaFuncSetAttribute(prefill_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              SMEM) == cudaSuccess &&
         cudaFuncGetAttributes(&a, prefill_kernel) == cudaSuccess && a.numRegs == 168;
}

cudaError_t launch_prefill(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                           const CUtensorMap& k_rope, const PrefillParams& p, unsigned tiles,
                           cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(tiles, p.H);
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = SMEM;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, prefill_kernel, q, k, v, k_rope, p);
}

}  // namespace klt
