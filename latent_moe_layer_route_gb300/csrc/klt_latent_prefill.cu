// Latent attention in expanded form over packed sequences (sm_103a).
//
// A pair of CTAs (cta_group::2) takes 512 queries of one head as two tiles of 256, 128 of each in
// either CTA, and goes over the keys 128 at a time: S = Q K^T (M = 256, N = 128, K = nope + rope),
// softmax with a row per thread, P as bf16 back into TMEM over S, O += P V with its first operand
// from TMEM.  Each CTA holds half of a tile's keys (64 rows) and half of its values (64 columns),
// which the tensor core reads from both: half of the copies, and half of the shared-memory reads
// that bound these products in one CTA (128 x 128 x 16 reads 8 KB in its 64 cycles).  The two
// tiles take turns: while the threads of one do its softmax, the tensor core works on the other.
//
// Roles in a CTA: warp 0 copies (three stages of 40 KB), warp 1 of the first CTA issues products,
// warps 4 to 7 and 8 to 11 do the tiles' softmax.  Their code is kept short (S is read twice, 64
// columns at a time): unrolled over the 128 columns it pushed the issuing thread's out of the
// instruction caches, which then took 5,500 cycles for the 2,560 of a round.  O is rescaled only
// when a row's maximum has grown by 2^8 (by the row's own thread, which knows that no product runs
// on it).
#include "klt_latent.cuh"

#include "../../include/klt.h"

namespace klt {
namespace {

constexpr int ROWS = 128, KEYS = 128;  // of a tile in one CTA
constexpr int BOX = 128 * 128;         // 128 rows x 128 bytes
constexpr int Q_BOXES = 3, STAGES = 3;
constexpr int K_BYTES = 3 * BOX / 2, STAGE = K_BYTES + BOX;  // keys: 64 rows; values: 128 rows
constexpr int THREADS = 384;
constexpr int SMEM = 1024 + 2 * Q_BOXES * BOX + STAGES * STAGE;
static_assert(4 * ROWS == PREFILL_ROWS, "");

// The first CTA's unless it says "each".
struct Bars {
  uint64_t k_full[STAGES], v_full[STAGES];    // bytes of both CTAs
  uint64_t k_empty[STAGES], v_empty[STAGES];  // each
  uint64_t q_full[2];
  uint64_t s_full[2], pv_done[2];             // each
  uint64_t p_full[2];                         // the softmax warps of both
  uint64_t v_last;                            // each: values of the last tile, where it is ragged
  uint64_t cleared;                           // ... cleared behind the sequence in both
  uint64_t drain;                             // each
  uint64_t ended;                             // the second CTA has issued its last copy
};

KLT_DEV void tma_load_3d_pair(void* dst, const CUtensorMap* map, uint32_t bar, int c0, int c1,
                              int c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      ".cta_group::2 [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2)
      : "memory");
}
// Four products of K = 16 over both CTAs, operands 32 bytes of a row apart.
KLT_DEV void mma4_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.eq.b32 q, 0, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %5, %6, %3, q;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %7, %8, %3, q;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %9, %10, %3, q;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "l"(a + 2), "l"(b + 2), "l"(a + 4),
      "l"(b + 4), "l"(a + 6), "l"(b + 6)
      : "memory");
}
KLT_DEV void mma_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.eq.b32 q, 0, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, q;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc)
      : "memory");
}
// ... with A in TMEM: bf16, two to a column, K = 16 in eight columns; B 16 rows of 128 bytes apart.
KLT_DEV void mma4_pair_ta(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                          uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.eq.b32 q, 0, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], [%5], %6, %3, q;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], [%7], %8, %3, q;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], [%9], %10, %3, q;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(a + 8), "l"(b + 128), "r"(a + 16),
      "l"(b + 256), "r"(a + 24), "l"(b + 384)
      : "memory");
}
// 64 columns of this thread's row; those from `seen` on are minus infinity.
KLT_DEV void load64(uint32_t taddr, int seen, uint32_t (*v)[32]) {
  tmem_start_ld32(taddr, v[0]);
  tmem_start_ld32(taddr + 32, v[1]);
  tmem_wait_ld32(v[0]);
  tmem_wait_ld32(v[1]);
  if (seen < 64) {
#pragma unroll
    for (int i = 0; i < 64; ++i)
      if (i >= seen) v[i >> 5][i & 31] = 0xFF800000u;
  }
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(THREADS, 1)
    prefill_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                   const __grid_constant__ CUtensorMap vmap,
                   const __grid_constant__ CUtensorMap rmap, const PrefillParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* qs = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  uint8_t* ring = qs + 2 * Q_BOXES * BOX;
  __shared__ Bars bars;
  __shared__ uint32_t tmem_holder, copies;
  __shared__ int abort_flag;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = static_cast<int>(cluster_rank());
  if (tid == 0) {
    for (int i = 0; i < STAGES; ++i) {
      mbar_init(&bars.k_full[i], 1);
      mbar_init(&bars.v_full[i], 1);
      mbar_init(&bars.k_empty[i], 1);
      mbar_init(&bars.v_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars.q_full[i], 1);
      mbar_init(&bars.s_full[i], 1);
      mbar_init(&bars.p_full[i], 8);
      mbar_init(&bars.pv_done[i], 1);
    }
    mbar_init(&bars.v_last, 1);
    mbar_init(&bars.cleared, 8);
    mbar_init(&bars.drain, 1);
    mbar_init(&bars.ended, 1);
    abort_flag = 0;
    fence_barrier_init();
    mbar_arrive_expect_tx(&bars.ended, 4);
    tma_prefetch_desc(&qmap);
    tma_prefetch_desc(&kmap);
    tma_prefetch_desc(&vmap);
    tma_prefetch_desc(&rmap);
  }
  if (warp == 2) tmem_alloc_pair(&tmem_holder, 512);
  pdl_trigger();
  pdl_wait();

  // this unit's sequence, 32 sequences at a time; a sequence's last units, which see most keys, first
  int unit = blockIdx.x >> 1, q0 = 0, q1 = 0, k0 = 0, k1 = 0;
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
    const uint32_t past = __ballot_sync(0xFFFFFFFFu, unit < in);
    if (past) {
      const int src = __ffs(past) - 1;
      found = true;
      unit = __shfl_sync(0xFFFFFFFFu, in, src) - 1 - unit;
      q0 = __shfl_sync(0xFFFFFFFFu, lo, src);
      q1 = __shfl_sync(0xFFFFFFFFu, hi, src);
      range_of(p.cu_k, b0 + src, p.S, k0, k1);
    } else {
      unit -= __shfl_sync(0xFFFFFFFFu, in, 31);
    }
  }
  const int h = blockIdx.y;
  const int n = q1 - q0, len = k1 - k0, r0 = unit * PREFILL_ROWS;
  const int nb = p.nope / 64;
  // tiles of keys that the last query of each tile of queries sees
  auto tiles_of = [&](int w) {
    const int last = min(r0 + (w + 1) * 2 * ROWS, n) - 1;
    const int seen =
        !found || last < r0 + w * 2 * ROWS ? 0 : p.causal ? len - (n - 1 - last) : len;
    return max(0, (seen + KEYS - 1) / KEYS);
  };
  const int tiles0 = tiles_of(0), tiles1 = tiles_of(1), nt = max(tiles0, tiles1);
  const bool ragged = nt * KEYS > len;  // the last tile of keys ends behind the sequence
  tc_fence_before();
  __syncthreads();
  cluster_arrive();  // the other CTA's barriers exist
  cluster_wait();
  tc_fence_after();
  const uint32_t tmem = tmem_holder;
  volatile int* stop = &abort_flag;
  auto wait = [&](uint64_t* bar, int phase) {
    return mbar_wait(bar, phase & 1, stop, p.err, p.timeout);
  };
  auto first = [&](uint64_t* bar) { return map_to_rank(smem_u32(bar), 0); };  // in the first CTA

  if (warp == 0) {
    if (elect_one()) {
      // ---------------------------------------------- copies
      for (int w = 0; w < 2; ++w)
        if ((w ? tiles1 : tiles0) > 0) {
          if (rank == 0) mbar_arrive_expect_tx(&bars.q_full[w], 2 * (nb + 1) * BOX);
          for (int i = 0; i <= nb; ++i)
            tma_load_3d_pair(qs + (w * Q_BOXES + i) * BOX, &qmap, first(&bars.q_full[w]), i * 64, h,
                             q0 + r0 + (2 * w + rank) * ROWS);
        }
      int it = 0;  // keys of tile it / 2, then its values
      bool ok = true;
      const int loads = 2 * (p.stall > 0 ? min(nt, p.stall) : nt);
      const int last = ragged ? 2 * nt - 1 : -1;
      for (; it < loads; ++it) {
        const int t = it >> 1, st = t % STAGES, row = k0 + t * KEYS;
        uint8_t* dst = ring + st * STAGE;
        if (!(it & 1)) {
          ok = wait(&bars.k_empty[st], t / STAGES + 1);
          if (!ok) break;
          if (rank == 0) mbar_arrive_expect_tx(&bars.k_full[st], (nb + 1) * BOX);
          const uint32_t bar = first(&bars.k_full[st]);
          for (int i = 0; i < nb; ++i)
            tma_load_3d_pair(dst + i * (BOX / 2), &kmap, bar, i * 64, h, row + rank * (KEYS / 2));
          tma_load_3d_pair(dst + nb * (BOX / 2), &rmap, bar, 0, 0, row + rank * (KEYS / 2));
        } else {
          ok = wait(&bars.v_empty[st], t / STAGES + 1);
          if (!ok) break;
          if (it == last) {
            mbar_arrive_expect_tx(&bars.v_last, BOX);
            tma_load_3d(dst + K_BYTES, &vmap, &bars.v_last, rank * 64, h, row);
          } else {
            if (rank == 0) mbar_arrive_expect_tx(&bars.v_full[st], 2 * BOX);
            tma_load_3d_pair(dst + K_BYTES, &vmap, first(&bars.v_full[st]), rank * 64, h, row);
          }
        }
      }
      // No copy of the pair is in flight past this point.  The first CTA waits for all, those too
      // that the second has issued beyond its own after a wait that ran out.
      int none = 0;
      if (last >= 0 && it > last) mbar_wait(&bars.v_last, 0, &none, p.err, p.timeout);
      auto landed = [&](int j) {
        const int t = j >> 1;
        if (j != last)
          mbar_wait(j & 1 ? &bars.v_full[t % STAGES] : &bars.k_full[t % STAGES], (t / STAGES) & 1,
                    &none, p.err, p.timeout);
      };
      if (rank == 0) {
        for (int w = 0; w < 2; ++w)
          if ((w ? tiles1 : tiles0) > 0)
            mbar_wait(&bars.q_full[w], 0, &none, p.err, p.timeout);
        for (int j = max(0, it - 2 * STAGES); j < it; ++j) landed(j);
        // its waits are bounded and began before this CTA's last ones ended
        if (mbar_wait(&bars.ended, 0, &none, p.err, 3 * p.timeout)) {
          const int others = static_cast<int>(*static_cast<volatile uint32_t*>(&copies));
          for (; it < others; ++it) {
            const int t = it >> 1;
            if (it == last) continue;
            if (it & 1)
              mbar_arrive_expect_tx(&bars.v_full[t % STAGES], BOX);
            else
              mbar_arrive_expect_tx(&bars.k_full[t % STAGES], (nb + 1) * (BOX / 2));
            landed(it);
          }
        }
      } else {
        st_async_u32(first(reinterpret_cast<uint64_t*>(&copies)), it, first(&bars.ended));
      }
    }
  } else if (warp == 1 && rank == 0) {
    if (elect_one()) {
      // ---------------------------------------------- products
      constexpr uint32_t sdesc = idesc_make(1, 256, 128);
      constexpr uint32_t vdesc = idesc_make(1, 256, 128) | IDESC_B_MN;
      bool ok = true;
      // of tile t of keys with tile w of queries; the last user hands the stage back
      auto scores = [&](int w, int t, bool wanted, bool last) {
        const int st = t % STAGES;
        if (wanted) ok = wait(&bars.k_full[st], t / STAGES);
        if (!ok) return;
        tc_fence_after();
        const uint64_t qa = sdesc_sw128(smem_u32(qs + w * Q_BOXES * BOX)),
                       ka = sdesc_sw128(smem_u32(ring + st * STAGE));
        const uint32_t d = tmem + w * 128;
        mma4_pair(d, qa, ka, sdesc, 0);
        if (nb > 1) mma4_pair(d, qa + BOX / 16, ka + BOX / 32, sdesc, 1);
        const uint64_t qr = qa + nb * (BOX / 16), kr = ka + nb * (BOX / 32);
        if (p.rope == 64)
          mma4_pair(d, qr, kr, sdesc, 1);
        else
          for (int s = 0; s < p.rope / 16; ++s) mma_pair(d, qr + 2 * s, kr + 2 * s, sdesc);
        tc_commit_pair(&bars.s_full[w], 3);
        if (last) tc_commit_pair(&bars.k_empty[st], 3);
      };
      auto values = [&](int w, int t, bool wanted, bool last) {
        const int st = t % STAGES;
        if (wanted)
          ok = ragged && t == nt - 1 ? wait(&bars.cleared, 0) : wait(&bars.v_full[st], t / STAGES);
        ok = ok && wait(&bars.p_full[w], t);
        if (!ok) return;
        tc_fence_after();
        const uint64_t va = sdesc_sw128_mn(smem_u32(ring + st * STAGE + K_BYTES), BOX);
        const uint32_t d = tmem + 256 + w * 128, a = tmem + w * 128;
        mma4_pair_ta(d, a, va, vdesc, t);
        mma4_pair_ta(d, a + 32, va + 512, vdesc, 1);
        tc_commit_pair(&bars.pv_done[w], 3);
        if (last) tc_commit_pair(&bars.v_empty[st], 3);
      };
      if (tiles0 > 0) {
        ok = wait(&bars.q_full[0], 0);
        if (ok) scores(0, 0, true, tiles1 <= 0);
      }
      if (tiles1 > 0 && ok) {
        ok = wait(&bars.q_full[1], 0);
        if (ok) scores(1, 0, tiles0 <= 0, true);
      }
      for (int t = 0; t < nt && ok; ++t) {
        if (t < tiles0) values(0, t, true, t >= tiles1);
        if (ok && t + 1 < tiles0) scores(0, t + 1, true, t + 1 >= tiles1);
        if (ok && t < tiles1) values(1, t, t >= tiles0, true);
        if (ok && t + 1 < tiles1) scores(1, t + 1, t + 1 >= tiles0, true);
      }
      tc_commit_pair(&bars.drain, 3);  // no product of the pair runs past this point
    }
  } else if (warp >= 4) {
    // ------------------------------------------------ softmax: a row per thread
    const int w = (warp - 4) >> 2, quad = warp & 3;
    const int row = r0 + (2 * w + rank) * ROWS + quad * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>(quad * 32) << 16;
    const uint32_t S = tmem + w * 128 + lanes, O = tmem + 256 + w * 128 + lanes;
    const int limit = row >= n ? 0 : p.causal ? len - (n - 1 - row) : len;
    float m = -INFINITY, l = 0.f;
    bool ok = true;
    const int mine = w ? tiles1 : tiles0;
    const uint32_t p_full = first(&bars.p_full[w]);
    for (int t = 0; t < mine; ++t) {
      ok = wait(&bars.s_full[w], t);
      ok = __all_sync(0xFFFFFFFFu, ok);
      if (!ok) break;
      tc_fence_after();
      if (ragged && t == nt - 1 && (w == 1 || tiles1 < nt)) {
        // what the values hold behind the sequence is cleared: it may not be finite
        ok = wait(&bars.v_last, 0);
        ok = __all_sync(0xFFFFFFFFu, ok);
        if (!ok) break;
        uint8_t* vs = ring + (t % STAGES) * STAGE + K_BYTES;
        for (int c = (len - t * KEYS) * 8 + quad * 32 + lane; c < KEYS * 8; c += 128)
          *reinterpret_cast<uint4*>(vs + c * 16) = make_uint4(0, 0, 0, 0);
        fence_proxy_async_shared();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster_release(first(&bars.cleared));
      }
      float top = -INFINITY;
#pragma unroll 1
      for (int c = 0; c < KEYS; c += 64) {
        uint32_t v[2][32];
        load64(S + c, limit - t * KEYS - c, v);
        float x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          x[i] = __uint_as_float(v[i >> 1][(i & 1) * 16]);
#pragma unroll
          for (int j = 1; j < 15; j += 2)
            x[i] = fmaxf(fmaxf(x[i], __uint_as_float(v[i >> 1][(i & 1) * 16 + j])),
                         __uint_as_float(v[i >> 1][(i & 1) * 16 + j + 1]));
          x[i] = fmaxf(x[i], __uint_as_float(v[i >> 1][(i & 1) * 16 + 15]));
        }
        top = fmaxf(fmaxf(top, fmaxf(x[0], x[1])), fmaxf(x[2], x[3]));
      }
      top *= p.scale;
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
#pragma unroll 1
      for (int c = 0; c < KEYS; c += 64) {
        uint32_t v[2][32], pk[32];
        load64(S + c, limit - t * KEYS - c, v);
#pragma unroll
        for (int i = 0; i < 64; i += 2) {
          float a, b;
          unpack2(fmaf2(pack2(__uint_as_float(v[i >> 5][i & 31]),
                              __uint_as_float(v[i >> 5][(i & 31) + 1])),
                        s2, b2),
                  a, b);
          a = exp2_fast(a);
          b = exp2_fast(b);
          add2(sum[i >> 1 & 1], pack2(a, b));
          pk[i / 2] = pack_bf16(a, b);
        }
        tmem_st32(S + c / 2, pk);  // over columns that have been read
      }
      add2(sum[0], sum[1]);
      float a, b;
      unpack2(sum[0], a, b);
      l += a + b;
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(p_full);
    }
    if (ok && mine > 0) ok = wait(&bars.pv_done[w], mine - 1);
    ok = __all_sync(0xFFFFFFFFu, ok);
    const int from = row - lane;  // this warp's first row
    if (ok && from < n) {
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
      for (int i = lane; i < 32 * chunks; i += 32) {
        const int r = i / chunks, c = i % chunks;
        if (from + r < n)
          *reinterpret_cast<uint4*>(p.out + static_cast<int64_t>(q0 + from + r) * p.out_token +
                                    h * p.out_head + c * 8) =
              *reinterpret_cast<const uint4*>(stage + r * 256 + ((c ^ (r & 7)) << 4));
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (tid == 0) {  // the products of both CTAs are done, and with them all signals to this one
    int none = 0;
    mbar_wait(&bars.drain, 0, &none, p.err, 4 * p.timeout);
  }
  cluster_arrive();
  cluster_wait();
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

}  // namespace

bool prepare_prefill() {
  return cudaFuncSetAttribute(prefill_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              SMEM) == cudaSuccess;
}

cudaError_t launch_prefill(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                           const CUtensorMap& k_rope, const PrefillParams& p, unsigned tiles,
                           cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * tiles, p.H);
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
