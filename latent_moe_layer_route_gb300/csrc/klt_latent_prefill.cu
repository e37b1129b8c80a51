// Latent attention in expanded form over packed sequences (sm_103a).
//
// A pair of CTAs (cta_group::2) takes 512 queries of one head as two tiles of 256, 128 of each in
// either CTA, and goes over the keys 128 at a time: S = Q K^T (M = 256, N = 128, K = nope + rope),
// softmax with a row per thread, P as bf16 back into TMEM over S, O += P V with its first operand
// from TMEM.  Each CTA holds half of a tile's keys (64 rows) and half of its values (64 columns),
// which the tensor core reads from both: half of the copies, and half of the shared-memory reads
// that bound these products in one CTA (128 x 128 x 16 reads 8 KB in its 64 cycles).  The two
// tiles take turns: while the threads of one do its softmax, the tensor core works on the other.
// Up to 256 queries (a sequence's last ones, or all of a short one) are one tile whose keys are shared
// out between the two groups of threads, even and odd tiles; at the end either takes half of the
// columns of both results (128 queries of 4 x 16 K keys, 32 heads: 247 us, one group alone 435).
//
// Roles in a CTA: warp 0 copies (three stages of 40 KB), warp 1 of the first CTA issues products,
// warp 3 finds the next unit (512 queries of a sequence and head), warps 4 to 7 and 8 to 11 do the
// tiles' softmax.  The grid has a pair for every unit; a running pair takes over units that have not
// started (clusterlaunchcontrol), so that it loads the next one's operands and computes its first
// scores while it writes the results of this one, and long and short sequences even out.
//
// The softmax goes over a tile's scores once, 64 keys at a time: they are weighted by the maximum in
// use while their own is found, and once more in the rare case that it has grown by 2^8 (then O is
// rescaled too).  Each half's weights are handed to the tensor core as they are written, as bf16, the
// type of the values that they multiply: unnormalised, below 2^8, each rounded by at most 2^-8 of
// itself.  The sum that divides results is that of the unrounded weights, and scores, maxima, sums and
// results are fp32.  Against 64 bits results are off by 0.0018 to 0.0023 (root of squares), 0.0016 to
// 0.0017 with fp32 weights.  8192 tokens of 64 heads take 774 to 811 us in a burst (up to 1.78
// PFLOP/s, 92 % of a large library product's rate), 846 to 869 in runs of seconds.  With the maximum
// found in a pass of its own, the kernel of 807 us before took 895; a quarter of the exponentials by
// a polynomial 937, two threads to a row 986: the exponential unit is not what bounds this on
// sm_103a, the way of a tile through scores, softmax and values is (some 4,300 cycles where a group
// is alone, of which its softmax 2,300).  Hence short sequences cost most: 12 ragged ones of up to
// 2500 tokens 262 to 275 us (0.93 PFLOP/s).  Values of 64 columns are multiplied as 128, the second
// CTA's half as zeros: 8192 tokens of 64 + 64 + 64 columns 683 us (1.21 PFLOP/s), 128 + 64 + 64 783.
// A unit's keys are never cut over pairs: 128 queries of 16 K keys take 124 us with 16 heads, which
// keep 16 of the 76 pairs, and 126 with 64.  First scores of the next unit issued while the second
// group ends this one: no gain; the first tile's maximum found ahead of its weights: 5 % slower.
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

// 512 queries of a sequence and head as two tiles that go over the same keys; or up to 256 as one,
// whose even tiles of keys are the first softmax group's and odd ones the second's.
struct Unit {
  int q0, n;           // the sequence's first query, its queries
  int k0, len;         // ... keys
  int r0, h;           // the unit's first query in the sequence, its head
  int split;           // one tile of queries
  int nt;              // tiles of keys that the last query sees
  int tiles0, tiles1;  // ... of each group
  int last;            // no unit: the pair is done
};

// The first CTA's unless it says "each".
struct Bars {
  uint64_t k_full[STAGES], v_full[STAGES];    // bytes of both CTAs
  uint64_t k_empty[STAGES], v_empty[STAGES];  // each
  uint64_t q_full[2], q_empty[2];             // q_empty: each
  uint64_t s_full[2], pv_done[2];             // each
  uint64_t p_half[2], p_full[2], o_free[2];   // the softmax warps of both
  uint64_t pv_half[2];                        // each: products with the first half of a tile
  uint64_t v_last[STAGES];                    // each: values of a sequence's ragged last tile
  uint64_t cleared;                           // ... cleared behind the sequence in both
  uint64_t unit_full[2], unit_empty[2];       // each
  uint64_t shared[2], shared_read[2];         // each: a group's sums are there, are read
  uint64_t loaded;                            // each: a unit's copies are issued
  uint64_t next_full[2];                      // each: the answer about the next unit
  uint64_t next_read;                         // the second CTA has read it
  uint64_t drain;                             // each
  uint64_t ended;                             // the second CTA has issued its last copy
  uint64_t asked;                             // the second's: the first has asked its last question
};
// What the second CTA has issued.
struct Copies {
  uint32_t it;       // keys of tile it / 2, then its values
  uint32_t queries[2];
  uint32_t alone;    // stages whose last values were signalled to the second CTA alone
};

// Asks for a cluster of the grid that has not started; the answer (16 bytes) and its signal go to
// the same places in both CTAs.
KLT_DEV void ask_next(void* answer, uint64_t* bar) {
  asm volatile(
      "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes"
      ".multicast::cluster::all.b128 [%0], [%1];" ::"r"(smem_u32(answer)),
      "r"(smem_u32(bar))
      : "memory");
}
// The first CTA of the cluster that was given, or false.
KLT_DEV bool read_next(const void* answer, int& x) {
  uint32_t ok, a;
  asm volatile(
      "{\n\t.reg .b128 r;\n\t.reg .pred p;\n\t"
      "ld.shared.b128 r, [%2];\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n\t"
      "selp.u32 %0, 1, 0, p;\n\tmov.u32 %1, 0;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, r;\n\t}"
      : "=r"(ok), "=r"(a)
      : "r"(smem_u32(answer))
      : "memory");
  x = static_cast<int>(a);
  return ok != 0;
}
// Where a search was: 32 sequences from b0 on, units before them.
struct Place {
  int b0 = 0, before = 0;
};
// Unit number `number` of head h, by a whole warp, 32 sequences at a time from where the search
// before ended (numbers mostly ascend); a sequence's last units, which see most keys, come first.
// Numbers past the last unit have no queries.
KLT_DEV Unit find_unit(const PrefillParams& p, int number, int h, Place& at) {
  const int lane = lane_id();
  Unit u = {};
  u.h = h;
  if (number < at.before) at = Place();
  for (; at.b0 < p.B; at.b0 += 32) {
    const int b0 = at.b0, unit = number - at.before;
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
      int k1;
      u.r0 = (__shfl_sync(0xFFFFFFFFu, in, src) - 1 - unit) * PREFILL_ROWS;
      u.q0 = __shfl_sync(0xFFFFFFFFu, lo, src);
      u.n = __shfl_sync(0xFFFFFFFFu, hi, src) - u.q0;
      range_of(p.cu_k, b0 + src, p.S, u.k0, k1);
      u.len = k1 - u.k0;
      auto tiles_of = [&](int w) {
        const int last = min(u.r0 + (w + 1) * 2 * ROWS, u.n) - 1;
        const int seen = p.causal ? u.len - (u.n - 1 - last) : u.len;
        return max(0, (seen + KEYS - 1) / KEYS);
      };
      u.split = u.n - u.r0 <= 2 * ROWS;
      u.nt = tiles_of(u.split ? 0 : 1);
      u.tiles0 = u.split ? (u.nt + 1) / 2 : tiles_of(0);
      u.tiles1 = u.split ? u.nt / 2 : u.nt;
      break;
    }
    at.before += __shfl_sync(0xFFFFFFFFu, in, 31);
  }
  return u;
}

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

// The weights of 64 scores, 2^(s scale - m), as bf16, and their sums (to be added up); returns the
// largest of s scale.
KLT_DEV float weights64(const uint32_t (*v)[32], float scale, float m, unsigned long long* sum,
                        uint32_t* out) {
  const float base = m == -INFINITY ? 0.f : m;
  const unsigned long long s2 = pack2(scale, scale), b2 = pack2(-base, -base);
  sum[0] = sum[1] = 0ull;
  float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
  for (int k = 0; k < 64; k += 2) {
    float a = __uint_as_float(v[k >> 5][k & 31]), b = __uint_as_float(v[k >> 5][(k & 31) + 1]);
    top[k >> 1 & 3] = fmaxf(fmaxf(top[k >> 1 & 3], a), b);
    unpack2(fmaf2(pack2(a, b), s2, b2), a, b);
    a = exp2_fast(a);
    b = exp2_fast(b);
    add2(sum[k >> 1 & 1], pack2(a, b));
    out[k / 2] = pack_bf16(a, b);
  }
  return fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * scale;
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(THREADS, 1)
    prefill_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                   const __grid_constant__ CUtensorMap vmap,
                   const __grid_constant__ CUtensorMap rmap, const PrefillParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* qs = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  uint8_t* ring = qs + 2 * Q_BOXES * BOX;
  __shared__ Bars bars;
  __shared__ Unit units[2];
  __shared__ float2 shares[2][ROWS];  // maximum and sum of each group's part of the keys
  __shared__ uint4 answers[2];
  __shared__ uint32_t tmem_holder;
  __shared__ Copies copies;
  __shared__ uint32_t questions;
  __shared__ int abort_flag;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = static_cast<int>(cluster_rank());
  if (tid == 0) {
    for (int i = 0; i < STAGES; ++i) {
      mbar_init(&bars.k_full[i], 1);
      mbar_init(&bars.v_full[i], 1);
      mbar_init(&bars.k_empty[i], 1);
      mbar_init(&bars.v_empty[i], 1);
      mbar_init(&bars.v_last[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars.q_full[i], 1);
      mbar_init(&bars.q_empty[i], 1);
      mbar_init(&bars.s_full[i], 1);
      mbar_init(&bars.p_half[i], 8);
      mbar_init(&bars.pv_half[i], 1);
      mbar_init(&bars.p_full[i], 8);
      mbar_init(&bars.o_free[i], 8);
      mbar_init(&bars.pv_done[i], 1);
      mbar_init(&bars.unit_full[i], 1);
      mbar_init(&bars.unit_empty[i], rank == 0 ? 10 : 9);  // copies, products, softmax warps
      mbar_init(&bars.next_full[i], 1);
      mbar_init(&bars.shared[i], 4);
      mbar_init(&bars.shared_read[i], 4);
    }
    mbar_init(&bars.loaded, 1);
    mbar_init(&bars.next_read, 1);
    mbar_init(&bars.cleared, 8);
    mbar_init(&bars.drain, 1);
    mbar_init(&bars.ended, 1);
    mbar_init(&bars.asked, 1);
    abort_flag = 0;
    fence_barrier_init();
    mbar_arrive_expect_tx(&bars.ended, sizeof(Copies));
    mbar_arrive_expect_tx(&bars.asked, 4);
    tma_prefetch_desc(&qmap);
    if (p.S > 0) {  // else they are empty
      tma_prefetch_desc(&kmap);
      tma_prefetch_desc(&vmap);
      tma_prefetch_desc(&rmap);
    }
  }
  if (warp == 2) tmem_alloc_pair(&tmem_holder, 512);
  pdl_trigger();
  pdl_wait();
  tc_fence_before();
  __syncthreads();
  cluster_arrive();  // the other CTA's barriers exist
  cluster_wait();
  tc_fence_after();
  const uint32_t tmem = tmem_holder;
  const int nb = p.nope / 64;
  volatile int* stop = &abort_flag;
  auto wait = [&](uint64_t* bar, int phase) {
    return mbar_wait(bar, phase & 1, stop, p.err, p.timeout);
  };
  auto wait_spin = [&](uint64_t* bar, int phase) {
    return mbar_wait_spin(bar, phase & 1, stop, p.err, p.timeout);
  };
  // ... for what the other CTA's threads have written or read
  auto wait_cluster = [&](uint64_t* bar, int phase) {
    return mbar_wait_cluster(bar, phase & 1, stop, p.err, p.timeout);
  };
  auto first = [&](uint64_t* bar) { return map_to_rank(smem_u32(bar), 0); };  // in the first CTA
  // the pair's unit number i, read by every role; false: there is none, or a wait ran out
  auto next_unit = [&](int i, Unit& u) {
    if (!wait(&bars.unit_full[i & 1], i >> 1)) return false;
    u = units[i & 1];
    return u.last == 0;
  };
  auto unit_read = [&](int i) { mbar_arrive(&bars.unit_empty[i & 1]); };

  if (warp == 3) {
    // ------------------------------------------------ units
    // The next one is asked for when this one's copies are issued, not earlier: other pairs may be
    // free first.  Numbers without tiles and queries are passed over.
    Place place;
    auto unit_of = [&](uint32_t x) {  // by groups of heads; in a group a number's heads side by side
      uint32_t at = x >> 1, h0 = 0, heads = p.H;
      if (p.side < p.H) {
        const uint32_t span = gridDim.x / (2 * heads) * p.side, group = at / span;
        at -= group * span;
        h0 = group * p.side;
        heads = min(p.side, p.H - h0);
      }
      const uint32_t number = at / heads;
      return find_unit(p, number, h0 + at - number * heads, place);
    };
    Unit u = unit_of(blockIdx.x);
    bool ok = true, more = true;
    int k = 0, armed = 0;  // answers that have come, that were waited for
    for (int i = 0; more; ++i) {
      if (i > 0) ok = wait(&bars.loaded, i - 1);
      while (ok && more && (i > 0 || u.n == 0)) {
        uint64_t* bar = &bars.next_full[k & 1];
        if (rank == 0 && k > 0) ok = wait_cluster(&bars.next_read, k - 1);
        if (!__all_sync(0xFFFFFFFFu, ok)) break;
        if (lane == 0) {
          mbar_arrive_expect_tx(bar, 16);
          if (rank == 0) ask_next(&answers[k & 1], bar);
        }
        armed = k + 1;
        __syncwarp();
        ok = __all_sync(0xFFFFFFFFu, wait(bar, k >> 1));
        if (!ok) break;
        int x;
        more = read_next(&answers[k & 1], x);
        fence_proxy_async_shared();
        __syncwarp();
        if (rank == 1 && lane == 0) mbar_arrive_cluster_release(first(&bars.next_read));
        ++k;
        if (more) {
          u = unit_of(x);
          if (u.n > 0) break;
        }
      }
      ok = __all_sync(0xFFFFFFFFu, ok && wait(&bars.unit_empty[i & 1], (i >> 1) + 1));
      if (!ok) break;
      u.last = !more;
      if (lane == 0) {
        units[i & 1] = u;
        mbar_arrive(&bars.unit_full[i & 1]);
      }
      __syncwarp();
    }
    // No answer to the pair is on its way past this point: after a wait that ran out the last one
    // may not have come, and the second CTA may not know of it.
    int none = 0, asked = armed;
    if (rank == 0) {
      if (lane == 0)
        st_async_u32(map_to_rank(smem_u32(&questions), 1), asked,
                     map_to_rank(smem_u32(&bars.asked), 1));
    } else {
      asked = 0;
      if (mbar_wait_cluster(&bars.asked, 0, &none, p.err, 3 * p.timeout))
        asked = static_cast<int>(questions);
      asked = __shfl_sync(0xFFFFFFFFu, asked, 0);
      if (asked > armed && lane == 0) mbar_arrive_expect_tx(&bars.next_full[k & 1], 16);
      __syncwarp();
    }
    if (asked > k) mbar_wait(&bars.next_full[k & 1], (k >> 1) & 1, &none, p.err, p.timeout);
    __syncwarp();
  } else if (warp == 0) {
    if (elect_one()) {
      // ---------------------------------------------- copies
      int nq[2] = {0, 0};  // tiles of queries so far
      int g = 0;           // tiles of keys
      int it = 0;          // keys of tile it / 2, then its values
      uint32_t lasts = 0, odd = 0;  // stages that have had a ragged last tile; an odd number of them
      uint32_t alone = 0;           // ... whose last tile was one
      // the second CTA stops a tile behind the first, so that its copies beyond the first one's own
      // are met too
      const int stall = p.stall > 0 ? min(p.stall, 0x7FFFFFFE) + rank : 0x7FFFFFFF;
      bool ok = true;
      Unit u;
      for (int i = 0; ok && next_unit(i, u); ++i) {
        unit_read(i);
        if (g >= stall) break;
        const int nt = u.nt;
        const bool ragged = nt * KEYS > u.len;
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          if ((w ? u.split ? 0 : u.tiles1 : u.tiles0) <= 0 || !ok) continue;
          ok = wait(&bars.q_empty[w], nq[w] + 1);
          if (!ok) break;
          ++nq[w];
          if (rank == 0) mbar_arrive_expect_tx(&bars.q_full[w], 2 * (nb + 1) * BOX);
          for (int c = 0; c <= nb; ++c)
            tma_load_3d_pair(qs + (w * Q_BOXES + c) * BOX, &qmap, first(&bars.q_full[w]), c * 64,
                             u.h, u.q0 + u.r0 + (2 * w + rank) * ROWS);
        }
        for (int t = 0; t < nt && ok; ++t, ++g) {
          if (g >= stall) ok = false;
          if (!ok) break;
          const int st = g % STAGES, row = u.k0 + t * KEYS;
          uint8_t* dst = ring + st * STAGE;
          ok = wait(&bars.k_empty[st], g / STAGES + 1);
          if (!ok) break;
          if (rank == 0) mbar_arrive_expect_tx(&bars.k_full[st], (nb + 1) * BOX);
          const uint32_t bar = first(&bars.k_full[st]);
          for (int c = 0; c < nb; ++c)
            tma_load_3d_pair(dst + c * (BOX / 2), &kmap, bar, c * 64, u.h, row + rank * (KEYS / 2));
          tma_load_3d_pair(dst + nb * (BOX / 2), &rmap, bar, 0, 0, row + rank * (KEYS / 2));
          ++it;
          ok = wait(&bars.v_empty[st], g / STAGES + 1);
          if (!ok) break;
          if (ragged && t == nt - 1) {
            lasts |= 1u << st;
            odd ^= 1u << st;
            alone |= 1u << st;
            mbar_arrive_expect_tx(&bars.v_last[st], BOX);
            tma_load_3d(dst + K_BYTES, &vmap, &bars.v_last[st], rank * 64, u.h, row);
            if (rank == 0) mbar_arrive(&bars.v_full[st]);  // a phase without bytes
          } else {
            alone &= ~(1u << st);
            if (rank == 0) mbar_arrive_expect_tx(&bars.v_full[st], 2 * BOX);
            tma_load_3d_pair(dst + K_BYTES, &vmap, first(&bars.v_full[st]), rank * 64, u.h, row);
          }
          ++it;
        }
        mbar_arrive(&bars.loaded);
      }
      // No copy of the pair is in flight past this point.  Each CTA waits for the values that were
      // signalled to it alone, and the first one for all else, that too which the second has issued
      // beyond the first one's own after a wait that ran out.  This is a tile at most for each place
      // in shared memory: what comes there next waits for products that lack the first CTA's part.
      int none = 0;
      for (int st = 0; st < STAGES; ++st)
        if (lasts >> st & 1)
          mbar_wait(&bars.v_last[st], (odd >> st & 1) ^ 1, &none, p.err, p.timeout);
      auto landed = [&](int j, int* stop) {
        const int t = j >> 1;
        mbar_wait(j & 1 ? &bars.v_full[t % STAGES] : &bars.k_full[t % STAGES], (t / STAGES) & 1,
                  stop, p.err, p.timeout);
      };
      if (rank == 0) {
#pragma unroll
        for (int w = 0; w < 2; ++w)
          if (nq[w] > 0) mbar_wait(&bars.q_full[w], (nq[w] - 1) & 1, &none, p.err, p.timeout);
        for (int j = max(0, it - 2 * STAGES); j < it; ++j) landed(j, &none);
        // its waits are bounded and began before this CTA's last ones ended
        int late = 0;
        if (mbar_wait_cluster(&bars.ended, 0, &late, p.err, 3 * p.timeout)) {
          const Copies second = copies;
#pragma unroll
          for (int w = 0; w < 2; ++w)
            if (static_cast<int>(second.queries[w]) > nq[w]) {
              mbar_arrive_expect_tx(&bars.q_full[w], (nb + 1) * BOX);
              mbar_wait(&bars.q_full[w], nq[w] & 1, &late, p.err, p.timeout);
            }
          for (; it < static_cast<int>(second.it); ++it) {
            const int st = (it >> 1) % STAGES;
            if ((it & 1) && (second.alone >> st & 1)) continue;
            if (it & 1)
              mbar_arrive_expect_tx(&bars.v_full[st], BOX);
            else
              mbar_arrive_expect_tx(&bars.k_full[st], (nb + 1) * (BOX / 2));
            landed(it, &late);
          }
        }
      } else {
        const uint32_t to = first(reinterpret_cast<uint64_t*>(&copies)), bar = first(&bars.ended);
        st_async_u32(to, it, bar);
        st_async_u32(to + 4, nq[0], bar);
        st_async_u32(to + 8, nq[1], bar);
        st_async_u32(to + 12, alone, bar);
      }
    }
  } else if (warp == 1 && rank == 0) {
    if (elect_one()) {
      // ---------------------------------------------- products
      constexpr uint32_t sdesc = idesc_make(1, 256, 128);
      constexpr uint32_t vdesc = idesc_make(1, 256, 128) | IDESC_B_MN;  // values of 64 columns too
      bool ok = true;
      int g = 0, nl = 0;         // tiles of keys before this unit; ragged units
      int nq0 = 0, nq1 = 0;      // tiles of queries
      int no0 = 0, no1 = 0;      // results
      int n0 = 0, n1 = 0;        // their tiles of keys
      // of tile t of keys with tile q of queries, for group w; the last user hands the stage back
      auto scores = [&](int w, int q, int t, bool wanted, bool last, bool q_last) {
        const int st = (g + t) % STAGES;
        if (wanted) ok = wait(&bars.k_full[st], (g + t) / STAGES);
        if (!ok) return;
        tc_fence_after();
        const uint64_t qa = sdesc_sw128(smem_u32(qs + q * Q_BOXES * BOX)),
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
        if (q_last) tc_commit_pair(&bars.q_empty[q], 3);
      };
      // ... tile i of the group's
      auto values = [&](int w, int t, int i, int tiles_before, int before, bool wanted, bool last,
                        bool tail) {
        const int st = (g + t) % STAGES;
        if (wanted)
          ok = wait(&bars.v_full[st], (g + t) / STAGES) &&
               (!tail || wait_cluster(&bars.cleared, nl));
        ok = ok && wait_spin(&bars.p_half[w], tiles_before + i) &&
             (i > 0 || wait(&bars.o_free[w], before + 1));
        if (!ok) return;
        tc_fence_after();
        const uint64_t va = sdesc_sw128_mn(smem_u32(ring + st * STAGE + K_BYTES), BOX);
        const uint32_t d = tmem + 256 + w * 128, a = tmem + w * 128;
        mma4_pair_ta(d, a, va, vdesc, i);
        tc_commit_pair(&bars.pv_half[w], 3);
        ok = wait_spin(&bars.p_full[w], tiles_before + i);
        if (!ok) return;
        tc_fence_after();
        mma4_pair_ta(d, a + 32, va + 512, vdesc, 1);
        tc_commit_pair(&bars.pv_done[w], 3);
        if (last) tc_commit_pair(&bars.v_empty[st], 3);
      };
      Unit u;
      for (int i = 0; ok && next_unit(i, u); ++i) {
        unit_read(i);
        const int t0 = u.tiles0, t1 = u.tiles1, nt = u.nt;
        const bool ragged_last = nt * KEYS > u.len;
        const int split = u.split, q1 = split ^ 1;  // the second group's tile of queries
        auto tile = [&](int w, int i) { return split ? 2 * i + w : i; };
        auto ends = [&](int w, int i, int n) { return split ? tile(w, i) == nt - 1 : i == n - 1; };
        if (t0 > 0) {
          ok = wait(&bars.q_full[0], nq0);
          if (ok) scores(0, 0, 0, true, split || t1 <= 0, ends(0, 0, t0));
        }
        if (t1 > 0 && ok) {
          if (!split) ok = wait(&bars.q_full[1], nq1);
          if (ok) scores(1, q1, split, split || t0 <= 0, true, ends(1, 0, t1));
        }
        for (int i = 0; i < max(t0, t1) && ok; ++i) {
          const int a = tile(0, i), b = tile(1, i), step = 1 + split;
          if (i < t0) values(0, a, i, n0, no0, true, split || i >= t1, ragged_last && a == nt - 1);
          if (ok && i + 1 < t0)
            scores(0, 0, a + step, true, split || i + 1 >= t1, ends(0, i + 1, t0));
          if (ok && i < t1)
            values(1, b, i, n1, no1, split || i >= t0, true, ragged_last && b == nt - 1);
          if (ok && i + 1 < t1)
            scores(1, q1, b + step, split || i + 1 >= t0, true, ends(1, i + 1, t1));
        }
        g += nt;
        nl += ragged_last && nt > 0;
        nq0 += t0 > 0;
        nq1 += t1 > 0 && !split;
        no0 += t0 > 0;
        no1 += t1 > 0;
        n0 += t0;
        n1 += t1;
      }
      tc_commit_pair(&bars.drain, 3);  // no product of the pair runs past this point
    }
  } else if (warp >= 4) {
    // ------------------------------------------------ softmax: a row per thread
    const int w = (warp - 4) >> 2, quad = warp & 3;
    const uint32_t lanes = static_cast<uint32_t>(quad * 32) << 16;
    const uint32_t S = tmem + w * 128 + lanes, O = tmem + 256 + w * 128 + lanes;
    const uint32_t p_half = first(&bars.p_half[w]), p_full = first(&bars.p_full[w]),
                   o_free = first(&bars.o_free[w]);
    int g = 0;          // tiles of keys before this unit
    uint32_t odd = 0;   // stages that have had an odd number of ragged last tiles
    int done = 0;       // this group's tiles before this unit
    int merged = 0;     // units whose keys both groups had
    bool ok = true;
    Unit u;
    for (int i = 0;; ++i) {
      ok = __all_sync(0xFFFFFFFFu, ok && next_unit(i, u));
      if (!ok) break;
      const int nt = u.nt, mine = w ? u.tiles1 : u.tiles0;
      const bool ragged = nt > 0 && nt * KEYS > u.len;
      const int row = u.r0 + ((u.split ? 0 : 2 * w) + rank) * ROWS + quad * 32 + lane;
      const int limit = row >= u.n ? 0 : p.causal ? u.len - (u.n - 1 - row) : u.len;
      float m = -INFINITY, l = 0.f, f;
      // the keys' ragged last tile is cleared by the group whose products with it come last
      const int ragged_at =
          ragged && (u.split ? ((nt - 1) & 1) == w : w == 1) ? mine - 1 : -1;
      int seen = u.split && w ? limit - KEYS : limit;  // keys from the tile's first on
      const int seen_step = u.split ? 2 * KEYS : KEYS;
      for (int j = 0; j < mine; ++j, seen -= seen_step) {
        ok = wait_spin(&bars.s_full[w], done + j);
        ok = __all_sync(0xFFFFFFFFu, ok);
        if (!ok) break;
        tc_fence_after();
        if (j == ragged_at) {
          // what the values hold behind the sequence is cleared: it may not be finite
          const int st = (g + nt - 1) % STAGES;
          ok = wait(&bars.v_last[st], odd >> st & 1);
          ok = __all_sync(0xFFFFFFFFu, ok);
          if (!ok) break;
          uint8_t* vs = ring + st * STAGE + K_BYTES;
          for (int c = (u.len - (nt - 1) * KEYS) * 8 + quad * 32 + lane; c < KEYS * 8; c += 128)
            *reinterpret_cast<uint4*>(vs + c * 16) = make_uint4(0, 0, 0, 0);
          fence_proxy_async_shared();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster_release(first(&bars.cleared));
        }
        // 64 keys at a time, weighted by the maximum in use while their own is found; it may lag by
        // 8, so weights stay below 2^8.  Where it lags by more O and the sum are rescaled and the
        // weights computed once more, from scores that are still in registers.
#pragma unroll 1
        for (int c = 0; c < KEYS; c += 64) {
          uint32_t v[2][32], pk[32];
          load64(S + c, seen - c, v);
          float a, b;
          unsigned long long sum[2];
          float top = weights64(v, p.scale, m, sum, pk);
          if (__any_sync(0xFFFFFFFFu, top > m + 8.f)) {
            const float now = fmaxf(m, top);
            const float f = now == -INFINITY ? 1.f : exp2_fast(m - now);
            m = now;
            l *= f;
            // O holds what came before; the products of the tile before are done (these scores
            // were issued behind them), those of this tile's first half may not be
            if (c > 0) {
              ok = wait(&bars.pv_half[w], done + j);
              ok = __all_sync(0xFFFFFFFFu, ok);
              if (!ok) break;
              tc_fence_after();
            }
            if (j > 0 || c > 0) {
#pragma unroll 1
              for (int o = 0; o < p.value; o += 16) {
                float x[16];
                tmem_ld16(O + o, x);
#pragma unroll
                for (int k = 0; k < 16; ++k) x[k] *= f;
                tmem_st16(O + o, x);
              }
            }
            weights64(v, p.scale, m, sum, pk);
          }
          add2(sum[0], sum[1]);
          unpack2(sum[0], a, b);
          l += a + b;
          tmem_st32(S + c / 2, pk);  // over columns that have been read
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(c == 0 ? p_half : p_full);
        }
        if (!ok) break;
      }
      if (ok && mine > 0) ok = wait(&bars.pv_done[w], done + mine - 1);
      ok = __all_sync(0xFFFFFFFFu, ok);
      if (!ok) break;
      tc_fence_after();
      // the two groups' shares of the keys come together: each takes half of the columns
      const bool both = u.split && u.tiles1 > 0;
      float f2 = 0.f;
      if (both) {
        shares[w][quad * 32 + lane] = make_float2(m, l);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.shared[w]);
        ok = wait(&bars.shared[w ^ 1], merged);
        ok = __all_sync(0xFFFFFFFFu, ok);
        if (!ok) break;
        tc_fence_after();
        const float2 other = shares[w ^ 1][quad * 32 + lane];
        const float now = fmaxf(m, other.x);
        const float a = m == -INFINITY ? 0.f : exp2_fast(m - now);
        f2 = other.x == -INFINITY ? 0.f : exp2_fast(other.x - now);
        l = l * a + other.y * f2;
        m = now;
        f2 = l != 0.f ? f2 / l : 0.f;
        f = l != 0.f ? a / l : 0.f;
      } else {
        f = l != 0.f ? 1.0f / l : 0.f;
      }
      if (row - lane < u.n && (both || !u.split || w == 0)) {
        if (p.lse && row < u.n && !(both && w))
          p.lse[static_cast<int64_t>(u.q0 + row) * p.H + u.h] =
              l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
        // 16 columns at a time; neighbouring lanes swap halves, so that a pair of them stores 32
        // bytes of a row
        __nv_bfloat16* dst = p.out + static_cast<int64_t>(u.q0 + row - (lane & 1)) * p.out_token +
                             static_cast<int64_t>(u.h) * p.out_head + (lane & 1) * 8;
        const bool there0 = row - (lane & 1) < u.n, there1 = row - (lane & 1) + 1 < u.n;
        const int c0 = both && w ? p.value / 2 : 0, c1 = both && !w ? p.value / 2 : p.value;
#pragma unroll 1
        for (int c = c0; c < c1; c += 16) {
          float o[16];
          if (mine > 0) {
            tmem_ld16(O + c, o);
          } else {
#pragma unroll
            for (int k = 0; k < 16; ++k) o[k] = 0.f;
          }
#pragma unroll
          for (int k = 0; k < 16; ++k) o[k] *= f;
          if (both) {
            float o2[16];
            tmem_ld16(tmem + 256 + (w ^ 1) * 128 + lanes + c, o2);
#pragma unroll
            for (int k = 0; k < 16; ++k) o[k] = fmaf(o2[k], f2, o[k]);
          }
          uint32_t x[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) x[k] = l == 0.f ? 0u : pack_bf16(o[2 * k], o[2 * k + 1]);
          uint32_t y[4];
#pragma unroll
          for (int k = 0; k < 4; ++k)
            y[k] = __shfl_xor_sync(0xFFFFFFFFu, lane & 1 ? x[k] : x[k + 4], 1);
          // the even lane's row: its first half from itself, its second goes to the odd lane
          if (there0)
            *reinterpret_cast<uint4*>(dst + c) = lane & 1 ? make_uint4(y[0], y[1], y[2], y[3])
                                                          : make_uint4(x[0], x[1], x[2], x[3]);
          if (there1)
            *reinterpret_cast<uint4*>(dst + p.out_token + c) =
                lane & 1 ? make_uint4(x[4], x[5], x[6], x[7]) : make_uint4(y[0], y[1], y[2], y[3]);
        }
      }
      if (both) {  // ... and neither's result and sums are overwritten before the other has read them
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.shared_read[w]);
        ok = wait(&bars.shared_read[w ^ 1], merged);
        ok = __all_sync(0xFFFFFFFFu, ok);
        if (!ok) break;
        tc_fence_after();
        ++merged;
      }
      if (mine > 0) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(o_free);
      }
      __syncwarp();
      if (lane == 0) unit_read(i);
      g += nt;
      if (ragged) odd ^= 1u << ((g - 1) % STAGES);
      done += mine;
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
  cfg.gridDim = dim3(2 * tiles * p.H);
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
