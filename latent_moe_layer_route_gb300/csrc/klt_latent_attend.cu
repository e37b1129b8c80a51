// Latent attention in absorbed form over a paged cache (sm_103a).
//
// 64 query rows (token, head) against 64 keys at a time: S = Q K^T (M = 64 rows, N = 64 keys),
// softmax in registers, O^T += V^T P^T (M = 128 latent columns, N = rows).  A key's row is its
// value too, so a tile of keys is loaded once and read by both products: K-major by the first,
// with its columns as rows by the second.  O^T rather than O, since 512 columns x 64 rows fill
// half of TMEM that way and the products have M = 128.
//
// Roles: warp 0 copies tiles (two stages of 72 KB in blocks of 128 columns, each handed back on
// its own), warp 1 issues the products of scores and warp 3 those of values (one thread for both
// took longer over its waits and signals than these small products take: 4,000 cycles a tile, for
// 2,000 of work), warp 2 loads the queries and records what the parts are, warps 4 to 11 do the
// softmax (32 of a tile's keys each) and write results.
//
// The work is cut evenly over the SMs, whatever the lengths.  An item (a sequence's row tile, or
// two side by side, a CTA of the group each) that several groups share leaves its parts (O, running
// maximum and sum, fp32) in the workspace, and a second kernel brings them together in order; so
// results do not depend on timing.  Each CTA records what its parts belong to on every call: the
// workspace holds no state between calls.
//
// Weights are rounded to bf16, since the tensor core multiplies them by the cache's bf16 values:
// unnormalised, below 2^8, each by at most 2^-8 of itself.  Scores, maxima, results and the sum that
// divides them, which is that of the unrounded weights, are fp32.  Against 64 bits results are off
// by 0.0017 to 0.0020 (root of squares), 0.0016 to 0.0017 with fp32 weights: what is above is this
// rounding.  Weights in two bf16 parts would double the second product.
//
// What bounds it.  A tile of 512 + 64 columns moves 72 KB from memory (3,130 cycles at an SM's share
// of its rate) and 325 KB through shared memory: 147 KB of operands of the scores, 98 KB of the
// values, 72 KB of the copy, 8 KB of weights, 2,540 cycles at 128 bytes a cycle; with its copies left
// out a tile takes 2,720.  130,001 keys of 64 heads take 47 us (3.2 TB/s; 14 tiles to an SM), 32
// ragged sequences 47 (3.5 TB/s): the stream itself is some 23.  One sequence of 64 heads over all
// SMs takes 8.5 us + 2.0 for each tile of an SM's (2 to 14 of them; 1.65 beyond) without the second
// kernel, which adds 10.4 (20 MB of fp32 parts out to L2 and back).  128 sequences of 128 heads take
// 110 (649 TFLOP/s): two row tiles to a sequence, 60 tiles to an SM, bound by shared memory.  77 keys
// of 16 heads take 9.8, all of it start and end.  Nothing else was it: a quarter of the products of
// scores or values took 7 and 4 us off those 110 (118 then), no exponentials none, keys multicast to
// both row tiles 3 us more, spinning waits none.
#include "klt_latent.cuh"

#include "../../include/klt.h"

namespace klt {
namespace {

constexpr int ROWS = 64, KEYS = 64, STAGES = 2;
constexpr int BOX = KEYS * 128;  // 64 rows x 128 bytes
constexpr int MAX_BOXES = 9;     // of a row: 512 columns and the position part
constexpr int SOFTMAX = 256;     // threads of the softmax: two warps per 16 rows
constexpr int THREADS = 128 + SOFTMAX;
constexpr int SMEM = 1024 + (MAX_BOXES * (1 + STAGES) + 1) * BOX;
constexpr int MIN_TILES = 2;     // a group's least share
constexpr int UNITS = 8;         // joining blocks per part
// What an item costs besides its tiles, in tiles: its queries' copy, its first scores, its results
// (128 x 128 heads: 142 us at 0, 126 at 3 and 4, 127 at 8).
constexpr int EXTRA = 4;
constexpr int JOIN = 128;        // threads of a joining block: a warp to each of four rows' weights
static_assert(2 * UNITS >= ROWS / 4 && JOIN == 4 * 32 && JOIN == 1 << 7, "");
constexpr int MAX_PARTS = 224;   // of an item
static_assert(SMEM <= 232448 - 2048, "shared memory of a block");

// What a part of an item in the workspace belongs to.
struct Record {
  int valid;   // 0: no part here
  int token;   // the sequence's first query
  int row;     // the item's first row in the sequence
  int rows;    // its rows
  int first;   // group of its first part
  int last;    // ... and of its last
  int slot;    // of its first part
  int member;
};
static_assert(sizeof(Record) == 32, "");

struct Space {  // the workspace: 2 slots per CTA
  Record* records;  // [slots]
  float2* ml;       // [ROWS][slots]: maximum (times scale log2 e), sum
  float4* o;        // [slots][ROWS / 4][R]: four rows of a latent column
};
__host__ __device__ inline Space space_of(float* base, int ctas) {
  Space s;
  s.records = reinterpret_cast<Record*>(base);
  s.ml = reinterpret_cast<float2*>(s.records + 2 * ctas);
  s.o = reinterpret_cast<float4*>(s.ml + 2 * ctas * ROWS);
  return s;
}

// One sequence's share of the work.
struct Seq {
  int q0, n, len;
  int supers;     // items: sets of `members` row tiles
  int tiles;      // tiles of keys of each
  KLT_DEV void load(const AttendParams& p, int b) {
    q0 = b;
    int q1 = b + 1;
    if (p.cu_q) range_of(p.cu_q, b, p.T, q0, q1);
    n = q1 - q0;
    len = static_cast<int>(max(0ll, min(static_cast<long long>(p.lens[b]),
                                        static_cast<long long>(p.max_pages) << p.page_log2)));
    const int shift = p.members == 2 ? 7 : 6;  // rows of an item
    supers = (n * p.H + (1 << shift) - 1) >> shift;
    tiles = max(1, (len + KEYS - 1) / KEYS);
  }
  KLT_DEV long long cost() const { return static_cast<long long>(supers) * (tiles + EXTRA); }
};

// a b / c for c <= 2^8 or so, without a 64-bit division where 32 bits hold a b.
KLT_DEV long long share(long long a, int b, int c) {
  const unsigned long long v = static_cast<unsigned long long>(a) * b;
  return v >> 32 ? static_cast<long long>(v / c) : static_cast<uint32_t>(v) / c;
}

// A CTA's part of an item.
struct Piece {
  int b, q0, n, len;
  int row, rows;       // first row of the row tile in the sequence, rows of it (may be 0)
  int t0, t1;          // tiles of keys that some row sees, in this part
  bool whole;          // the item is this CTA's alone
  int slot;            // else: where its part goes
  long long start;     // the item's first tile's place in the flat order
  int tiles;
};
struct Walk {
  long long pos, lo, hi, base;
  int b;
  int first, parts;  // items shared out one by one: the group of this one's first part, its parts
  Seq s;
  KLT_DEV bool next(const AttendParams& p, Piece& w) {
    if (pos >= hi) return false;
    while (pos >= base + s.cost()) {
      base += s.cost();
      s.load(p, ++b);
    }
    // An item is EXTRA units and then its tiles.  A border within the first ones is as good as at
    // the item's start: the group before it stops there, the one behind it starts there.
    const long long local = pos - base;
    const int units = s.tiles + EXTRA;
    const int super = static_cast<int>(local >> 32 ? local / units
                                                   : static_cast<uint32_t>(local) / units);
    const int u = static_cast<int>(local - static_cast<long long>(super) * units);
    const int end = static_cast<int>(min(static_cast<long long>(units), u + (hi - pos)));
    if (end <= EXTRA) return false;
    fill(p, w, super, max(0, u - EXTRA), end - EXTRA);
    pos += end - u;
    return true;
  }
  // The piece of tiles t .. e of an item of this sequence.
  KLT_DEV void fill(const AttendParams& p, Piece& w, int super, int t, int e) const {
    const int member = blockIdx.x & (p.members - 1);
    w.b = b;
    w.q0 = s.q0;
    w.n = s.n;
    w.len = s.len;
    w.row = (super * p.members + member) * ROWS;
    w.rows = max(0, min(ROWS, s.n * p.H - w.row));
    const int last = (w.row + max(w.rows, 1) - 1) / p.H;  // the tile's last query
    const int seen = max(0, s.len - (s.n - 1 - last));
    w.t0 = t;
    w.t1 = max(t, min(e, (seen + KEYS - 1) / KEYS));
    w.whole = t == 0 && e == s.tiles;
    w.slot = 2 * blockIdx.x + (pos == lo ? 0 : 1);  // by its place in this group's share
    w.start = base + static_cast<long long>(super) * (s.tiles + EXTRA) + EXTRA;
    w.tiles = s.tiles;
  }
};

struct Bars {
  uint64_t full[STAGES][5], empty[STAGES][5];  // blocks of a tile: 128 columns; position part
  uint64_t s_full[2], s_empty[2];
  uint64_t p_full, pv_done;  // weights are written; the products that read them are done
  uint64_t o_free;           // O has been read
  uint64_t q_full, q_free;
  uint64_t drain;
};

KLT_DEV float quad_max(float v) {
  v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 1));
  return fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 2));
}
KLT_DEV float quad_sum(float v) {
  v += __shfl_xor_sync(0xFFFFFFFFu, v, 1);
  return v + __shfl_xor_sync(0xFFFFFFFFu, v, 2);
}
// Barrier of the softmax warps; whether any of their threads says so.
KLT_DEV bool softmax_any(bool v) {
  int r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, 1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(static_cast<int>(v)), "n"(SOFTMAX)
      : "memory");
  return r != 0;
}

__global__ void __launch_bounds__(THREADS, 1)
    attend_kernel(const __grid_constant__ CUtensorMap latents,
                  const __grid_constant__ CUtensorMap ropes,
                  const __grid_constant__ CUtensorMap queries, const AttendParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* qs = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  const int NJ = p.R / 128, NB = p.R / 64, KB = NB + 1;
  uint8_t* ks = qs + MAX_BOXES * BOX;
  uint8_t* ps = ks + STAGES * MAX_BOXES * BOX;
  __shared__ Bars bars;
  __shared__ float factor[ROWS];
  __shared__ float tops[2][ROWS];  // of each half of a tile's keys: maxima; at the end sums
  __shared__ int64_t out_at[ROWS];
  __shared__ long long sums[THREADS / 32];
  __shared__ int counts[THREADS / 32], longest[THREADS / 32], needs[THREADS / 32];
  __shared__ long long found_base;
  __shared__ int found_b;
  __shared__ uint32_t tmem_holder;
  __shared__ int abort_flag;
  const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;
  if (tid == 0) {
    for (int s = 0; s < STAGES; ++s)
      for (int i = 0; i < 5; ++i) {
        mbar_init(&bars.full[s][i], 1);
        mbar_init(&bars.empty[s][i], 1);
      }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars.s_full[i], 1);
      mbar_init(&bars.s_empty[i], SOFTMAX / 32);
    }
    mbar_init(&bars.p_full, SOFTMAX / 32);
    mbar_init(&bars.pv_done, 1);
    mbar_init(&bars.o_free, SOFTMAX / 32);
    mbar_init(&bars.q_full, p.q_box ? 1 : 32);
    mbar_init(&bars.q_free, 1);
    mbar_init(&bars.drain, 2);
    abort_flag = 0;
    fence_barrier_init();
    if (p.max_pages > 0) {  // else they may be empty
      tma_prefetch_desc(&latents);
      tma_prefetch_desc(&ropes);
    }
    if (p.q_box) tma_prefetch_desc(&queries);
  }
  if (warp == 1) {
    tmem_alloc(&tmem_holder, 512);
    tmem_relinquish();
  }
  pdl_trigger();
  pdl_wait();

  // The work of all, and this group's share of it.  Where there are fewer items than groups, each
  // item has groups of its own: the smallest share t with sum(ceil(tiles / t)) <= groups is found,
  // twelve candidates at once, a warp each, between W / groups and W / (groups - items) or the
  // longest item, which are always enough.  Else, and where t is above 1.2 equal shares, the tiles of
  // all items in a row are cut into equal shares, and a group may have the end of one item and the
  // start of the next.  That costs some us: 32 ragged sequences of up to 8192 keys take 43.3 by items
  // and 44.8 in equal shares, 130 of 4096 112 and 122.  But items of their own leave groups idle (77
  // of 4096 105 and 80) or a long sequence with one group (130 ragged ones 177 and 122, 150 short ones
  // and one of 30,000 keys 339 and 48).  At 1.2 both take the same (120 of 4096 110 and 115, 110 of
  // them, at 1.3, 109 and 106).
  const int group = blockIdx.x >> (p.members - 1);  // one or two members
  long long W = 0, mine = 0, excl = 0;
  int groups = gridDim.x >> (p.members - 1), items = 0, top = 0;
  Walk walk;
  Piece w;
  bool more = false;  // w is a piece
  {
    constexpr int WARPS = THREADS / 32;
    static_assert(THREADS * sizeof(Seq) <= BOX, "");
    Seq* seqs = reinterpret_cast<Seq*>(ps);  // of one pass over the batch
    Seq s;
    for (int b = tid; b < p.B; b += THREADS) {
      s.load(p, b);
      mine += s.cost();
      items += s.supers;
      if (s.supers > 0) top = max(top, s.tiles);
      seqs[tid] = s;
    }
    // block-wide sum; where one pass covers the batch, also this sequence's place in it
    long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long v = __shfl_up_sync(0xFFFFFFFFu, incl, o);
      if (lane >= o) incl += v;
    }
    items = __reduce_add_sync(0xFFFFFFFFu, items);
    top = __reduce_max_sync(0xFFFFFFFFu, top);
    if (lane == 31) sums[warp] = incl, counts[warp] = items, longest[warp] = top;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    items = 0;
    for (int i = 0; i < WARPS; ++i) {
      if (i == warp) excl = W + incl - mine;
      W += sums[i];
      items += counts[i];
      top = max(top, longest[i]);
    }
    walk.parts = 0;
    walk.pos = walk.lo = walk.hi = 0;
    bool apart = p.B <= THREADS && items < groups;
    int t = 0;
    if (apart) {
      // the tiles, in units of 8 where 32 bits do not hold them
      const long long all = W - static_cast<long long>(items) * EXTRA;
      const int shift = all >> 31 ? 3 : 0;
      const uint32_t sum = static_cast<uint32_t>((all + (1 << shift) - 1) >> shift);
      const uint32_t least = max(static_cast<uint32_t>(MIN_TILES), (sum + groups - 1) / groups);
      const uint32_t most = max(least, min((sum + groups - items - 1) / (groups - items),
                                           (top + (1u << shift) - 1) >> shift));
      auto candidate = [&](int i) {
        return static_cast<int>((least + (most - least) / (WARPS - 1) * i +
                                 (most - least) % (WARPS - 1) * i / (WARPS - 1)) << shift);
      };
      t = candidate(0);
      if (least != most) {  // (one sequence: nothing to search, 0.4 us)
        t = candidate(warp);
        int need = 0;
        for (int b = lane; b < p.B; b += 32)
          need += seqs[b].supers * ((seqs[b].tiles + t - 1) / t);
        need = __reduce_add_sync(0xFFFFFFFFu, need);
        if (lane == 0) needs[warp] = need;
        __syncthreads();
        int i = 0;
        while (i < WARPS - 1 && needs[i] > groups) ++i;
        t = candidate(i);
      }
      apart = 5ll * t * groups <= 6 * W + 10ll * groups;  // or two tiles more than 1.2, if all is short
    }
    if (apart) {
      int before = 0;
      for (int b0 = 0; b0 < p.B; b0 += 32) {
        const bool there = b0 + lane < p.B;
        const int supers = there ? seqs[b0 + lane].supers : 0;
        const int parts = there ? (seqs[b0 + lane].tiles + t - 1) / t : 1;
        int in = supers * parts;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int v = __shfl_up_sync(0xFFFFFFFFu, in, o);
          if (lane >= o) in += v;
        }
        const uint32_t past = __ballot_sync(0xFFFFFFFFu, group < before + in);
        if (past) {
          const int src = __ffs(past) - 1;
          walk.b = b0 + src;
          walk.s = seqs[walk.b];
          walk.base = 0;
          walk.parts = __shfl_sync(0xFFFFFFFFu, parts, src);
          const int at =  // this group's number among the sequence's
              group - before - __shfl_sync(0xFFFFFFFFu, in - supers * parts, src);
          const int super = at / walk.parts, part = at - super * walk.parts;
          walk.first = group - part;
          walk.fill(p, w, super, static_cast<int>(share(walk.s.tiles, part, walk.parts)),
                    static_cast<int>(share(walk.s.tiles, part + 1, walk.parts)));
          more = true;
          break;
        }
        before += __shfl_sync(0xFFFFFFFFu, in, 31);
      }
    } else {
      groups = static_cast<int>(max(1ll, min(static_cast<long long>(groups), W / MIN_TILES)));
      if (group < groups) {
        walk.lo = share(W, group, groups);
        walk.hi = share(W, group + 1, groups);
      }
      if (p.B <= THREADS) {
        if (mine > 0 && walk.lo >= excl && walk.lo < excl + mine) found_b = tid, found_base = excl;
        __syncthreads();
      } else {  // pass by pass
        long long before = 0;
        for (int b0 = 0; b0 < p.B; b0 += THREADS) {
          long long c = 0;
          if (b0 + tid < p.B) {
            s.load(p, b0 + tid);
            c = s.cost();
          }
          long long in = c;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const long long v = __shfl_up_sync(0xFFFFFFFFu, in, o);
            if (lane >= o) in += v;
          }
          __syncthreads();
          if (lane == 31) sums[warp] = in;
          __syncthreads();
          for (int i = 0; i < warp; ++i) in += sums[i];
          in += before;
          if (c > 0 && walk.lo >= in - c && walk.lo < in) found_b = b0 + tid, found_base = in - c;
          for (int i = 0; i < WARPS; ++i) before += sums[i];
        }
        __syncthreads();
      }
      if (walk.lo < walk.hi) {
        walk.b = found_b;
        walk.base = found_base;
        walk.s.load(p, walk.b);
        walk.pos = walk.lo;
        more = walk.next(p, w);
      }
    }
    __syncthreads();  // the weights' memory is free
  }
  const uint32_t tmem = tmem_holder, S = tmem + 256;
  volatile int* stop = &abort_flag;
  const Space ws = space_of(p.part, gridDim.x);
  auto wait = [&](uint64_t* bar, int phase) {
    return mbar_wait(bar, phase & 1, stop, p.err, p.timeout);
  };

  if (warp == 0) {
    // ------------------------------------------------ copies
    if (elect_one()) {
      const int box_log2 = min(p.page_log2, 6), box_keys = 1 << box_log2;
      const int page_mask = (1 << p.page_log2) - 1;
      int it = 0, cut = 0;  // tiles; blocks of the last one, where it was cut short
      bool ok = true;
      for (; ok && more; more = walk.next(p, w)) {
        if (w.rows == 0) continue;
        const int* table = p.table + w.b * p.ld_table;
        auto pages_of = [&](int t, int* page) {
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const int key = t * KEYS + (x << box_log2);
            if (x << box_log2 < KEYS && key < w.len && t < w.t1) page[x] = table[key >> p.page_log2];
          }
        };
        int page[4], ahead[4];
        pages_of(w.t0, ahead);
        for (int t = w.t0; t < w.t1; ++t, ++it) {
          if (p.stall > 0 && it >= p.stall) ok = false;
          if (!ok) break;
#pragma unroll
          for (int x = 0; x < 4; ++x) page[x] = ahead[x];
          pages_of(t + 1, ahead);
          if (it >= STAGES && box_keys == KEYS && page[0] >= 0 && page[0] < p.pages) {
            // into L2 while its stage is still in use (3 % off large batches; small pages take too
            // many of these to gain)
            for (int c = 0; c < NB; c += 2)
              tma_prefetch_4d(&latents, 0, t * KEYS & page_mask, c, page[0]);
            tma_prefetch_3d(&ropes, 0, t * KEYS & page_mask, page[0]);
          }
          const int st = it % STAGES;
          uint8_t* const stage = ks + st * MAX_BOXES * BOX;
          if (box_keys == KEYS) {  // both boxes of 128 columns by one copy
            const int row = t * KEYS & page_mask;
            const int at = page[0] >= 0 && page[0] < p.pages ? page[0] : p.pages;
            for (cut = 0; cut <= NJ; ++cut) {
              ok = wait(&bars.empty[st][cut], (it / STAGES) + 1);
              if (!ok) break;
              uint64_t* full = &bars.full[st][cut];
              mbar_arrive_expect_tx(full, cut < NJ ? 2 * BOX : BOX);
              if (cut < NJ)
                tma_load_4d(stage + 2 * cut * BOX, &latents, full, 0, row, 2 * cut, at);
              else
                tma_load_3d(stage + 2 * cut * BOX, &ropes, full, 0, row, at);
            }
          } else {
            const int boxes = (min(KEYS, w.len - t * KEYS) + box_keys - 1) >> box_log2;
            for (cut = 0; cut <= NJ; ++cut) {
              ok = wait(&bars.empty[st][cut], (it / STAGES) + 1);
              if (!ok) break;
              uint64_t* full = &bars.full[st][cut];
              mbar_arrive_expect_tx(full, boxes * (cut < NJ ? 2 : 1) * (box_keys * 128));
#pragma unroll
              for (int x = 0; x < 4; ++x) {
                if (x >= boxes) break;
                const int row = (t * KEYS + (x << box_log2)) & page_mask;
                const int at = page[x] >= 0 && page[x] < p.pages ? page[x] : p.pages;
                uint8_t* dst = stage + 2 * cut * BOX + x * box_keys * 128;
                if (cut < NJ) {
                  tma_load_4d(dst, &latents, full, 0, row, 2 * cut, at);
                  tma_load_4d(dst + BOX, &latents, full, 0, row, 2 * cut + 1, at);
                } else {
                  tma_load_3d(dst, &ropes, full, 0, row, at);
                }
              }
            }
          }
          if (!ok) break;
          cut = 0;
        }
      }
      // no copy of this CTA is in flight past this point
      int none = 0;
      for (int i = 0; i <= NJ; ++i)
        for (int s = 0; s < STAGES; ++s) {
          const int j = (i < cut ? it : it - 1) - s;
          if (j >= 0)
            mbar_wait(&bars.full[j % STAGES][i], (j / STAGES) & 1, &none, p.err, p.timeout);
        }
    }
  } else if (warp == 1) {
    // ------------------------------------------------ scores
    if (elect_one()) {
      int it = 0, piece = 0;  // tiles; pieces with rows and tiles
      bool ok = true;
      const uint32_t qa = smem_u32(qs);
      for (; ok && more; more = walk.next(p, w)) {
        if (w.rows == 0 || w.t0 == w.t1) continue;
        ok = wait(&bars.q_full, piece++);
        for (int t = w.t0; t < w.t1 && ok; ++t, ++it) {
          const int st = it % STAGES, buf = it & 1;
          const uint32_t ka = smem_u32(ks + st * MAX_BOXES * BOX), d = S + buf * 64;
          ok = wait(&bars.s_empty[buf], (it >> 1) + 1);
          for (int j = 0; j < NJ && ok; ++j) {
            ok = wait(&bars.full[st][j], it / STAGES);
            if (!ok) break;
            tc_fence_after();
            const uint64_t qd = sdesc_sw128(qa + 2 * j * BOX), kd = sdesc_sw128(ka + 2 * j * BOX);
            mma4_bf16(d, qd, kd, idesc_make(1, 64, 64), j);
            mma4_bf16(d, qd + BOX / 16, kd + BOX / 16, idesc_make(1, 64, 64), 1);
          }
          ok = ok && wait(&bars.full[st][NJ], it / STAGES);
          if (!ok) break;
          tc_fence_after();
          const uint64_t qd = sdesc_sw128(qa + NB * BOX), kd = sdesc_sw128(ka + NB * BOX);
          if (p.rope == 64)
            mma4_bf16(d, qd, kd, idesc_make(1, 64, 64), 1);
          else
            for (int s = 0; s < p.rope / 16; ++s)
              mma_bf16(d, qd + 2 * s, kd + 2 * s, idesc_make(1, 64, 64), 1);
          tc_commit(&bars.s_full[buf]);
          tc_commit(&bars.empty[st][NJ]);
        }
        if (ok) tc_commit(&bars.q_free);
      }
      tc_commit(&bars.drain);  // none of this thread's products runs past this point
      int none = 0;
      mbar_wait(&bars.drain, 0, &none, p.err, 3 * p.timeout);
    }
  } else if (warp == 3) {
    // ------------------------------------------------ values
    if (elect_one()) {
      int it = 0, piece = 0;
      bool ok = true;
      const uint64_t pd = sdesc_sw128(smem_u32(ps));
      for (; ok && more; more = walk.next(p, w)) {
        if (w.rows == 0 || w.t0 == w.t1) continue;
        const uint32_t idesc = idesc_make(1, 128, (w.rows + 15) & ~15) | IDESC_A_MN;
        ++piece;
        for (int t = w.t0; t < w.t1; ++t, ++it) {
          const int st = it % STAGES;
          ok = wait(&bars.p_full, it) && (t > w.t0 || wait(&bars.o_free, piece));
          if (!ok) break;
          tc_fence_after();
          const uint64_t va = sdesc_sw128_mn(smem_u32(ks + st * MAX_BOXES * BOX), BOX);
          for (int j = 0; j < NJ; ++j) {
            mma4_bf16_mn(tmem + j * 64, va + j * (2 * BOX / 16), pd, idesc, t > w.t0);
            tc_commit(&bars.empty[st][j]);
          }
          tc_commit(&bars.pv_done);
        }
      }
      tc_commit(&bars.drain);
      int none = 0;
      mbar_wait(&bars.drain, 0, &none, p.err, 3 * p.timeout);
    }
  } else if (warp == 2) {
    // ------------------------------------------------ queries
    int piece = 0, tiles = 0;  // pieces so far; tiles of the last one
    bool ok = true, left[2] = {false, false};
    for (; more; more = walk.next(p, w)) {
      if (w.rows == 0) continue;
      if (!w.whole) {  // record what the part belongs to
        left[0] = left[0] || !(w.slot & 1);
        left[1] = left[1] || (w.slot & 1);
        if (lane == 31) {
          Record r;
          r.valid = 1;
          r.token = w.q0;
          r.row = w.row;
          r.rows = w.rows;
          r.member = blockIdx.x & (p.members - 1);
          if (walk.parts > 0) {
            r.first = walk.first;
            r.last = walk.first + walk.parts - 1;
          } else {
            r.first = static_cast<int>(((w.start + 1) * groups - 1) / W);
            r.last = static_cast<int>(((w.start + w.tiles) * groups - 1) / W);
          }
          r.slot = 2 * (r.first * p.members + r.member) +
                   (walk.parts > 0 || share(W, r.first, groups) >= w.start - EXTRA ? 0 : 1);
          ws.records[w.slot] = r;
        }
      }
      if (!ok || w.t0 == w.t1) continue;
      // until the piece before is through, however long it is
      ok = mbar_wait(&bars.q_free, (piece + 1) & 1, stop, p.err, p.timeout + tiles * TILE_CYCLES);
      ok = __all_sync(0xFFFFFFFFu, ok);
      tiles = w.t1 - w.t0;
      if (!ok) continue;
      ++piece;
      if (p.q_box) {
        if (lane == 0) {
          mbar_arrive_expect_tx(&bars.q_full, KB * BOX);
          for (int r = 0; r < ROWS; r += p.q_box) {
            // rows past the item are other queries' or lie outside: their scores are masked
            const int row = w.row + r, t = w.q0 + row / p.H, h = row % p.H;
            const int at = p.q_packed ? w.q0 * p.H + row : h;
            for (int c = 0; c < KB; ++c)
              tma_load_3d(qs + c * BOX + r * 128, &queries, &bars.q_full, c * 64, at,
                          p.q_packed ? 0 : t);
          }
        }
        continue;
      }
      // a row at a time, lanes neighbouring chunks of 8; all copies are in flight at once (some 7 us
      // where a bulk copy takes 2)
      const int chunks = (p.R + p.rope) >> 3;
      for (int r = 0; r < ROWS; ++r) {
        const int row = w.row + r;
        const bool there = r < w.rows;
        const int t = there ? row / p.H : 0, h = there ? row - t * p.H : 0;
        const __nv_bfloat16* src =
            p.q + static_cast<int64_t>(w.q0 + t) * p.q_token + static_cast<int64_t>(h) * p.q_head;
        for (int c = lane; c < KB * 8; c += 32) {
          const bool inside = there && c < chunks;
          cp_async16(qs + (c >> 3) * BOX + r * 128 + (((c & 7) ^ (r & 7)) << 4),
                     inside ? src + c * 8 : p.q, inside ? 16 : 0);
        }
      }
      cp_async_wait();
      fence_proxy_async_shared();
      mbar_arrive(&bars.q_full);
    }
    if (lane == 31) {
      if (!left[0]) ws.records[2 * blockIdx.x].valid = 0;
      if (!left[1]) ws.records[2 * blockIdx.x + 1].valid = 0;
    }
    int none = 0;
    if (piece > 0 && p.q_box && lane == 0)  // no copy is in flight past this point
      mbar_wait(&bars.q_full, (piece - 1) & 1, &none, p.err, p.timeout);
  } else {
    // ------------------------------------------------ softmax and results
    // This warp: rows 16 quad .. + 15 of the scores, keys 32 half .. + 31 of a tile; of O^T latent
    // columns 32 quad .. + 31 of every 128, those of every second 128 or rows.
    const int quad = warp & 3, half = (warp - 4) >> 2, st = tid - 128;
    const uint32_t lanes = static_cast<uint32_t>(quad * 32) << 16;
    const int r0 = quad * 16 + (lane >> 2);  // this thread's rows: r0 and r0 + 8
    int it = 0;
    bool ok = true;
    for (; more; more = walk.next(p, w)) {
      if (w.rows == 0) continue;
      int limit[2];
      float m[2], l[2] = {0.f, 0.f};
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = r0 + 8 * i;
        limit[i] = r < w.rows ? w.len - (w.n - 1 - (w.row + r) / p.H) : 0;
        m[i] = -INFINITY;
      }
      if (st < ROWS) {
        const int row = w.row + st, t = row / p.H;
        out_at[st] = (w.q0 + t) * p.out_token + (row - t * p.H) * p.out_head;
      }
      for (int t = w.t0; t < w.t1; ++t, ++it) {
        const int buf = it & 1, first = t * KEYS + half * 32;
        // a warp that gave up still meets the others' barriers
        ok = ok && wait(&bars.s_full[buf], it >> 1);
        ok = __all_sync(0xFFFFFFFFu, ok);
        float v[16];
        if (ok) {
          tc_fence_after();
          tmem_ld_rows16(S + buf * 64 + half * 32 + lanes, v);
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars.s_empty[buf]);
        } else {
#pragma unroll
          for (int i = 0; i < 16; ++i) v[i] = 0.f;
        }
        // The maximum in use may lag by 2^8: weights stay below that, and O is rarely rescaled.
        // Either half of the keys can make it grow, so the halves' maxima and the vote share one
        // barrier.  They are read only where there is a second barrier behind.
        float top[2];
        bool grows = false;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (first + 32 > limit[i]) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
              if (first + 8 * (e >> 1) + 2 * (lane & 3) + (e & 1) >= limit[i])
                v[4 * (e >> 1) + 2 * i + (e & 1)] = -INFINITY;
          }
          float x = -INFINITY;
#pragma unroll
          for (int e = 0; e < 8; ++e) x = fmaxf(x, v[4 * (e >> 1) + 2 * i + (e & 1)]);
          top[i] = quad_max(x) * p.scale;
          grows = grows || top[i] > m[i] + 8.f;
          if ((lane & 3) == 0) tops[half][r0 + 8 * i] = top[i];
        }
        const bool rescale = softmax_any(grows);
        if (ok && w.len - t * KEYS < KEYS) {  // rows behind the last token hold anything
          uint8_t* vs = ks + (it % STAGES) * MAX_BOXES * BOX;
          for (int r = w.len - t * KEYS + (warp - 4); r < KEYS; r += SOFTMAX / 32)
            for (int c = lane; c < NB * 8; c += 32)
              *reinterpret_cast<uint4*>(vs + (c >> 3) * BOX + r * 128 + ((c & 7) << 4)) =
                  make_uint4(0, 0, 0, 0);
        }
        // the products of the tile before have read the weights
        ok = ok && wait(&bars.pv_done, it + 1);
        ok = __all_sync(0xFFFFFFFFu, ok);
        if (rescale) {  // O's columns are all warps' rows
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float now = fmaxf(m[i], fmaxf(top[i], tops[half ^ 1][r0 + 8 * i]));
            const float f = now == -INFINITY ? 1.f : exp2_fast(m[i] - now);
            l[i] *= f;
            m[i] = now;
            if (half == 0 && (lane & 3) == 0) factor[r0 + 8 * i] = f;
          }
          softmax_any(false);
          if (t > w.t0 && ok) {
            tc_fence_after();
#pragma unroll 1
            for (int c = half * 16; c < NJ * 64; c += 32) {
              float o[16];
              tmem_ld16(tmem + lanes + c, o);
#pragma unroll
              for (int i = 0; i < 16; ++i) o[i] *= factor[(c & 63) + i];
              tmem_st16(tmem + lanes + c, o);
            }
            tmem_wait_st();
          }
        }
        if (!ok) continue;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float base = m[i] == -INFINITY ? 0.f : m[i];
          uint8_t* row = ps + (r0 + 8 * i) * 128 + (lane & 3) * 4;
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            const float a = exp2_fast(fmaf(v[4 * g + 2 * i], p.scale, -base)),
                        c = exp2_fast(fmaf(v[4 * g + 2 * i + 1], p.scale, -base));
            l[i] += a + c;
            *reinterpret_cast<uint32_t*>(row + (((4 * half + g) ^ (r0 & 7)) << 4)) =
                pack_bf16(a, c);
          }
        }
        fence_proxy_async_shared();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.p_full);
      }
      // the part's result
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        l[i] = quad_sum(l[i]);
        if ((lane & 3) == 0) tops[half][r0 + 8 * i] = l[i];
      }
      softmax_any(false);
      if (half == 0 && (lane & 3) == 0) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int r = r0 + 8 * i;
          const float sum = l[i] + tops[1][r];
          factor[r] = !w.whole ? 1.f : sum != 0.f ? 1.0f / sum : 0.f;
          if (!w.whole) {
            ws.ml[r * 2 * gridDim.x + w.slot] = make_float2(m[i], sum);
          } else if (p.lse && r < w.rows) {
            p.lse[static_cast<int64_t>(w.q0) * p.H + w.row + r] =
                sum == 0.f ? -INFINITY : (m[i] + log2f(sum)) * 0.6931471805599453f;
          }
        }
      }
      if (ok && w.t0 < w.t1) ok = wait(&bars.pv_done, it - 1);
      ok = __all_sync(0xFFFFFFFFu, ok);
      if (softmax_any(!ok)) {
        ok = false;
        continue;
      }
      tc_fence_after();
#pragma unroll 1
      for (int c = half * 16; c < NJ * 64; c += 32) {
        const int col = (c >> 6) * 128 + quad * 32 + lane, r = c & 63;
        if (r >= w.rows) continue;
        float o[16];
        if (w.t0 < w.t1) {
          tmem_ld16(tmem + lanes + c, o);
        } else {
#pragma unroll
          for (int i = 0; i < 16; ++i) o[i] = 0.f;
        }
        if (w.whole) {
          // eight rows' factors and places first: read between the stores, ahead of which the
          // compiler cannot move them, they were one latency behind the other (16 rows of 512
          // columns 5,400 cycles, now 2,300)
#pragma unroll
          for (int i = 0; i < 16; i += 8) {
            __nv_bfloat16* dst[8];
            __nv_bfloat16 v[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const float f = factor[r + i + k];
              dst[k] = p.out + out_at[r + i + k] + col;
              v[k] = __float2bfloat16(f == 0.f ? 0.f : o[i + k] * f);
            }
#pragma unroll
            for (int k = 0; k < 8; ++k)
              if (r + i + k < w.rows) *dst[k] = v[k];
          }
        } else if (w.t0 < w.t1) {
          float4* dst = ws.o + static_cast<int64_t>(w.slot * (ROWS / 4) + (r >> 2)) * p.R + col;
#pragma unroll
          for (int i = 0; i < 4; ++i)
            dst[i * p.R] = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
        }
      }
      if (w.t0 < w.t1) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.o_free);
      }
      softmax_any(false);  // factor, tops and out_at are free
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Brings an item's parts together: weights 2^(m_i - M) per row and part, with M the largest maximum,
// and the sum of weighted O over the sum of weighted sums.  Four rows of the item and some of their
// columns are a block's, eight blocks to a part, so a thread has some eight loads however many parts
// there are: of several columns where the parts are few, of one column, shared by several threads,
// where they are many.  The first go out before the weights are known.  Lean on purpose: with
// divisions and 64-bit addresses per load this was bound by its instructions (11 us for 152 parts of
// 64 x 512, 20 MB; now 6 to 8).
__global__ void __launch_bounds__(JOIN, 8)
    join_kernel(const AttendParams p, int ctas) {
  __shared__ float4 weight[MAX_PARTS], inverse;
  __shared__ int64_t out_at[4];
  pdl_trigger();
  pdl_wait();
  const Space ws = space_of(p.part, ctas);
  const int cta = blockIdx.x;
  const Record rec = ws.records[2 * cta + blockIdx.z];
  if (!rec.valid) return;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int parts = rec.last - rec.first + 1;
  const int unit = ((cta >> (p.members - 1)) - rec.first) * UNITS + blockIdx.y;
  const int four = unit & (ROWS / 4 - 1), chunk = unit / (ROWS / 4);
  const int chunks = parts * UNITS / (ROWS / 4);  // >= 1: at least two parts
  const int per = (p.R + chunks - 1) / chunks;    // columns of a block
  const int c0 = chunk * per, c1 = min(p.R, c0 + per);
  if (chunk >= chunks || c0 >= c1 || four * 4 >= rec.rows) return;
  // threads that share a column's parts: a power of two, so that the block's columns just fit
  const int step_log2 = per >= JOIN ? 7 : max(2, 32 - __clz(per - 1));
  const int split = JOIN >> step_log2, step = 1 << step_log2;
  const int mine = tid & (split - 1), first = c0 + (tid >> (7 - step_log2));
  // part i is in slot 2 CTA of its group, the first one perhaps in the slot behind
  const int cta0 = rec.first * p.members + rec.member;
  const int64_t part_step = static_cast<int64_t>(2 * p.members) * (ROWS / 4) * p.R;
  const float4* const o0 = ws.o + (2 * cta0 * (ROWS / 4) + four) * static_cast<int64_t>(p.R);
  const int64_t odd = static_cast<int64_t>(rec.slot & 1) * (ROWS / 4) * p.R;
  float4 v[2][4];
  auto load = [&](int c, int i) {  // two columns, four parts
#pragma unroll
    for (int k = 0; k < 4; ++k, i += split) {
      if (i >= parts) break;
      const float4* src = o0 + i * part_step + (i == 0 ? odd : 0);
      if (c < c1) v[0][k] = src[c];
      if (c + step < c1) v[1][k] = src[c + step];
    }
  };
  load(first, mine);
  {
    const int row = four * 4 + warp;  // this warp's row
    const float2* ml = ws.ml + (row * 2 * ctas + 2 * cta0);
    float* const weights = reinterpret_cast<float*>(weight) + warp;
    float top = -INFINITY, sum = 0.f;
    float2 x[MAX_PARTS / 32];
#pragma unroll
    for (int j = 0; j < MAX_PARTS / 32; ++j) {
      if (j * 32 >= parts) break;
      const int i = j * 32 + lane;
      x[j] = make_float2(-INFINITY, 0.f);
      if (i < parts) x[j] = ml[i == 0 ? rec.slot & 1 : i * 2 * p.members];
    }
#pragma unroll
    for (int j = 0; j < MAX_PARTS / 32; ++j) {
      if (j * 32 >= parts) break;
      top = fmaxf(top, x[j].x);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
#pragma unroll
    for (int j = 0; j < MAX_PARTS / 32; ++j) {
      if (j * 32 >= parts) break;
      const float f = x[j].x == -INFINITY ? 0.f : exp2_fast(x[j].x - top);
      sum += x[j].y == 0.f ? 0.f : f * x[j].y;
      if (j * 32 + lane < parts) weights[(j * 32 + lane) * 4] = f;
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    if (lane == 0) {
      const int r = rec.row + row, t = r / p.H;
      out_at[warp] = row < rec.rows
                         ? (rec.token + t) * p.out_token + (r - t * p.H) * p.out_head
                         : -1;
      reinterpret_cast<float*>(&inverse)[warp] = sum != 0.f ? 1.0f / sum : 0.f;
      if (p.lse && chunk == 0 && row < rec.rows)
        p.lse[static_cast<int64_t>(rec.token) * p.H + r] =
            sum == 0.f ? -INFINITY : (top + log2f(sum)) * 0.6931471805599453f;
    }
  }
  __syncthreads();
#pragma unroll 1
  for (int c = first; c - (tid >> (7 - step_log2)) < c1; c += 2 * step) {
    float acc[2][4] = {};
#pragma unroll 1
    for (int i0 = mine; i0 - mine < parts; i0 += 4 * split) {
      if (c != first || i0 != mine) load(c, i0);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int i = i0 + k * split;
        if (i >= parts) break;
        const float4 f = weight[i];
        const float w[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          if (c + n * step >= c1) break;
          const float x[4] = {v[n][k].x, v[n][k].y, v[n][k].z, v[n][k].w};
#pragma unroll
          for (int r = 0; r < 4; ++r)  // a part in which a row sees no key may have left no O
            acc[n][r] = w[r] == 0.f ? acc[n][r] : fmaf(w[r], x[r], acc[n][r]);
        }
      }
    }
    for (int d = split >> 1; d; d >>= 1)
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          acc[n][r] += __shfl_down_sync(0xFFFFFFFFu, acc[n][r], d, split);
    if (mine == 0) {
      const float inv[4] = {inverse.x, inverse.y, inverse.z, inverse.w};
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (out_at[r] >= 0) {
          __nv_bfloat16* out = p.out + out_at[r] + c;
          if (c < c1) out[0] = __float2bfloat16(acc[0][r] * inv[r]);
          if (c + step < c1) out[step] = __float2bfloat16(acc[1][r] * inv[r]);
        }
    }
  }
}

}  // namespace

uint64_t attend_workspace(int num_sms, int latent) {
  return 2ull * num_sms * (sizeof(Record) + 2 * ROWS * 4 + ROWS * 4ull * latent);
}

bool prepare_attend() {
  return cudaFuncSetAttribute(attend_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM) ==
         cudaSuccess;
}

cudaError_t launch_attend(const CUtensorMap& latents, const CUtensorMap& ropes,
                          const CUtensorMap& queries, AttendParams p, int num_sms,
                          cudaStream_t s) {
  // Two row tiles of a sequence side by side read the same keys at the same time, the second from
  // L2: 128 sequences of 4096 keys and 128 heads take 185 us, 212 one by one (up to 72 sequences:
  // the same).  But where a sequence has an odd number of tiles a CTA stands idle (one to each of 32
  // sequences: 61.5 us, 42.7 one by one; three to each of 128: 360, 303).  The numbers of queries
  // are on the device, so two it is where every number makes an even one, or where all sequences
  // seem to have the same.
  const int64_t each = static_cast<int64_t>(p.T / p.B) * p.H;
  const bool even = p.H % (2 * ROWS) == 0 || (p.T % p.B == 0 && (each + ROWS - 1) / ROWS % 2 == 0);
  p.members = even ? 2 : 1;
  // at most as many items and parts of one as the sizes allow, whatever the lengths are
  const int64_t per = ROWS * p.members, rows = static_cast<int64_t>(p.T) * p.H;
  const int64_t items = p.cu_q ? rows / per + min(p.B, p.T) : p.B * ((p.H + per - 1) / per);
  const int64_t tiles = ((static_cast<int64_t>(p.max_pages) << p.page_log2) + KEYS - 1) / KEYS;
  const int64_t parts = max(int64_t{1}, (tiles + MIN_TILES - 1) / MIN_TILES);
  int groups = min(num_sms, MAX_PARTS) / p.members;
  const bool by_items = p.B <= THREADS && items < groups;
  if (by_items && items * parts < groups) groups = static_cast<int>(max(items * parts, items + 1));
  const int ctas = groups * p.members;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = SMEM;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, attend_kernel, latents, ropes, queries, p);
  if (e != cudaSuccess || (by_items && parts == 1)) return e;
  // Where groups are seven times the items no share is above 7/6 of an equal one and a tile: the items
  // have groups of their own, which leave nothing in their second slots.
  const int slots = by_items && items * 7 <= groups ? 1 : 2;
  cfg.gridDim = dim3(ctas, UNITS, slots);  // blocks of second slots, often empty ones, come last
  cfg.blockDim = dim3(JOIN);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, join_kernel, static_cast<const AttendParams>(p), ctas);
}

}  // namespace klt
