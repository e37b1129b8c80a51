// Shared parts of latent attention: the parameters of its kernels, and the tensor-core
// descriptors and TMEM accesses that only they use.
#pragma once

#include "klt_linear.cuh"

namespace klt {

struct AttendParams {
  const __nv_bfloat16* q;
  const int* table;
  const int* lens;
  const int* cu_q;       // or null: one query a sequence
  __nv_bfloat16* out;
  float* lse;
  float* part;           // workspace
  int64_t q_token, q_head, ld_table, out_token, out_head;
  int B, T, H;
  int members;           // row tiles of a sequence that are computed side by side
  int q_box;             // rows of the queries' map that a bulk copy takes, 0: none can
  bool q_packed;         // that map's rows are (token, head) in one direction
  int R, rope;           // latent, position part
  int page_log2, max_pages, pages;
  float scale;           // of the scores, times log2(e)
  int stall;             // test hook: copies stop after this many tiles (0 = never)
  int* err;
  long long timeout;     // SM cycles
};

struct PrefillParams {
  const int* cu_q;
  const int* cu_k;
  __nv_bfloat16* out;
  float* lse;
  int64_t out_token, out_head;
  int B, T, S, H;
  int nope, rope, value;
  int causal;
  int side;              // heads whose units are started side by side
  float scale;           // as above
  int stall;
  int* err;
  long long timeout;
};

// Added per tile of keys to the bounds of waits that last for all of a sequence's: some five times
// what a tile takes.
constexpr long long TILE_CYCLES = 16384;

// The range cu[b] .. cu[b + 1] cut to 0 .. n (whatever cu holds).
KLT_DEV void range_of(const int* cu, int b, int n, int& lo, int& hi) {
  lo = min(max(cu[b], 0), n);
  hi = min(max(cu[b + 1], lo), n);
}

// ------------------------------------------------------------------ tcgen05
// Shared-memory descriptor of an operand whose rows (its M or N direction) are contiguous: boxes
// of 64 columns x k rows of 128 bytes in the 128-byte swizzle, 8 rows (1024 bytes) to an atom,
// boxes `box_bytes` apart.  Its instruction descriptor has the operand's transpose bit set.
KLT_DEV uint64_t sdesc_sw128_mn(uint32_t saddr, uint32_t box_bytes) {
  return static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4) |
         (static_cast<uint64_t>(box_bytes >> 4) << 16) |
         (static_cast<uint64_t>(1024 >> 4) << 32) | (static_cast<uint64_t>(1) << 46) |
         (static_cast<uint64_t>(2) << 61);
}
constexpr uint32_t IDESC_A_MN = 1u << 15, IDESC_B_MN = 1u << 16;

// Arrive on a barrier of any CTA of the cluster, publishing this thread's writes to the cluster.
KLT_DEV void mbar_arrive_cluster_release(uint32_t addr) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(addr)
               : "memory");
}
// As mbar_wait, for what a thread of another CTA of the cluster has published (mbar_wait alone
// acquires at CTA scope).  The phase that is over stays the last one until this thread goes on.
KLT_DEV bool mbar_wait_cluster(uint64_t* bar, uint32_t parity, volatile int* abort_flag,
                               int* err_word, long long timeout) {
  if (!mbar_wait(bar, parity, abort_flag, err_word, timeout)) return false;
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}
// 3-D tiled load of the box at (c0 = inner element, c1, c2).
KLT_DEV void tma_load_3d(void* dst, const CUtensorMap* map, uint64_t* bar, int c0, int c1,
                         int c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2)
      : "memory");
}

// 32 columns of the 64 rows of an M = 64 accumulator: warp w of a warpgroup holds rows 16 w ..
// 16 w + 15 in its first 16 lanes.  Register 4 g + 2 i + j is row lane / 4 + 8 i, column
// 8 g + 2 (lane % 4) + j.
KLT_DEV void tmem_ld_rows16(uint32_t taddr, float* v) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
        "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}
KLT_DEV void tmem_st32(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
      "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]),
      "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
      "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}

// One lane of a converged warp, in a form that the compiler knows to be one (64 x 64 x 16 products
// issued one after another: 35 cycles each, under lane == 0 47).
KLT_DEV bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r != 0;
}

KLT_DEV void tma_load_4d(void* dst, const CUtensorMap* map, uint64_t* bar, int c0, int c1, int c2,
                         int c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
      : "memory");
}
// Asks L2 to fetch a box.
KLT_DEV void tma_prefetch_3d(const CUtensorMap* map, int c0, int c1, int c2) {
  asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global.tile [%0, {%1, %2, %3}];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(c0), "r"(c1), "r"(c2)
               : "memory");
}
KLT_DEV void tma_prefetch_4d(const CUtensorMap* map, int c0, int c1, int c2, int c3) {
  asm volatile("cp.async.bulk.prefetch.tensor.4d.L2.global.tile [%0, {%1, %2, %3, %4}];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(c0), "r"(c1), "r"(c2), "r"(c3)
               : "memory");
}
// A value that all lanes of a converged warp share, in a form that the compiler knows to be so.
template <typename T>
KLT_DEV T uniform(T v) {
  return static_cast<T>(__shfl_sync(0xFFFFFFFFu, static_cast<int>(v), 0));
}
// Four products of K = 16 whose A has its rows contiguous: 16 rows of K (2048 bytes) apart, B's 32
// bytes.
KLT_DEV void mma4_bf16_mn(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                          uint32_t accumulate) {
  mma_bf16(d, a, b, idesc, accumulate);
  mma_bf16(d, a + 128, b + 2, idesc, 1);
  mma_bf16(d, a + 256, b + 4, idesc, 1);
  mma_bf16(d, a + 384, b + 6, idesc, 1);
}
// Asynchronous copy of `bytes` (16 or 0) from global to shared memory; the rest of 16 is zeros.
KLT_DEV void cp_async16(void* dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src),
               "r"(bytes)
               : "memory");
}
KLT_DEV void cp_async_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// 2^x by the hardware approximation (2 ulp; subnormal results flushed, far below what a sum of
// weights of at least one holds).
KLT_DEV float exp2_fast(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
KLT_DEV uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 t = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&t);
}

// ------------------------------------------------------------------ launches
uint64_t attend_workspace(int num_sms, int latent);
cudaError_t launch_attend(const CUtensorMap& latents, const CUtensorMap& ropes,
                          const CUtensorMap& queries, AttendParams p, int num_sms,
                          cudaStream_t s);
cudaError_t launch_prefill(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                           const CUtensorMap& k_rope, const PrefillParams& p, unsigned tiles,
                           cudaStream_t s);
constexpr int PREFILL_ROWS = 512;  // queries of a pair of CTAs
// Once per device, before the first launch; false when a kernel is not what its launch expects.
bool prepare_attend();
bool prepare_prefill();

}  // namespace klt
