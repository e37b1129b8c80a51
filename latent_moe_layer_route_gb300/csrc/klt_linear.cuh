// Shared parts of the FP8 linear layer's two kernels: the parameters, and the cluster and
// CTA-pair forms of barriers, copies and tensor-core instructions.  Inline PTX only.
#pragma once

#include "klt_device.cuh"

namespace klt {

// The weights are kept tile-major: row block rb (128 rows) and k-block kb (128 columns) is
// one contiguous 16 KB image in the 128-byte swizzle, at ((rb * KB + kb) * 16384); rows and
// columns past N and K are zero codes.
constexpr int LIN_TILE = 128;
constexpr int LIN_TILE_BYTES = LIN_TILE * LIN_TILE;

struct LinParams {
  const uint8_t* w;   // tile-major image
  const float* ws;    // [NB + 1, KB], the last row zero
  const float* xs;    // [M, KB]
  void* out;          // bf16 / fp32 / e4m3
  float* out_s;       // e4m3 outputs: [M, width / 128]
  int64_t ld_out;     // elements
  int M, KB, NB;      // tokens, k-blocks, row blocks of W
  int width;          // output columns (N; N / 2 for SwiGLU)
  int up;             // SwiGLU: row block of the up tile minus that of the gate tile
  int out_dtype;      // enum klt_dtype
  // token-major kernel: tiles of 256 tokens and of 256 rows of W, the step from one tile of a
  // CTA pair to its next, and from the first weight tile's scales to the second's
  int tiles_m, tiles_n, step_m, step_n, step_ws;
  bool out_wide;      // output rows start on 16 bytes
  int stall;          // test hook: producers stop after this many k-blocks (0 = never)
  int* err;
  long long timeout;  // SM cycles
};

// ------------------------------------------------------------------ clusters
KLT_DEV uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
KLT_DEV void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release;" ::: "memory");
}
KLT_DEV void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }
// Address of this CTA's shared-memory address `saddr` in CTA `rank` of the cluster.
KLT_DEV uint32_t map_to_rank(uint32_t saddr, uint32_t rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(saddr), "r"(rank));
  return r;
}
// As cluster_arrive, publishing nothing but what a fence before it has (fence_barrier_init).
KLT_DEV void cluster_arrive_relaxed() {
  asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory");
}
// Stores four values (16-byte aligned) into shared memory of any CTA of the cluster, completing
// 16 bytes on a barrier of that CTA (both addresses from map_to_rank).
KLT_DEV void st_async_f4(uint32_t addr, float a, float b, float c, float d, uint32_t bar) {
  asm volatile(
      "st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1, %2, %3, %4}, "
      "[%5];" ::"r"(addr),
      "r"(__float_as_uint(a)), "r"(__float_as_uint(b)), "r"(__float_as_uint(c)),
      "r"(__float_as_uint(d)), "r"(bar)
      : "memory");
}
KLT_DEV void st_async_u32(uint32_t addr, uint32_t v, uint32_t bar) {  // one value, 4 bytes
  asm volatile(
      "st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.b32 [%0], %1, [%2];" ::"r"(addr),
      "r"(v), "r"(bar)
      : "memory");
}
KLT_DEV ulonglong2 ld_shared_u64x2(uint32_t addr) {
  ulonglong2 v;
  asm volatile("ld.shared.v2.u64 {%0, %1}, [%2];" : "=l"(v.x), "=l"(v.y) : "r"(addr) : "memory");
  return v;
}
KLT_DEV void st_cluster_f4(uint32_t addr, float a, float b, float c, float d) {
  asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "f"(a), "f"(b),
               "f"(c), "f"(d)
               : "memory");
}
// Arrive on a barrier of any CTA of the cluster (`addr` from map_to_rank).  For hand-offs of
// TMEM, whose reads have completed: nothing written to memory is published, so the release
// stays at CTA scope (at cluster scope it is a memory barrier, and the wide kernel stood in
// it for half of its time: 4096 x 7168 x 3584 in 189 us).
KLT_DEV void mbar_arrive_cluster(uint32_t addr) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(addr)
               : "memory");
}

// ------------------------------------------------------------------ CTA pairs
// 2-D tiled load into this CTA's shared memory, completing on a barrier of either CTA of the
// pair (`bar` from map_to_rank).
KLT_DEV void tma_load_2d_pair(void* dst, const CUtensorMap* map, uint32_t bar, int c0, int c1) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      ".cta_group::2 [%0], [%1, {%3, %4}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1)
      : "memory");
}
// Stores the shared-memory box at (c0 = inner element index, c1 = row) of a tensor; parts
// outside of it are not written.  Completion is tracked per thread (bulk groups).
KLT_DEV void tma_store_2d(const CUtensorMap* map, const void* src, int c0, int c1) {
  asm volatile(
      "cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
          reinterpret_cast<uint64_t>(map)),
      "r"(smem_u32(src)), "r"(c0), "r"(c1)
      : "memory");
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
// All but this thread's last N bulk stores have read their shared memory.
template <int N>
KLT_DEV void tma_store_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}
// All of this thread's bulk stores are complete.
KLT_DEV void tma_store_wait() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }
// Orders this thread's shared-memory writes before later bulk copies that read them.
KLT_DEV void fence_proxy_async_shared() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}
KLT_DEV void tmem_alloc_pair(uint32_t* dst_smem, uint32_t ncols) {  // a warp of both CTAs
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                   smem_u32(dst_smem)),
               "r"(ncols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
KLT_DEV void tmem_dealloc_pair(uint32_t taddr, uint32_t ncols) {  // a warp of both CTAs
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr),
               "r"(ncols)
               : "memory");
}
// Arrive once on the barrier at the same offset in the CTAs of `mask` (bit = rank) when every
// MMA issued so far by this thread has completed.
KLT_DEV void tc_commit_pair(uint64_t* bar, uint16_t mask) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
      " [%0], %1;" ::"r"(smem_u32(bar)),
      "h"(mask)
      : "memory");
}
// The four MMAs of one 128-byte K block over both CTAs' tiles (M = 256: 128 rows of A in each
// CTA; half of B's rows in each CTA), replacing the accumulator.
KLT_DEV void mma4_fp8_pair(uint32_t d, uint64_t da, uint64_t db, uint32_t idesc) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, 0, 0;\n\tsetp.eq.b32 q, 0, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t"
      "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %4, %5, %3, q;\n\t"
      "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %6, %7, %3, q;\n\t"
      "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %8, %9, %3, q;\n\t}" ::"r"(d),
      "l"(da), "l"(db), "r"(idesc), "l"(da + 2), "l"(db + 2), "l"(da + 4), "l"(db + 4),
      "l"(da + 6), "l"(db + 6)
      : "memory");
}

// ------------------------------------------------------------------ TMEM loads
// Starts the load of 32 consecutive fp32 columns of this thread's TMEM lane; the registers
// hold them after tmem_wait_ld32 on the same array.
KLT_DEV void tmem_start_ld32(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
        "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]),
        "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]),
        "=r"(r[31])
      : "r"(taddr)
      : "memory");
}
// Waits for this thread's TMEM loads; the registers pass through, so that no use of them
// moves above the wait.
KLT_DEV void tmem_wait_ld32(uint32_t* r) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                 "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
                 "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]),
                 "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                 "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]),
                 "+r"(r[30]), "+r"(r[31])
               :
               : "memory");
}

// As tmem_start_ld32 / tmem_wait_ld32, 16 columns.
KLT_DEV void tmem_start_ld16(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
        "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
KLT_DEV void tmem_wait_ld16(uint32_t* r) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                 "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
                 "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :
               : "memory");
}

// ------------------------------------------------------------------ arithmetic
// Two fp32 fused multiply-adds in one instruction: a += p * s, each lane rounded as fmaf.
KLT_DEV void fma2(unsigned long long& a, unsigned long long p, unsigned long long s) {
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(a) : "l"(p), "l"(s));
}
KLT_DEV unsigned long long mul2(unsigned long long a, unsigned long long b) {
  unsigned long long r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
KLT_DEV unsigned long long fmaf2(unsigned long long a, unsigned long long b,
                                 unsigned long long c) {
  unsigned long long r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
KLT_DEV void add2(unsigned long long& a, unsigned long long b) {
  asm("add.rn.f32x2 %0, %0, %1;" : "+l"(a) : "l"(b));
}
KLT_DEV unsigned long long pack2(float lo, float hi) {
  unsigned long long r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
KLT_DEV void unpack2(unsigned long long v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}

// 1 / (1 + e^-x) to 4 ulp over the whole range: with e = e^-|x| as 1 / (1 + e) or e / (1 + e), so
// that the divisor lies in 1 .. 2, and far below 0 the result runs to 0 as e does.  expf, not the
// fast exponential, which is 13 ulp off at -10 and 95 at -80; the fast reciprocal (1 ulp).
KLT_DEV float sigmoid(float x) {
  const float e = expf(-fabsf(x));
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
  return x < 0.f ? e * r : r;
}
// SiLU; far below 0 the factor is 0, so that g, however large, leaves nothing.
KLT_DEV float silu(float g) { return g * sigmoid(g); }

// amax / 448, correctly rounded: the quotient by the rounded 1/448 corrected by its residual,
// or by division where that would leave the normal range.
KLT_DEV float over_448(float amax) {
  if (amax > 1e-25f && amax < 1e38f) {
    const float q0 = amax * (1.0f / 448.0f);
    return fmaf(-fmaf(q0, 448.0f, -amax), 1.0f / 448.0f, q0);
  }
  return amax / 448.0f;
}
// The scale of a quantised group from its largest magnitude; a scale that is zero becomes 1.
KLT_DEV float group_scale(float amax) {
  const float s = over_448(amax);
  return s == 0.f ? 1.0f : s;
}
// quot_rn needs the scale, its reciprocal and the residual in the normal range.  Brings a scale
// far from 1 there by a power of two, which it returns: the group's values times that power
// (exact as far as a code can tell) divided by the new scale have the same quotients.  A scale
// that is not finite stays so and turns every code of its group into NaN.
KLT_DEV float rescale(float& s) {
  if (s > 1e-30f && s < 1e30f) return 1.0f;
  const float k = s < 1.0f ? 0x1p100f : 0x1p-60f;
  s *= k;
  return k;
}
// fp32(x / s), correctly rounded, for s > 0 and inv = 1/s correctly rounded (Markstein's
// correction, the residual taken as q0 s - x so that a zero keeps its sign).
KLT_DEV float quot_group(float x, float s, float inv) {
  const float q0 = x * inv;
  return fmaf(-fmaf(q0, s, -x), inv, q0);
}
// The negatives of quot_group of two values, signs of zero included, from s and -1/s in both
// halves: a packed operation has no operand signs, a code's sign is one bit.
KLT_DEV unsigned long long neg_quot_group2(unsigned long long x, unsigned long long s,
                                           unsigned long long ninv) {
  const unsigned long long q0 = mul2(x, ninv);
  return fmaf2(fmaf2(q0, s, x), ninv, q0);
}
// The larger magnitude; a NaN wins over every number.
KLT_DEV float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(fabsf(a)), "f"(fabsf(b)));
  return r;
}

// The same of three.
KLT_DEV float max_nan(float a, float b, float c) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// ------------------------------------------------------------------ launches
cudaError_t launch_linear_narrow(const CUtensorMap& tok, const LinParams& p, int bn, int split,
                                 bool swiglu, cudaStream_t s);
cudaError_t launch_linear_wide(const CUtensorMap& tok, const CUtensorMap& wmap,
                               const CUtensorMap& omap, const LinParams& p, bool swiglu,
                               int parts, int num_sms, cudaStream_t s);
// Once per device, before the first launch: shared-memory sizes, and whether the kernels are
// what their launches expect.
// clusters[i]: clusters of 2^i CTAs, one per SM, that are resident at once
bool prepare_linear_narrow(int clusters[4]);
bool prepare_linear_wide(int* max_tiles);  // tiles that two pairs each share at once

}  // namespace klt
