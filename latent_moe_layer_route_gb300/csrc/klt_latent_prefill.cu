// Latent attention in expanded form over packed sequences (sm_103a).
//
// 128 queries of one head against 128 keys at a time: S = Q K^T, a row of which is one thread's,
// softmax in registers, P back into TMEM as the first operand of O += P V.
#include "klt_latent.cuh"

#include "../../include/klt.h"

namespace klt {
namespace {

constexpr int BOX = 128 * 128;  // 128 rows x 128 bytes
constexpr int KEYS = 128;
constexpr int SMEM = 1024 + 8 * BOX;

__global__ void __launch_bounds__(128, 1)
    prefill_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                   const __grid_constant__ CUtensorMap vmap,
                   const __grid_constant__ CUtensorMap rmap, const PrefillParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* qs = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  uint8_t* ks = qs + 3 * BOX;
  uint8_t* vs = ks + 3 * BOX;
  __shared__ uint64_t full, done;
  __shared__ uint32_t tmem_holder;
  __shared__ int abort_flag;
  const int tid = threadIdx.x, warp = tid >> 5;
  if (tid == 0) {
    mbar_init(&full, 1);
    mbar_init(&done, 1);
    abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 0) {
    tmem_alloc(&tmem_holder, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_holder, S = tmem + 128, P = tmem + 256;
  const uint32_t mine = static_cast<uint32_t>(warp * 32) << 16;
  pdl_trigger();
  pdl_wait();
  volatile int* stop = &abort_flag;

  // this tile's sequence
  int tile = blockIdx.x, b = 0, q0 = 0, q1 = 0;
  for (; b < p.B; ++b) {
    range_of(p.cu_q, b, p.T, q0, q1);
    const int t = (q1 - q0 + PREFILL_ROWS - 1) / PREFILL_ROWS;
    if (tile < t) break;
    tile -= t;
  }
  const int h = blockIdx.y;
  bool ok = b < p.B;
  if (ok) {
    int k0, k1;
    range_of(p.cu_k, b, p.S, k0, k1);
    const int n = q1 - q0, len = k1 - k0, r0 = tile * PREFILL_ROWS;
    const int row = r0 + tid;
    const int nb = p.nope / 64, vb = p.value / 64;
    const int limit = row >= n ? 0 : p.causal ? len - (n - 1 - row) : len;
    const int last = min(r0 + PREFILL_ROWS, n) - 1;
    const int most = p.causal ? len - (n - 1 - last) : len;
    const int tiles = most > 0 ? (most + KEYS - 1) / KEYS : 0;
    float m = -INFINITY, l = 0.f;
    int phase = 0, dphase = 0;
    for (int kt = 0; kt < tiles; ++kt) {
      const int left = min(KEYS, len - kt * KEYS);
      if (tid == 0 && (p.stall == 0 || kt < p.stall)) {
        mbar_arrive_expect_tx(&full, ((kt == 0 ? nb + 1 : 0) + nb + 1 + vb) * BOX);
        if (kt == 0)
          for (int i = 0; i <= nb; ++i) tma_load_3d(qs + i * BOX, &qmap, &full, i * 64, h, q0 + r0);
        for (int i = 0; i < nb; ++i)
          tma_load_3d(ks + i * BOX, &kmap, &full, i * 64, h, k0 + kt * KEYS);
        tma_load_3d(ks + nb * BOX, &rmap, &full, 0, 0, k0 + kt * KEYS);
        for (int i = 0; i < vb; ++i)
          tma_load_3d(vs + i * BOX, &vmap, &full, i * 64, h, k0 + kt * KEYS);
      }
      ok = mbar_wait(&full, phase, stop, p.err, p.timeout);
      phase ^= 1;
      if (!__syncthreads_and(ok)) {
        ok = false;
        break;
      }
      if (left < KEYS) {  // the next sequence's values
        for (int i = tid; i < (KEYS - left) * vb * 8; i += 128) {
          const int r = left + i / (vb * 8), c = i % (vb * 8);
          *reinterpret_cast<uint4*>(vs + (c >> 3) * BOX + r * 128 + ((c & 7) << 4)) =
              make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_shared();
        __syncthreads();
      }
      if (tid == 0) {
        tc_fence_after();
        for (int i = 0; i <= nb; ++i) {
          const int steps = i < nb ? 4 : p.rope / 16;
          for (int s = 0; s < steps; ++s)
            mma_bf16(S, sdesc_sw128(smem_u32(qs + i * BOX)) + 2 * s,
                     sdesc_sw128(smem_u32(ks + i * BOX)) + 2 * s, idesc_make(1, 128, 128), i | s);
        }
        tc_commit(&done);
      }
      ok = mbar_wait(&done, dphase, stop, p.err, p.timeout);
      dphase ^= 1;
      if (!__syncthreads_and(ok)) {
        ok = false;
        break;
      }
      tc_fence_after();
      float top = m;
#pragma unroll 1
      for (int c = 0; c < KEYS; c += 32) {
        float v[32];
        tmem_ld16x2(S + mine + c, S + mine + c + 16, v, v + 16);
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if (kt * KEYS + c + i < limit) top = fmaxf(top, v[i] * p.scale);
      }
      const float base = top == -INFINITY ? 0.f : top;
      const float f = exp2_fast(m - base);
      m = top;
      l *= f;
#pragma unroll 1
      for (int c = 0; c < KEYS; c += 64) {
        uint32_t w[32];
#pragma unroll
        for (int g = 0; g < 64; g += 32) {
          float v[32];
          tmem_ld16x2(S + mine + c + g, S + mine + c + g + 16, v, v + 16);
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            v[i] = kt * KEYS + c + g + i < limit ? exp2_fast(v[i] * p.scale - base) : 0.f;
            l += v[i];
          }
#pragma unroll
          for (int i = 0; i < 16; ++i) w[g / 2 + i] = pack_bf16(v[2 * i], v[2 * i + 1]);
        }
        tmem_st32(P + mine + c / 2, w);
      }
      if (kt > 0)
        for (int c = 0; c < p.value; c += 16) {
          float o[16];
          tmem_ld16(tmem + mine + c, o);
#pragma unroll
          for (int i = 0; i < 16; ++i) o[i] *= f;
          tmem_st16(tmem + mine + c, o);
        }
      tmem_wait_st();
      tc_fence_before();
      __syncthreads();
      if (tid == 0) {
        tc_fence_after();
        for (int s = 0; s < 8; ++s)
          mma_bf16_ta(tmem, P + 8 * s, sdesc_sw128_mn(smem_u32(vs + s * 2048), BOX),
                      idesc_make(1, 128, p.value) | IDESC_B_MN, kt | s);
        tc_commit(&done);
      }
      ok = mbar_wait(&done, dphase, stop, p.err, p.timeout);
      dphase ^= 1;
      if (!__syncthreads_and(ok)) {
        ok = false;
        break;
      }
      tc_fence_after();
    }
    if (ok) {
      const float f = l > 0.f || l != l ? 1.0f / l : 0.f;
      if (p.lse && row < n)
        p.lse[(q0 + row) * static_cast<int64_t>(p.H) + h] =
            l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
      for (int c = 0; c < p.value; c += 16) {
        float o[16] = {};
        if (tiles > 0) tmem_ld16(tmem + mine + c, o);
        if (row < n)
#pragma unroll
          for (int i = 0; i < 16; ++i)
            p.out[(q0 + row) * p.out_token + h * p.out_head + c + i] =
                __float2bfloat16(f == 0.f ? 0.f : o[i] * f);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
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
  cfg.gridDim = dim3(tiles, p.H);
  cfg.blockDim = dim3(128);
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
