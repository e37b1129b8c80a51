// Latent attention in absorbed form over a paged cache (sm_103a).
//
// 64 query rows (token, head) at a time against 64 keys at a time: S = Q K^T (M = 64 rows, N = 64
// keys), softmax in registers, O^T += V^T P^T (M = 128 latent columns, N = 64 rows).  A key's row
// is its value too, so each tile of keys is loaded once and read by both products: K-major by the
// first, and by the second with its columns as rows.
#include "klt_latent.cuh"

#include "../../include/klt.h"

namespace klt {
namespace {

constexpr int ROWS = 64, KEYS = 64;
constexpr int BOX = KEYS * 128;  // 64 rows x 128 bytes

KLT_DEV float quad_max(float v) {
  v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 1));
  return fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 2));
}
KLT_DEV float quad_sum(float v) {
  v += __shfl_xor_sync(0xFFFFFFFFu, v, 1);
  return v + __shfl_xor_sync(0xFFFFFFFFu, v, 2);
}

__global__ void __launch_bounds__(128, 1)
    attend_kernel(const __grid_constant__ CUtensorMap cache, const AttendParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* qs = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  const int NB = p.R / 64, KB = NB + 1;  // boxes of a row: latent, and position part
  uint8_t* ks = qs + 9 * BOX;
  uint8_t* ps = ks + 9 * BOX;
  __shared__ float factor[ROWS];
  __shared__ uint64_t full, done;
  __shared__ uint32_t tmem_holder;
  __shared__ int abort_flag;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
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
  const uint32_t tmem = tmem_holder;
  pdl_trigger();
  pdl_wait();
  volatile int* stop = &abort_flag;

  const int b = blockIdx.x;
  int q0 = b, q1 = b + 1;
  if (p.cu_q) range_of(p.cu_q, b, p.T, q0, q1);
  const int n = q1 - q0;
  const int len =
      static_cast<int>(max(0ll, min(static_cast<long long>(p.lens[b]),
                                    static_cast<long long>(p.max_pages) << p.page_log2)));
  const int box_keys = p.page_log2 < 6 ? 1 << p.page_log2 : 64;
  const int64_t rows = static_cast<int64_t>(n) * p.H;
  int phase = 0, dphase = 0, copies = 0;
  bool ok = true;
  for (int64_t r0 = blockIdx.y * static_cast<int64_t>(ROWS); r0 < rows && ok;
       r0 += static_cast<int64_t>(gridDim.y) * ROWS) {
    // queries
    for (int i = tid; i < ROWS * KB * 8; i += 128) {
      const int r = i / (KB * 8), c = i - r * KB * 8;
      uint4 v = make_uint4(0, 0, 0, 0);
      if (r0 + r < rows && c * 8 < p.R + p.rope) {
        const int t = static_cast<int>((r0 + r) / p.H), h = static_cast<int>((r0 + r) % p.H);
        v = *reinterpret_cast<const uint4*>(p.q + (q0 + t) * p.q_token + h * p.q_head + c * 8);
      }
      *reinterpret_cast<uint4*>(qs + (c >> 3) * BOX + r * 128 + (((c & 7) ^ (r & 7)) << 4)) = v;
    }
    fence_proxy_async_shared();
    __syncthreads();
    // this thread's rows: warp * 16 + lane / 4, and 8 further on
    int limit[2];
    float m[2], l[2] = {0.f, 0.f};
    int most = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int64_t r = r0 + warp * 16 + lane / 4 + 8 * i;
      limit[i] = r < rows ? len - (n - 1 - static_cast<int>(r / p.H)) : 0;
      m[i] = -INFINITY;
    }
    {
      const int64_t last = min(r0 + ROWS, rows) - 1;
      most = len - (n - 1 - static_cast<int>(last / p.H));
    }
    const int tiles = most > 0 ? (most + KEYS - 1) / KEYS : 0;
    for (int kt = 0; kt < tiles; ++kt) {
      const int left = min(KEYS, len - kt * KEYS);
      if (tid == 0 && (p.stall == 0 || copies < p.stall)) {
        const int boxes = (left + box_keys - 1) / box_keys;
        mbar_arrive_expect_tx(&full, boxes * KB * box_keys * 128);
        for (int x = 0; x < boxes; ++x) {
          const int key = kt * KEYS + x * box_keys;
          int page = p.table[b * p.ld_table + (key >> p.page_log2)];
          if (page < 0 || page >= p.pages) page = p.pages;
          for (int kb = 0; kb < KB; ++kb)
            tma_load_3d(ks + kb * BOX + x * box_keys * 128, &cache, &full, kb * 64,
                        key & ((1 << p.page_log2) - 1), page);
        }
      }
      ++copies;
      ok = mbar_wait(&full, phase, stop, p.err, p.timeout);
      phase ^= 1;
      if (!__syncthreads_and(ok)) {
        ok = false;
        break;
      }
      if (left < KEYS) {  // rows behind the last token hold anything
        for (int i = tid; i < (KEYS - left) * NB * 8; i += 128) {
          const int r = left + i / (NB * 8), c = i % (NB * 8);
          *reinterpret_cast<uint4*>(ks + (c >> 3) * BOX + r * 128 + ((c & 7) << 4)) =
              make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_shared();
        __syncthreads();
      }
      if (tid == 0) {
        tc_fence_after();
        for (int kb = 0; kb < KB; ++kb) {
          const int steps = kb < NB ? 4 : p.rope / 16;
          for (int s = 0; s < steps; ++s)
            mma_bf16(tmem + 256, sdesc_sw128(smem_u32(qs + kb * BOX)) + 2 * s,
                     sdesc_sw128(smem_u32(ks + kb * BOX)) + 2 * s, idesc_make(1, 64, 64),
                     kb | s);
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
      float v[32];
      tmem_ld_rows16(tmem + 256 + (static_cast<uint32_t>(warp * 32) << 16), v);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float top = m[i];
#pragma unroll
        for (int g = 0; g < 8; ++g)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int key = kt * KEYS + 8 * g + 2 * (lane & 3) + j;
            float& s = v[4 * g + 2 * i + j];
            s = key < limit[i] ? s * p.scale : -INFINITY;
            top = fmaxf(top, s);
          }
        top = quad_max(top);
        const float base = top == -INFINITY ? 0.f : top;
        const float f = exp2_fast(m[i] - base);
        m[i] = top;
        const int row = warp * 16 + lane / 4 + 8 * i;
        if ((lane & 3) == 0) factor[row] = f;
        l[i] *= f;
#pragma unroll
        for (int g = 0; g < 8; ++g) {
          const float a = exp2_fast(v[4 * g + 2 * i] - base),
                      c = exp2_fast(v[4 * g + 2 * i + 1] - base);
          l[i] += a + c;
          *reinterpret_cast<uint32_t*>(ps + row * 128 + ((g ^ (row & 7)) << 4) + (lane & 3) * 4) =
              pack_bf16(a, c);
        }
      }
      fence_proxy_async_shared();
      tc_fence_before();
      __syncthreads();
      if (kt > 0) {
        tc_fence_after();
        for (int c = 0; c < p.R / 128 * 64; c += 16) {
          float o[16];
          const uint32_t at = tmem + (static_cast<uint32_t>(warp * 32) << 16) + c;
          tmem_ld16(at, o);
#pragma unroll
          for (int i = 0; i < 16; ++i) o[i] *= factor[(c & 63) + i];
          tmem_st16(at, o);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncthreads();
      }
      if (tid == 0) {
        tc_fence_after();
        for (int j = 0; j < p.R / 128; ++j)
          for (int s = 0; s < 4; ++s)
            mma_bf16(tmem + j * 64, sdesc_sw128_mn(smem_u32(ks + 2 * j * BOX + s * 2048), BOX),
                     sdesc_sw128(smem_u32(ps)) + 2 * s, idesc_make(1, 128, 64) | IDESC_A_MN,
                     kt | s);
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
    if (!ok) break;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float sum = quad_sum(l[i]);
      const int64_t r = r0 + warp * 16 + lane / 4 + 8 * i;
      if ((lane & 3) == 0) {
        factor[r - r0] = sum > 0.f || sum != sum ? 1.0f / sum : 0.f;
        if (p.lse && r < rows)
          p.lse[static_cast<int64_t>(q0) * p.H + r] =
              sum == 0.f ? -INFINITY : (m[i] + log2f(sum)) * 0.6931471805599453f;
      }
    }
    __syncthreads();
    for (int c = 0; c < p.R / 128 * 64; c += 16) {
      float o[16] = {};
      if (tiles > 0) tmem_ld16(tmem + (static_cast<uint32_t>(warp * 32) << 16) + c, o);
      for (int i = 0; i < 16; ++i) {
        const int64_t r = r0 + (c & 63) + i;
        if (r < rows) {
          const float f = factor[(c & 63) + i];
          p.out[(q0 + r / p.H) * p.out_token + r % p.H * p.out_head + (c >> 6) * 128 + warp * 32 +
                lane] = __float2bfloat16(f == 0.f ? 0.f : o[i] * f);
        }
      }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

constexpr int SMEM = 1024 + 19 * BOX;

}  // namespace

uint64_t attend_workspace(int num_sms) { return 16; }

bool prepare_attend() {
  return cudaFuncSetAttribute(attend_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM) ==
         cudaSuccess;
}

cudaError_t launch_attend(const CUtensorMap& cache, const AttendParams& p, int num_sms,
                          cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.B, 4);
  cfg.blockDim = dim3(128);
  cfg.dynamicSmemBytes = SMEM;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, attend_kernel, cache, p);
}

}  // namespace klt
