// Latent attention, host side (argument checks, the handle, tensor maps) and the step that fills
// the cache (sm_103a).
#include <cuda.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <new>

#include "../../include/klt.h"
#include "klt_latent.cuh"

using namespace klt;

struct klt_latent {
  klt_latent_dims d;
  int device;
  int num_sms;
  int page_log2;
  float* inv_freq;       // [rope / 2]
  __nv_bfloat16* gamma;  // [latent] or null
  int* err;              // device error word
};

namespace {

// ------------------------------------------------------------------ append
// A block takes one token, or two where there are many.  The latent part (R / 8 lanes of 8 values)
// is normed in registers between the sum of its squares and its outputs; angles are fp64 up to the
// reduced turn (at position 10^6 fp32 angles are off by 0.03), one lane per pair, shared by the
// block; then the block's threads turn the row's and the queries' pairs, 16 elements a thread, whose
// loads went out first.  Every value is read and written once: 8192 tokens of 512 + 64 columns and
// 64 heads take 31 us (5.2 TB/s), bound by what six blocks an SM keep in flight (one token to a
// block, loads behind the norm: 37; four or eight blocks an SM by registers: 33, 35); 16 tokens take
// 2.7.  Six blocks leave a thread 40 registers: with two tokens to a block 24 to 60 bytes of them
// spill, 327,680 requests of the 8192 tokens' traffic to L1, which runs at 75 % of its rate.
// Tokens from which on a block takes two.  One and two to a block, us, 64 heads: 600 tokens 3.8, 4.4;
// 1200 5.9, 6.4; 1500 7.2, 7.0; 3000 15.6, 13.8; 8192 35.2, 30.5.  48 heads cross there too, 40 heads
// of 256 + 32 columns are alike from 600 on, 128 heads lose up to 5 % between 1900 and 2700 (16.5,
// 17.2 at 2000).
constexpr int APPEND_TWO = 1500;
struct AppendParams {
  const void* kv;
  const int64_t* positions;
  const int64_t* slots;
  const float* inv_freq;
  const __nv_bfloat16* gamma;
  __nv_bfloat16* cache;
  __nv_bfloat16* kv_out;
  const __nv_bfloat16* q;
  __nv_bfloat16* q_out;
  int64_t ld_kv, page_stride, row_stride, ld_kv_out, q_token, q_head, q_out_token, q_out_head;
  int64_t n_slots;
  int T, R, rope, H, page_log2;
  float eps;
};

KLT_DEV void unpack8(uint4 a, float* v) {
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
KLT_DEV uint4 pack8(const float* v) {
  return make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]),
                    pack_bf16(v[6], v[7]));
}
template <bool F32>
KLT_DEV void load8(const void* base, int64_t off, float* v) {
  if (F32) {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(base) + off);
    const float4 a = p[0], b = p[1];
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
    v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  } else {
    unpack8(*reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(base) + off), v);
  }
}
// Turns the eight pairs of unit u: halves (a[e], b[e]), neighbours (a's four, then b's).
KLT_DEV void turn8(float* a, float* b, const float4* cs, bool neighbours) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    float* x = !neighbours ? &a[e] : e < 4 ? &a[2 * e] : &b[2 * e - 8];
    float* y = !neighbours ? &b[e] : x + 1;
    const float4 w = cs[e >> 1];
    const float c = e & 1 ? w.z : w.x, s = e & 1 ? w.w : w.y;
    const float t = *x * c - *y * s;
    *y = *y * c + *x * s;
    *x = t;
  }
}

template <bool F32, bool NEIGHBOURS, int TOKENS>
__global__ void __launch_bounds__(256, 6) append_kernel(const AppendParams p) {
  __shared__ float4 turns[TOKENS][16];  // cos, sin of two pairs
  __shared__ float sums[TOKENS][2];
  pdl_trigger();
  pdl_wait();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int chunks = p.R >> 3, units = p.rope >> 4, half = p.rope >> 1, queries = p.H * units;
  // first element of a unit's second eight, from the first's
  const int second = NEIGHBOURS ? 8 : half, step = NEIGHBOURS ? 16 : 8;
  const int t0 = blockIdx.x * TOKENS;
  // the first units of this thread's queries are on their way while the rows are normed
  const int h0 = tid / units, u0 = tid - h0 * units;
  auto query = [&](int k, int64_t token, int64_t head, int h, int u) {
    return (t0 + k) * token + h * head + u * step;
  };
  uint4 qa[TOKENS], qb[TOKENS];
#pragma unroll
  for (int k = 0; k < TOKENS; ++k)
    if (p.q && tid < queries && t0 + k < p.T) {
      const __nv_bfloat16* src = p.q + query(k, p.q_token, p.q_head, h0, u0);
      qa[k] = *reinterpret_cast<const uint4*>(src);
      qb[k] = *reinterpret_cast<const uint4*>(src + second);
    }
  // two warps norm a row, the last ones find the angles
  const int mine = warp >> 1, at = tid & 63;
  float c[8] = {};
  if (mine < TOKENS && t0 + mine < p.T) {
    if (at < chunks) load8<F32>(p.kv, (t0 + mine) * p.ld_kv + at * 8, c);
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) s = fmaf(c[i], c[i], s);
#pragma unroll
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
    if (lane == 0) sums[mine][warp & 1] = s;
  }
  const int turner = static_cast<int>(blockDim.x >> 5) - 1 - warp;
  if (turner < TOKENS && t0 + turner < p.T && lane < half) {
    const double turn = static_cast<double>(p.positions[t0 + turner]) *
                        static_cast<double>(p.inv_freq[lane]) * 0.15915494309189535;
    float s, cosine;
    sincospif(2.0f * static_cast<float>(turn - rint(turn)), &s, &cosine);
    reinterpret_cast<float2*>(turns[turner])[lane] = make_float2(cosine, s);
  }
  __syncthreads();
  auto row_of = [&](int k) -> __nv_bfloat16* {
    const int64_t slot = p.cache ? p.slots[t0 + k] : -1;
    if (slot < 0 || slot >= p.n_slots) return nullptr;
    return p.cache + (slot >> p.page_log2) * p.page_stride +
           (slot & ((1ll << p.page_log2) - 1)) * p.row_stride;
  };
  const int part = tid - 64 * TOKENS;  // threads that turn the rows' position parts
  if (mine < TOKENS && t0 + mine < p.T && at < chunks) {
    __nv_bfloat16* const row = row_of(mine);
    __nv_bfloat16* const dense = p.kv_out ? p.kv_out + (t0 + mine) * p.ld_kv_out : nullptr;
    const float r = 1.0f / sqrtf((sums[mine][0] + sums[mine][1]) / static_cast<float>(p.R) + p.eps);
    float g[8] = {1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f};
    if (p.gamma) unpack8(*reinterpret_cast<const uint4*>(p.gamma + at * 8), g);
#pragma unroll
    for (int i = 0; i < 8; ++i) c[i] = c[i] * r * g[i];
    const uint4 w = pack8(c);
    if (row) *reinterpret_cast<uint4*>(row + at * 8) = w;
    if (dense) *reinterpret_cast<uint4*>(dense + at * 8) = w;
  } else if (part >= 0 && part < TOKENS * units && t0 + part / units < p.T) {
    const int k = part / units, u = part - k * units, e = p.R + u * step;
    __nv_bfloat16* const row = row_of(k);
    __nv_bfloat16* const dense = p.kv_out ? p.kv_out + (t0 + k) * p.ld_kv_out : nullptr;
    float a[8], b[8];
    load8<F32>(p.kv, (t0 + k) * p.ld_kv + e, a);
    load8<F32>(p.kv, (t0 + k) * p.ld_kv + e + second, b);
    turn8(a, b, turns[k] + u * 4, NEIGHBOURS);
    const uint4 wa = pack8(a), wb = pack8(b);
    if (row) {
      *reinterpret_cast<uint4*>(row + e) = wa;
      *reinterpret_cast<uint4*>(row + e + second) = wb;
    }
    if (dense) {
      *reinterpret_cast<uint4*>(dense + e) = wa;
      *reinterpret_cast<uint4*>(dense + e + second) = wb;
    }
  }
  if (!p.q) return;
#pragma unroll
  for (int k = 0; k < TOKENS; ++k) {
    if (t0 + k >= p.T) break;
    int h = h0, u = u0;
    for (int i = tid; i < queries; i += blockDim.x) {
      if (i != tid) {
        h = i / units, u = i - h * units;
        const __nv_bfloat16* src = p.q + query(k, p.q_token, p.q_head, h, u);
        qa[k] = *reinterpret_cast<const uint4*>(src);
        qb[k] = *reinterpret_cast<const uint4*>(src + second);
      }
      float a[8], b[8];
      unpack8(qa[k], a);
      unpack8(qb[k], b);
      turn8(a, b, turns[k] + u * 4, NEIGHBOURS);
      __nv_bfloat16* dst = p.q_out + query(k, p.q_out_token, p.q_out_head, h, u);
      *reinterpret_cast<uint4*>(dst) = pack8(a);
      *reinterpret_cast<uint4*>(dst + second) = pack8(b);
    }
  }
}

// ------------------------------------------------------------------ checks
bool aligned(const void* p, uintptr_t bytes) {
  return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0;
}
// [n, m] rows of `width` elements at the strides a and b do not overlap.
bool disjoint(int64_t n, int64_t a, int64_t m, int64_t b, int64_t width) {
  if (n <= 1 || m <= 1) {
    const int64_t s = n > 1 ? a : m > 1 ? b : width;
    return s >= width;
  }
  return a < b ? a >= width && (b - width) / a >= n - 1 : b >= width && (a - width) / b >= m - 1;
}
constexpr int64_t MOST = 0x7FFFFFFFll - 4096;  // rows, with room to round up to tiles
constexpr int64_t MAX_STRIDE = 1ll << 38;  // elements: the tensor maps' strides end at 2^40 bytes

int check_dims(const klt_latent_dims* d) {
  if (d->heads < 1 || !(d->eps >= 0.f) || !std::isfinite(d->scale) || d->scale <= 0.f)
    return KLT_ERR_INVALID_ARG;
  if (d->heads > 256 || d->latent < 128 || d->latent > 512 || d->latent % 128 || d->rope < 16 ||
      d->rope > 64 || d->rope % 16 || (d->nope != 64 && d->nope != 128) ||
      (d->value != 64 && d->value != 128) || d->page < 16 || d->page > 1024 ||
      (d->page & (d->page - 1)) ||
      (d->pairs != KLT_ROPE_HALVES && d->pairs != KLT_ROPE_NEIGHBOURS))
    return KLT_ERR_UNSUPPORTED;
  return KLT_OK;
}
int check_device(const klt_latent* h) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return KLT_ERR_CUDA;
  return dev == h->device ? KLT_OK : KLT_ERR_INVALID_ARG;
}
long long timeout_cycles(const klt_latent_debug* dbg) {  // at about 2 GHz
  return static_cast<long long>(dbg && dbg->timeout_ms > 0 ? dbg->timeout_ms : 1000) * 2000000LL;
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiledFn get_encode() {
  static const EncodeTiledFn fn = [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    const bool found = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000,
                                                        cudaEnableDefault, &q) == cudaSuccess &&
                       q == cudaDriverEntryPointSuccess;
    return found ? reinterpret_cast<EncodeTiledFn>(ptr) : nullptr;
  }();
  return fn;
}
// bf16 [n2, n1, n0] with strides s2, s1 (elements) and contiguous n0, in swizzled boxes of
// [1 or b2, b1, 64]; what lies outside reads as 0.  A dimension of one has any stride.
bool encode_rows(CUtensorMap* m, const void* base, int64_t n0, int64_t n1, int64_t s1, int64_t n2,
                 int64_t s2, uint32_t b1, uint32_t b2) {
  EncodeTiledFn enc = get_encode();
  if (!enc) return false;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(n0), static_cast<cuuint64_t>(n1),
                              static_cast<cuuint64_t>(n2)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(n1 > 1 ? s1 * 2 : 1024),
                                 static_cast<cuuint64_t>(n2 > 1 ? s2 * 2 : 1024)};
  const cuuint32_t box[3] = {64, b1, b2};
  const cuuint32_t estr[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box,
             estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// bf16 [n2, n1, 64 blocks] as [n2, blocks, n1, 64], in swizzled boxes of [1, b2, b1, 64].
bool encode_columns(CUtensorMap* m, const void* base, int64_t blocks, int64_t n1, int64_t s1,
                    int64_t n2, int64_t s2, uint32_t b1, uint32_t b2) {
  EncodeTiledFn enc = get_encode();
  if (!enc) return false;
  const cuuint64_t dims[4] = {64, static_cast<cuuint64_t>(n1), static_cast<cuuint64_t>(blocks),
                              static_cast<cuuint64_t>(n2)};
  const cuuint64_t strides[3] = {static_cast<cuuint64_t>(n1 > 1 ? s1 * 2 : 1024), 128,
                                 static_cast<cuuint64_t>(n2 > 1 ? s2 * 2 : 1024)};
  const cuuint32_t box[4] = {64, b1, b2, 1};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, box,
             estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int outcome(cudaError_t e) {
  if (e == cudaSuccess) return KLT_OK;
  cudaGetLastError();  // reported here, not to the caller's next call
  return KLT_ERR_CUDA;
}

void free_all(klt_latent* h) {
  cudaFree(h->inv_freq);
  cudaFree(h->gamma);
  cudaFree(h->err);
  delete h;
}

template <typename Kernel, typename... Args>
cudaError_t launch_pdl(Kernel k, unsigned grid, unsigned block, cudaStream_t s, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k, args...);
}

}  // namespace

extern "C" {

int klt_latent_create(const klt_latent_dims* d, const float* inv_freq, const void* gamma,
                      klt_latent** out) {
  if (!out) return KLT_ERR_INVALID_ARG;
  *out = nullptr;
  if (!d || !inv_freq) return KLT_ERR_INVALID_ARG;
  const int rc = check_dims(d);
  if (rc) return rc;
  if (!aligned(inv_freq, 4) || !aligned(gamma, 2)) return KLT_ERR_ALIGN;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return KLT_ERR_CUDA;
  cudaDeviceProp prop;
  if (cudaGetDeviceProperties(&prop, dev) != cudaSuccess) return KLT_ERR_CUDA;
  if (prop.major != 10 || prop.minor != 3) return KLT_ERR_UNSUPPORTED;
  if (!get_encode()) return KLT_ERR_CUDA;
  if (!prepare_attend() || !prepare_prefill()) return KLT_ERR_UNSUPPORTED;
  klt_latent* h = new (std::nothrow) klt_latent();
  if (!h) return KLT_ERR_OOM;
  h->d = *d;
  h->device = dev;
  h->num_sms = prop.multiProcessorCount;
  while ((1 << h->page_log2) < d->page) ++h->page_log2;
  const size_t freqs = d->rope / 2 * sizeof(float), gammas = d->latent * sizeof(__nv_bfloat16);
  if (cudaMalloc(reinterpret_cast<void**>(&h->inv_freq), freqs) != cudaSuccess ||
      (gamma && cudaMalloc(reinterpret_cast<void**>(&h->gamma), gammas) != cudaSuccess) ||
      cudaMalloc(reinterpret_cast<void**>(&h->err), 4) != cudaSuccess) {
    cudaGetLastError();  // the failed allocation is reported here, not to the caller's next call
    free_all(h);
    return KLT_ERR_OOM;
  }
  if (cudaMemcpyAsync(h->inv_freq, inv_freq, freqs, cudaMemcpyDeviceToDevice, 0) != cudaSuccess ||
      (gamma &&
       cudaMemcpyAsync(h->gamma, gamma, gammas, cudaMemcpyDeviceToDevice, 0) != cudaSuccess) ||
      cudaMemsetAsync(h->err, 0, 4, 0) != cudaSuccess || cudaDeviceSynchronize() != cudaSuccess) {
    cudaGetLastError();
    free_all(h);
    return KLT_ERR_CUDA;
  }
  *out = h;
  return KLT_OK;
}

int klt_latent_append(klt_latent* h, const klt_latent_append_args* a, void* stream) {
  if (!h || !a || a->T < 0) return KLT_ERR_INVALID_ARG;
  if (a->T == 0) return KLT_OK;
  const klt_latent_dims& d = h->d;
  const int width = d.latent + d.rope;
  if (!a->kv || !a->positions || (!a->cache && !a->kv_out && !a->q_out) ||
      !a->cache != !a->slots || !a->q != !a->q_out || a->pages < 0)
    return KLT_ERR_INVALID_ARG;
  if (a->kv_dtype != KLT_DT_BF16 && a->kv_dtype != KLT_DT_F32) return KLT_ERR_UNSUPPORTED;
  if (a->pages > (0x7FFFFFFFll >> h->page_log2)) return KLT_ERR_UNSUPPORTED;
  if (a->ld_kv < 0 || a->page_stride < 0 || a->row_stride < 0 || a->ld_kv_out < 0 ||
      a->q_token < 0 || a->q_head < 0 || a->q_out_token < 0 || a->q_out_head < 0)
    return KLT_ERR_INVALID_ARG;
  if (a->cache && !disjoint(a->pages, a->page_stride, d.page, a->row_stride, width))
    return KLT_ERR_INVALID_ARG;
  if (a->kv_out && !disjoint(a->T, a->ld_kv_out, 1, 0, width)) return KLT_ERR_INVALID_ARG;
  if (a->q_out && !disjoint(a->T, a->q_out_token, d.heads, a->q_out_head, d.rope))
    return KLT_ERR_INVALID_ARG;
  const int64_t kv_unit = a->kv_dtype == KLT_DT_F32 ? 4 : 8;
  if (!aligned(a->kv, 16) || !aligned(a->cache, 16) || !aligned(a->kv_out, 16) ||
      !aligned(a->q, 16) || !aligned(a->q_out, 16) || !aligned(a->positions, 8) ||
      !aligned(a->slots, 8) || a->ld_kv % kv_unit || a->page_stride % 8 || a->row_stride % 8 ||
      a->ld_kv_out % 8 || a->q_token % 8 || a->q_head % 8 || a->q_out_token % 8 ||
      a->q_out_head % 8)
    return KLT_ERR_ALIGN;
  const int rc = check_device(h);
  if (rc) return rc;
  AppendParams p = {};
  p.kv = a->kv;
  p.positions = a->positions;
  p.slots = a->slots;
  p.inv_freq = h->inv_freq;
  p.gamma = h->gamma;
  p.cache = static_cast<__nv_bfloat16*>(a->cache);
  p.kv_out = static_cast<__nv_bfloat16*>(a->kv_out);
  p.q = static_cast<const __nv_bfloat16*>(a->q);
  p.q_out = static_cast<__nv_bfloat16*>(a->q_out);
  p.ld_kv = a->ld_kv;
  p.page_stride = a->page_stride;
  p.row_stride = a->row_stride;
  p.ld_kv_out = a->ld_kv_out;
  p.q_token = a->q_token;
  p.q_head = a->q_head;
  p.q_out_token = a->q_out_token;
  p.q_out_head = a->q_out_head;
  p.n_slots = a->pages << h->page_log2;
  p.T = a->T;
  p.R = d.latent;
  p.rope = d.rope;
  p.H = d.heads;
  p.page_log2 = h->page_log2;
  p.eps = d.eps;
  const bool f32 = a->kv_dtype == KLT_DT_F32, nb = d.pairs == KLT_ROPE_NEIGHBOURS;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  // four warps where the queries' units are no more; two tokens to a block where there are enough
  // of them to fill the SMs that way
  const unsigned threads = p.q && d.heads * (d.rope / 16) > 128 ? 256 : 128;
  const bool two = threads == 256 && a->T > APPEND_TWO;
  const unsigned grid = two ? (a->T + 1u) / 2 : a->T;
  auto launch = [&](auto kernel) { return outcome(launch_pdl(kernel, grid, threads, s, p)); };
  if (two)
    return f32 ? nb ? launch(append_kernel<true, true, 2>) : launch(append_kernel<true, false, 2>)
               : nb ? launch(append_kernel<false, true, 2>)
                    : launch(append_kernel<false, false, 2>);
  return f32 ? nb ? launch(append_kernel<true, true, 1>) : launch(append_kernel<true, false, 1>)
             : nb ? launch(append_kernel<false, true, 1>) : launch(append_kernel<false, false, 1>);
}

int klt_latent_workspace(const klt_latent* h, int32_t B, int32_t T, uint64_t* bytes) {
  if (!h || !bytes || B < 1 || T < 0) return KLT_ERR_INVALID_ARG;
  *bytes = attend_workspace(h->num_sms, h->d.latent);
  return KLT_OK;
}

int klt_latent_attend(klt_latent* h, const klt_latent_attend_args* a, const klt_latent_debug* dbg,
                      void* stream) {
  if (!h || !a || a->B < 1 || a->T < 0 || a->max_pages < 0 || a->pages < 0)
    return KLT_ERR_INVALID_ARG;
  if (dbg && (dbg->stall_after_tiles < 0 || dbg->timeout_ms < 0)) return KLT_ERR_INVALID_ARG;
  if (a->T == 0) return KLT_OK;
  const klt_latent_dims& d = h->d;
  const int width = d.latent + d.rope;
  if (!a->q || !a->out || !a->seq_lens || !a->workspace ||
      (!a->block_table && a->max_pages > 0) || (!a->cache && a->pages > 0) ||
      (!a->cu_q && a->T != a->B))
    return KLT_ERR_INVALID_ARG;
  if (a->q_token < 0 || a->q_head < 0 || a->page_stride < 0 || a->row_stride < 0 ||
      a->ld_table < 0 || a->out_token < 0 || a->out_head < 0)
    return KLT_ERR_INVALID_ARG;
  if ((a->B > 1 && a->ld_table < a->max_pages) ||
      !disjoint(a->pages, a->page_stride, d.page, a->row_stride, width) ||
      !disjoint(a->T, a->out_token, d.heads, a->out_head, d.latent))
    return KLT_ERR_INVALID_ARG;
  if (a->pages > (MOST >> h->page_log2) || a->max_pages > (MOST >> h->page_log2) ||
      a->T > MOST / d.heads || a->page_stride >= MAX_STRIDE ||
      a->row_stride >= MAX_STRIDE || a->q_token >= MAX_STRIDE || a->q_head >= MAX_STRIDE)
    return KLT_ERR_UNSUPPORTED;
  if (!aligned(a->q, 16) || !aligned(a->cache, 16) || !aligned(a->out, 16) ||
      !aligned(a->workspace, 16) || !aligned(a->lse, 4) || !aligned(a->block_table, 4) ||
      !aligned(a->seq_lens, 4) || !aligned(a->cu_q, 4) || a->q_token % 8 || a->q_head % 8 ||
      a->page_stride % 8 || a->row_stride % 8 || a->out_token % 8 || a->out_head % 8)
    return KLT_ERR_ALIGN;
  if (a->workspace_bytes < attend_workspace(h->num_sms, h->d.latent)) return KLT_ERR_INVALID_ARG;
  const int rc = check_device(h);
  if (rc) return rc;
  AttendParams p = {};
  p.q = static_cast<const __nv_bfloat16*>(a->q);
  p.table = a->block_table;
  p.lens = a->seq_lens;
  p.cu_q = a->cu_q;
  p.out = static_cast<__nv_bfloat16*>(a->out);
  p.lse = a->lse;
  p.part = static_cast<float*>(a->workspace);
  p.q_token = a->q_token;
  p.q_head = a->q_head;
  p.ld_table = a->ld_table;
  p.out_token = a->out_token;
  p.out_head = a->out_head;
  p.B = a->B;
  p.T = a->T;
  p.H = d.heads;
  p.R = d.latent;
  p.rope = d.rope;
  p.page_log2 = h->page_log2;
  p.max_pages = a->pages > 0 ? a->max_pages : 0;
  p.pages = static_cast<int>(a->pages);
  p.scale = d.scale * 1.4426950408889634f;
  p.stall = dbg ? dbg->stall_after_tiles : 0;
  p.err = h->err;
  p.timeout = timeout_cycles(dbg);
  // the cache's latent part by 64 columns as a direction of its own, so that one copy brings two
  // boxes of them, and its position part, which may be narrower than a box
  const uint32_t keys = d.page < 64 ? d.page : 64;
  CUtensorMap latents = {}, ropes = {};
  if (a->pages > 0 &&
      (!encode_columns(&latents, a->cache, d.latent / 64, d.page, a->row_stride, a->pages,
                       a->page_stride, keys, keys == 64 ? 2 : 1) ||
       !encode_rows(&ropes, static_cast<const __nv_bfloat16*>(a->cache) + d.latent, d.rope, d.page,
                    a->row_stride, a->pages, a->page_stride, keys, 1)))
    return KLT_ERR_CUDA;
  // queries by bulk copies: 64 rows where (token, head) is one direction, else the heads that a
  // token's 64 rows are made of; heads that are no multiple of 8 at other strides are copied by
  // threads (7 us a tile of rows)
  CUtensorMap queries = {};
  const int heads = d.heads & -d.heads;  // largest power of two that divides them
  if (d.heads == 1 ? a->T == 1 || a->q_token > 0
                   : a->q_head > 0 && (a->T == 1 || a->q_token == d.heads * a->q_head)) {
    p.q_packed = true;
    p.q_box = 64;
    if (!encode_rows(&queries, a->q, width, static_cast<int64_t>(a->T) * d.heads,
                     d.heads > 1 ? a->q_head : a->q_token, 1, 0, 64, 1))
      return KLT_ERR_CUDA;
  } else if (heads >= 8 && a->q_token > 0 && a->q_head > 0) {
    p.q_box = heads < 64 ? heads : 64;
    if (!encode_rows(&queries, a->q, width, d.heads, a->q_head, a->T, a->q_token, p.q_box, 1))
      return KLT_ERR_CUDA;
  }
  return outcome(
      launch_attend(latents, ropes, queries, p, h->num_sms, static_cast<cudaStream_t>(stream)));
}

int klt_latent_prefill(klt_latent* h, const klt_latent_prefill_args* a,
                       const klt_latent_debug* dbg, void* stream) {
  if (!h || !a || a->B < 1 || a->T < 0 || a->S < 0) return KLT_ERR_INVALID_ARG;
  if (dbg && (dbg->stall_after_tiles < 0 || dbg->timeout_ms < 0)) return KLT_ERR_INVALID_ARG;
  if (a->T == 0) return KLT_OK;
  const klt_latent_dims& d = h->d;
  if (!a->q || !a->out || !a->cu_q || !a->cu_k ||
      (a->S > 0 && (!a->k || !a->v || !a->k_rope)))
    return KLT_ERR_INVALID_ARG;
  const bool heads = d.heads > 1, queries = a->T > 1, keys = a->S > 1;
  if (a->q_token < queries || a->q_head < heads || a->k_token < keys || a->k_head < heads ||
      a->v_token < keys || a->v_head < heads || a->ld_k_rope < keys || a->out_token < 0 ||
      a->out_head < 0)
    return KLT_ERR_INVALID_ARG;
  if (!disjoint(a->T, a->out_token, d.heads, a->out_head, d.value)) return KLT_ERR_INVALID_ARG;
  const int64_t tiles = (a->T + PREFILL_ROWS - 1ll) / PREFILL_ROWS + a->B;
  if (a->T > MOST / d.heads || a->S > MOST || tiles > 0x3FFFFFFFll / d.heads ||
      a->q_token >= MAX_STRIDE || a->q_head >= MAX_STRIDE || a->k_token >= MAX_STRIDE ||
      a->k_head >= MAX_STRIDE || a->v_token >= MAX_STRIDE || a->v_head >= MAX_STRIDE ||
      a->ld_k_rope >= MAX_STRIDE)
    return KLT_ERR_UNSUPPORTED;
  if (!aligned(a->q, 16) || !aligned(a->k, 16) || !aligned(a->v, 16) || !aligned(a->k_rope, 16) ||
      !aligned(a->out, 16) || !aligned(a->lse, 4) || !aligned(a->cu_q, 4) ||
      !aligned(a->cu_k, 4) || a->q_token % 8 || a->q_head % 8 || a->k_token % 8 ||
      a->k_head % 8 || a->v_token % 8 || a->v_head % 8 || a->ld_k_rope % 8 || a->out_token % 8 ||
      a->out_head % 8)
    return KLT_ERR_ALIGN;
  const int rc = check_device(h);
  if (rc) return rc;
  PrefillParams p = {};
  p.cu_q = a->cu_q;
  p.cu_k = a->cu_k;
  p.out = static_cast<__nv_bfloat16*>(a->out);
  p.lse = a->lse;
  p.out_token = a->out_token;
  p.out_head = a->out_head;
  p.B = a->B;
  p.T = a->T;
  p.S = a->S;
  p.H = d.heads;
  p.nope = d.nope;
  p.rope = d.rope;
  p.value = d.value;
  p.causal = a->causal;
  // Units of a number are alike in length, and the last numbers are a sequence's first queries,
  // which see few keys: with all heads of a number side by side a launch ends with short units
  // (12 ragged sequences 281 -> 258 us).  But all these heads' keys and values are read again for
  // the next number, so no more than half of L2 holds, or 16 (8192 tokens of 64 heads: 16 side by
  // side 775 us, 32 790, all 803, one 816; 2048 queries of 128 K keys 6.53, 6.61, 6.68, 6.51 ms).
  const int64_t head_bytes = static_cast<int64_t>(a->S) * (d.nope + d.value) * 2;
  int64_t fit = (64ll << 20) / (head_bytes + 1);
  if (fit < 16) fit = 16;
  const int groups = static_cast<int>((p.H + fit - 1) / fit);
  p.side = (p.H + groups - 1) / groups;
  p.scale = d.scale * 1.4426950408889634f;
  p.stall = dbg ? dbg->stall_after_tiles : 0;
  p.err = h->err;
  p.timeout = timeout_cycles(dbg);
  // several of its waits last for a unit: its threads that have no queries, the next unit's search
  p.timeout += (a->S / 128 + 1) * TILE_CYCLES;
  CUtensorMap q, k = {}, v = {}, k_rope = {};
  if (!encode_rows(&q, a->q, d.nope + d.rope, d.heads, a->q_head, a->T, a->q_token, 1, 128))
    return KLT_ERR_CUDA;
  if (a->S > 0 &&
      (!encode_rows(&k, a->k, d.nope, d.heads, a->k_head, a->S, a->k_token, 1, 64) ||
       !encode_rows(&v, a->v, d.value, d.heads, a->v_head, a->S, a->v_token, 1, 128) ||
       !encode_rows(&k_rope, a->k_rope, d.rope, 1, 0, a->S, a->ld_k_rope, 1, 64)))
    return KLT_ERR_CUDA;
  return outcome(launch_prefill(q, k, v, k_rope, p, static_cast<unsigned>(tiles),
                                static_cast<cudaStream_t>(stream)));
}

int klt_latent_status(klt_latent* h) {
  if (!h) return KLT_ERR_INVALID_ARG;
  int e = 0;
  if (cudaMemcpy(&e, h->err, 4, cudaMemcpyDeviceToHost) != cudaSuccess) return KLT_ERR_CUDA;
  return e & DEV_ERR_TIMEOUT ? KLT_ERR_DEVICE_TIMEOUT : KLT_OK;
}

int klt_latent_destroy(klt_latent* h) {
  if (!h) return KLT_OK;
  int dev = 0;
  const bool other = cudaGetDevice(&dev) == cudaSuccess && dev != h->device;
  if (other) cudaSetDevice(h->device);
  const cudaError_t e = cudaDeviceSynchronize();
  free_all(h);
  if (other) cudaSetDevice(dev);
  return e == cudaSuccess ? KLT_OK : KLT_ERR_CUDA;
}

}  // extern "C"
