// The norms before and after a block, fused with the gate, the residual scale and the e4m3
// quantisation of the next operand; and the quantiser alone (sm_103a).
//
//   u  = RMSNorm(y) * gamma_post            (fp32 statistics of the row)
//   h' = res_scale * h + branch_scale * gate * u
//   n  = RMSNorm(h') * gamma_pre            (statistics of the unrounded fp32 h')
//   q, s: per 128 columns s = amax / 448 (1 where that is 0), codes e4m3(fp32(n / s))
//
// Both are bound by memory: every value is read once and written once, and a row stays in
// registers between its two reductions.  h' is rounded to its stored type and n to bf16 or
// e4m3 once each, n from the unrounded h' (one rounding on each path, not two in a row).
#include "klt_linear.cuh"

#include "../../include/klt.h"

namespace klt {
namespace {

// ------------------------------------------------------------------ eight values of a row
// A row of C elements is handled in vectors of eight.  `wide` says that the row's start is
// 16-byte aligned, so a whole vector is one (bf16) or two (fp32) 16-byte accesses; the last
// partial vector and unaligned rows go element by element.  Elements past C read as 0.
// Plain loads, not the read-only path: the launch may begin while the kernel that writes
// these tensors still runs, and h_out may be h.
KLT_DEV void load8(const void* base, bool f32, int64_t off, int col, int C, bool wide, float* v) {
  if (f32) {
    const float* p = static_cast<const float*>(base) + off + col;
    if (wide && col + 8 <= C) {
      const float4 a = reinterpret_cast<const float4*>(p)[0];
      const float4 b = reinterpret_cast<const float4*>(p)[1];
      v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
      v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = col + i < C ? p[i] : 0.f;
    }
  } else {
    const __nv_bfloat16* p = static_cast<const __nv_bfloat16*>(base) + off + col;
    if (wide && col + 8 <= C) {
      const uint4 a = *reinterpret_cast<const uint4*>(p);
      const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = col + i < C ? __bfloat162float(p[i]) : 0.f;
    }
  }
}
KLT_DEV void store8(void* base, bool f32, int64_t off, int col, int C, bool wide,
                    const float* v) {
  if (f32) {
    float* p = static_cast<float*>(base) + off + col;
    if (wide && col + 8 <= C) {
      reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
      reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (col + i < C) p[i] = v[i];
    }
  } else {
    __nv_bfloat16* p = static_cast<__nv_bfloat16*>(base) + off + col;
    if (wide && col + 8 <= C) {
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&b);
      }
      *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (col + i < C) p[i] = __float2bfloat16(v[i]);
    }
  }
}

// The group's scale and this lane's eight codes: the 16 lanes of a half warp hold one group
// of 128 columns.  The largest magnitude is taken on the bit patterns, so a group that holds
// an infinity or a NaN gets a scale that is not finite and dequantises to NaN as a whole.
KLT_DEV uint2 quant8(const float* v, float& s_out) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
#pragma unroll
  for (int o = 8; o; o >>= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
  float s = group_scale(m);
  s_out = s;
  const float k = rescale(s), inv = 1.0f / s;
  float t[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) t[i] = quot_group(v[i] * k, s, inv);
  return make_uint2(f32x2_to_e4m3x2(t[0], t[1]) | (f32x2_to_e4m3x2(t[2], t[3]) << 16),
                    f32x2_to_e4m3x2(t[4], t[5]) | (f32x2_to_e4m3x2(t[6], t[7]) << 16));
}
KLT_DEV void store_codes(uint8_t* q, int64_t off, int col, int C, bool wide, uint2 c) {
  uint8_t* p = q + off + col;
  if (wide && col + 8 <= C) {
    *reinterpret_cast<uint2*>(p) = c;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (col + i < C) p[i] = static_cast<uint8_t>((i < 4 ? c.x : c.y) >> (8 * (i & 3)));
  }
}

// ------------------------------------------------------------------ the quantiser
struct QuantParams {
  const void* x;
  uint8_t* q;
  float* s;
  int64_t ld_x, ld_q;
  int64_t items;  // rows x groups
  int K, G;
  bool f32, wide_x, wide_q;
};

// One half warp per group of 128 columns, U groups per half warp with their loads in flight
// together.
template <int U>
__global__ void __launch_bounds__(256) quant_kernel(QuantParams p) {
  pdl_trigger();
  pdl_wait();
  const int hw = threadIdx.x >> 4, lane = threadIdx.x & 15;
  const int64_t base = static_cast<int64_t>(blockIdx.x) * (16 * U) + hw;
  float v[U][8];
  int64_t row[U];
  int col[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t it = base + 16 * u;
    if (it < p.items) {
      row[u] = it / p.G;
      col[u] = static_cast<int>(it - row[u] * p.G) * 128 + lane * 8;
      load8(p.x, p.f32, row[u] * p.ld_x, col[u], p.K, p.wide_x, v[u]);
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t it = base + 16 * u;
    // both halves of a warp take part in the shuffles; a half past the end holds zeros
    if (it >= p.items) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[u][i] = 0.f;
    }
    float s;
    const uint2 c = quant8(v[u], s);
    if (it < p.items) {
      store_codes(p.q, row[u] * p.ld_q, col[u], p.K, p.wide_q, c);
      if (lane == 0) p.s[it] = s;
    }
  }
}

// ------------------------------------------------------------------ the block norms
struct NormParams {
  const void *h, *y, *gate, *gamma_post, *gamma_pre;
  void *h_out, *n;
  uint8_t* q;
  float* s;
  int64_t ld_h, ld_y, gate_row, gate_col, ld_h_out, ld_n, ld_q;
  int H, G;
  float eps, res_scale, branch_scale;
  bool h_f32, y_f32, gate_f32, sigmoid;
  bool wide_h, wide_y, wide_gate, wide_gpost, wide_gpre, wide_h_out, wide_n, wide_q;
};

// Sum over the block of one value per thread; `part` is 32 floats of its own.
KLT_DEV float block_sum(float v, float* part) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  if (lane == 0) part[warp] = v;
  __syncthreads();
  v = lane < warps ? part[lane] : 0.f;
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

// One block per row, VPT vectors of eight columns per thread.
template <int VPT>
__global__ void __launch_bounds__(1024 / (VPT > 1 ? 2 : 1)) norm_kernel(NormParams p) {
  __shared__ float part[2][32];
  pdl_trigger();
  const int64_t row = blockIdx.x;
  const int nt = blockDim.x;
  float u[VPT][8], h[VPT][8];
  pdl_wait();
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = (threadIdx.x + i * nt) * 8;
    if (c < p.H) {
      if (p.y) load8(p.y, p.y_f32, row * p.ld_y, c, p.H, p.wide_y, u[i]);
      load8(p.h, p.h_f32, row * p.ld_h, c, p.H, p.wide_h, h[i]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) u[i][j] = h[i][j] = 0.f;
    }
  }
  if (p.y) {
    float r = 1.0f;
    if (p.gamma_post) {
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) ss = fmaf(u[i][j], u[i][j], ss);
      r = 1.0f / sqrtf(block_sum(ss, part[0]) / static_cast<float>(p.H) + p.eps);
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = (threadIdx.x + i * nt) * 8;
      if (c < p.H) {
        float g[8];
        if (p.gamma_post) {
          load8(p.gamma_post, false, 0, c, p.H, p.wide_gpost, g);
#pragma unroll
          for (int j = 0; j < 8; ++j) u[i][j] = u[i][j] * r * g[j];
        }
        if (p.gate) {
          if (p.gate_col == 1) {
            load8(p.gate, p.gate_f32, row * p.gate_row, c, p.H, p.wide_gate, g);
          } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const int64_t o =
                  row * p.gate_row + static_cast<int64_t>(min(c + j, p.H - 1)) * p.gate_col;
              g[j] = p.gate_f32 ? static_cast<const float*>(p.gate)[o]
                                : __bfloat162float(static_cast<const __nv_bfloat16*>(p.gate)[o]);
            }
          }
#pragma unroll
          for (int j = 0; j < 8; ++j)
            u[i][j] *= p.sigmoid ? 1.0f / (1.0f + expf(-g[j])) : g[j];
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
          h[i][j] = c + j < p.H ? fmaf(p.branch_scale, u[i][j], p.res_scale * h[i][j]) : 0.f;
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = (threadIdx.x + i * nt) * 8;
#pragma unroll
      for (int j = 0; j < 8; ++j) h[i][j] = c + j < p.H ? p.res_scale * h[i][j] : 0.f;
    }
  }
  if (p.h_out) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = (threadIdx.x + i * nt) * 8;
      if (c < p.H) store8(p.h_out, p.h_f32, row * p.ld_h_out, c, p.H, p.wide_h_out, h[i]);
    }
  }
  if (!p.n && !p.q) return;
  if (p.gamma_pre) {
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) ss = fmaf(h[i][j], h[i][j], ss);
    const float r = 1.0f / sqrtf(block_sum(ss, part[1]) / static_cast<float>(p.H) + p.eps);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = (threadIdx.x + i * nt) * 8;
      if (c < p.H) {
        float g[8];
        load8(p.gamma_pre, false, 0, c, p.H, p.wide_gpre, g);
#pragma unroll
        for (int j = 0; j < 8; ++j) h[i][j] = c + j < p.H ? h[i][j] * r * g[j] : 0.f;
      }
    }
  }
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = (threadIdx.x + i * nt) * 8;
    if (p.n && c < p.H) store8(p.n, false, row * p.ld_n, c, p.H, p.wide_n, h[i]);
    if (p.q) {  // 16 neighbouring threads hold one group of 128 columns
      float s;
      const uint2 codes = quant8(h[i], s);
      if (c < p.H) {
        store_codes(p.q, row * p.ld_q, c, p.H, p.wide_q, codes);
        if ((threadIdx.x & 15) == 0) p.s[row * p.G + c / 128] = s;
      }
    }
  }
}

template <typename Kernel, typename Params>
cudaError_t launch_pdl(Kernel k, unsigned grid, unsigned block, cudaStream_t s, const Params& p) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k, p);
}

bool aligned(const void* p, uintptr_t bytes) {
  return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0;
}
bool known(int32_t dtype) { return dtype == KLT_DT_BF16 || dtype == KLT_DT_F32; }
uintptr_t esize(int32_t dtype) { return dtype == KLT_DT_F32 ? 4 : 2; }
// Every row of a tensor starts on `bytes` bytes.
bool wide(const void* p, int64_t ld, uintptr_t es, uintptr_t bytes) {
  return aligned(p, bytes) && (static_cast<uint64_t>(ld) * es) % bytes == 0;
}
// Rows of `cols` elements `ld` apart do not overlap (the stride of a single row is free).
bool rows_ok(int64_t ld, int32_t rows, int32_t cols) { return rows <= 1 || ld >= cols; }

}  // namespace
}  // namespace klt

using namespace klt;

extern "C" int klt_quantize(const void* x, int32_t x_dtype, int64_t ld_x, int32_t M, int32_t K,
                            uint8_t* q, int64_t ld_q, float* s, void* stream) {
  if (M < 0 || K < 1) return KLT_ERR_INVALID_ARG;
  if (!known(x_dtype)) return KLT_ERR_UNSUPPORTED;
  if (M == 0) return KLT_OK;
  if (!x || !q || !s) return KLT_ERR_INVALID_ARG;
  if (ld_x < 0 || !rows_ok(ld_q, M, K)) return KLT_ERR_INVALID_ARG;
  if (!aligned(x, esize(x_dtype)) || !aligned(s, 4)) return KLT_ERR_ALIGN;
  QuantParams p = {};
  p.x = x;
  p.q = q;
  p.s = s;
  p.ld_x = ld_x;
  p.ld_q = ld_q;
  p.K = K;
  p.G = (K + 127) / 128;
  p.items = static_cast<int64_t>(M) * p.G;
  p.f32 = x_dtype == KLT_DT_F32;
  p.wide_x = wide(x, ld_x, esize(x_dtype), 16);
  p.wide_q = wide(q, ld_q, 1, 8);
  // four groups per half warp hide the load latency once the groups fill the device
  // anyway; below that one group each spreads them over more SMs
  const bool many = p.items >= 4 * 16 * 152 * 4;
  const int64_t blocks = (p.items + (many ? 64 : 16) - 1) / (many ? 64 : 16);
  if (blocks > 0x7FFFFFFF) return KLT_ERR_UNSUPPORTED;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = many ? launch_pdl(quant_kernel<4>, static_cast<unsigned>(blocks), 256, st, p)
                             : launch_pdl(quant_kernel<1>, static_cast<unsigned>(blocks), 256, st, p);
  return e == cudaSuccess ? KLT_OK : KLT_ERR_CUDA;
}

extern "C" int klt_block_norm(const klt_block_norm_args* a, void* stream) {
  if (!a) return KLT_ERR_INVALID_ARG;
  if (a->M < 0 || a->H < 1 || !(a->eps >= 0.f)) return KLT_ERR_INVALID_ARG;
  if (a->H > KLT_BLOCK_NORM_MAX_H) return KLT_ERR_UNSUPPORTED;
  if (!known(a->h_dtype) || !known(a->y_dtype) || !known(a->gate_dtype))
    return KLT_ERR_UNSUPPORTED;
  if (a->M == 0) return KLT_OK;
  if (!a->h_out && !a->n && !a->q) return KLT_ERR_INVALID_ARG;
  if ((a->q == nullptr) != (a->s == nullptr)) return KLT_ERR_INVALID_ARG;
  if (!a->y && (a->gate || a->gamma_post)) return KLT_ERR_INVALID_ARG;
  if (!a->h) return KLT_ERR_INVALID_ARG;
  const int32_t M = a->M, H = a->H;
  if (a->ld_h < 0 || a->ld_y < 0 || a->gate_row < 0 || a->gate_col < 0 ||
      (a->h_out && !rows_ok(a->ld_h_out, M, H)) || (a->n && !rows_ok(a->ld_n, M, H)) ||
      (a->q && !rows_ok(a->ld_q, M, H)))
    return KLT_ERR_INVALID_ARG;
  const uintptr_t he = esize(a->h_dtype), ye = esize(a->y_dtype), ge = esize(a->gate_dtype);
  if (!aligned(a->h, he) || !aligned(a->y, ye) || !aligned(a->gate, ge) ||
      !aligned(a->h_out, he) || !aligned(a->n, 2) || !aligned(a->gamma_post, 2) ||
      !aligned(a->gamma_pre, 2) || !aligned(a->s, 4))
    return KLT_ERR_ALIGN;
  NormParams p = {};
  p.h = a->h;
  p.y = a->y;
  p.gate = a->gate;
  p.gamma_post = a->gamma_post;
  p.gamma_pre = a->gamma_pre;
  p.h_out = a->h_out;
  p.n = a->n;
  p.q = a->q;
  p.s = a->s;
  p.ld_h = a->ld_h;
  p.ld_y = a->ld_y;
  p.gate_row = a->gate_row;
  p.gate_col = a->gate_col;
  p.ld_h_out = a->ld_h_out;
  p.ld_n = a->ld_n;
  p.ld_q = a->ld_q;
  p.H = H;
  p.G = (H + 127) / 128;
  p.eps = a->eps;
  p.res_scale = a->res_scale;
  p.branch_scale = a->branch_scale;
  p.h_f32 = a->h_dtype == KLT_DT_F32;
  p.y_f32 = a->y_dtype == KLT_DT_F32;
  p.gate_f32 = a->gate_dtype == KLT_DT_F32;
  p.sigmoid = a->gate_sigmoid != 0;
  p.wide_h = wide(a->h, a->ld_h, he, 16);
  p.wide_y = wide(a->y, a->ld_y, ye, 16);
  p.wide_gate = wide(a->gate, a->gate_row, ge, 16);
  p.wide_gpost = aligned(a->gamma_post, 16);
  p.wide_gpre = aligned(a->gamma_pre, 16);
  p.wide_h_out = wide(a->h_out, a->ld_h_out, he, 16);
  p.wide_n = wide(a->n, a->ld_n, 2, 16);
  p.wide_q = wide(a->q, a->ld_q, 1, 8);
  // one vector per thread while the row's vectors fit in a block, four above
  const int vecs = (H + 7) / 8;
  const int vpt = vecs <= 1024 ? 1 : 4;
  const int threads = ((vecs + vpt - 1) / vpt + 31) / 32 * 32;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (vpt == 1)
    e = launch_pdl(norm_kernel<1>, static_cast<unsigned>(M), threads, st, p);
  else
    e = launch_pdl(norm_kernel<4>, static_cast<unsigned>(M), threads, st, p);
  return e == cudaSuccess ? KLT_OK : KLT_ERR_CUDA;
}
