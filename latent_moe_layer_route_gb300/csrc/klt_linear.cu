// Host side of the FP8 linear layer: argument checks, the handle's re-laid-out weights, TMA
// descriptors and the choice of kernel.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <new>

#include "../../include/klt.h"
#include "klt_linear.cuh"

using namespace klt;

struct klt_linear {
  klt_linear_dims d;
  int device;
  int num_sms;
  int max_tiles;     // tiles of the token-major kernel that two pairs each share at once
  int clusters[4];   // clusters of 2^i CTAs of the feature-major kernel, one per SM, at once
  int NB, KB;        // row blocks and k-blocks of W
  uint8_t* w;        // tile-major image [NB, KB, 16384]
  float* ws;         // [NB + 1, KB], the last row zero
  int* err;          // device error word
  CUtensorMap wmap;  // the image as [NB * KB * 128, 128] bytes
};

namespace {

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

// Rows of `cols` bytes `ld` bytes apart; box of box_bytes x box_rows; bytes outside read as 0
// and are not written.
bool encode_bytes(CUtensorMap* m, const void* base, uint64_t rows, uint64_t cols, uint64_t ld,
                  uint32_t box_bytes, uint32_t box_rows, CUtensorMapSwizzle swizzle) {
  EncodeTiledFn enc = get_encode();
  if (!enc) return false;
  const cuuint64_t dims[2] = {cols, rows};
  const cuuint64_t strides[1] = {ld};
  const cuuint32_t box[2] = {box_bytes, box_rows};
  const cuuint32_t estr[2] = {1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box,
             estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
             swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool aligned(const void* p, uintptr_t bytes) {
  return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0;
}

// One thread per 16 bytes of the image: tile (rb, kb), row r, physical chunk c holds columns
// (c ^ (r & 7)) * 16 .. + 15 of the k-block.
__global__ void relayout_kernel(const uint8_t* w, uint8_t* img, int N, int K, int KB,
                                int64_t chunks) {
  for (int64_t i = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x; i < chunks;
       i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    const int c = static_cast<int>(i & 7), r = static_cast<int>(i >> 3) & 127;
    const int64_t tile = i >> 10;
    const int64_t row = tile / KB * 128 + r;
    const int64_t col = tile % KB * 128 + (c ^ (r & 7)) * 16;
    uint32_t v[4] = {0, 0, 0, 0};
    if (row < N) {
      const uint8_t* src = w + row * K + col;
#pragma unroll
      for (int j = 0; j < 16; ++j)
        if (col + j < K) v[j / 4] |= static_cast<uint32_t>(src[j]) << (8 * (j % 4));
    }
    reinterpret_cast<uint4*>(img)[i] = make_uint4(v[0], v[1], v[2], v[3]);
  }
}

int check_dims(const klt_linear_dims* d) {
  if (d->N < 1 || d->K < 1) return KLT_ERR_INVALID_ARG;
  if (d->N > (1 << 20) || d->K > (1 << 20)) return KLT_ERR_UNSUPPORTED;
  const int64_t nb = (d->N + 127) / 128, kb = (d->K + 127) / 128;
  if (nb * kb >= (1 << 24)) return KLT_ERR_UNSUPPORTED;  // 32-bit rows of the image's map
  if (d->act == KLT_ACT_NONE) {
    if (d->out_dtype != KLT_DT_BF16 && d->out_dtype != KLT_DT_F32) return KLT_ERR_UNSUPPORTED;
  } else if (d->act == KLT_ACT_SWIGLU) {
    if (d->N % 256) return KLT_ERR_UNSUPPORTED;
    if (d->out_dtype != KLT_DT_BF16 && d->out_dtype != KLT_DT_E4M3) return KLT_ERR_UNSUPPORTED;
  } else {
    return KLT_ERR_UNSUPPORTED;
  }
  return KLT_OK;
}

void free_all(klt_linear* h) {
  cudaFree(h->w);
  cudaFree(h->ws);
  cudaFree(h->err);
  delete h;
}

// Token tile and K split for M tokens: the fastest by a model of every form, in us.  Its
// constants are fits to sizes within 1 x 64 x 64 .. 8192 x 8192 x 8192, 6 to 18 forms each; over 298
// sizes, 118 of them not fitted to, its choices take 0.5 % longer than the fastest form on average,
// 28 % at worst (a short K, many tokens and few columns).
//   narrow kernel: the waves that its clusters need, each of a start (first: longer for wider
//     tiles) and its k-blocks, which take longer where two CTAs share an SM;
//   wide kernel: 1.5 + per wave of pairs its tile's end and k-blocks; two pairs that share a
//     tile take half of the k-blocks, and bring their parts together.
// E.g. 1 x 7168 x 2048: 4 parts 4.8 us, 8 parts 6.9; 98 x 256 x 429 SwiGLU: tiles of 16 in 4
// parts 3.1, of 64 in 4 parts 5.4; 2368 x 194 x 4096: tiles of 64 in 4 parts 8.7, of 128 in 4
// parts 15.5 (they run alone on their SMs, and 38 clusters of 4 are two waves), wide 17.6; 256 x
// 7168 x 7168: narrow 25.5, wide 27.9, by two pairs 21.0.
void choose(const klt_linear* h, int M, int* tile, int* split) {
  const bool act = h->d.act == KLT_ACT_SWIGLU;
  struct Cost {
    double first, kblock;
  };
  static const Cost costs[2][4] = {{{2.51, 0.29}, {3.01, 0.29}, {4.28, 0.34}, {5.65, 0.39}},
                                   {{2.80, 0.42}, {3.60, 0.47}, {4.78, 0.55}, {}}};
  double best = 0.0;
  auto offer = [&](int t, int parts, double us) {
    if (best == 0.0 || us < best) best = us, *tile = t, *split = parts;
  };
  for (int i = 0; i < (act ? 3 : 4); ++i) {
    const int bn = 16 << i;
    if (i > 0 && M <= bn / 4) break;  // three quarters of it empty: the smaller one is as good
    const int64_t units = static_cast<int64_t>(act ? h->NB / 2 : h->NB) * ((M + bn - 1) / bn);
    const bool alone = bn == (act ? 64 : 128);  // one CTA per SM
    if ((M + bn - 1) / bn > 65535) continue;    // the grid's second dimension
    for (int j = 0; j < 4 && (1 << j) <= h->KB; ++j) {
      const int one = h->clusters[j];
      // two per SM: leftovers of the GPCs make up two more clusters (74 of 4 and 32 of 8 run at
      // once, 75 and 36 do not)
      const int64_t room = alone ? one : 2 * one + (j >= 2 ? 2 : 0);
      const int64_t waves = (units + room - 1) / room;
      const int kb = (h->KB + (1 << j) - 1) >> j;
      offer(bn, 1 << j, costs[act][i].first + (waves - 1) * 3.4 +
                            waves * kb * costs[act][i].kblock * (alone || units <= one ? 1 : 1.47));
    }
  }
  const int64_t tiles = static_cast<int64_t>((M + 255) / 256) * ((h->NB + 1) / 2);
  const int64_t pairs = h->num_sms / 2;
  const double end = act ? 2.71 : 4.99;
  offer(256, 1, 1.5 + ((tiles + pairs - 1) / pairs) * (end + 0.43 * h->KB));
  if (h->KB >= 4 && tiles <= h->max_tiles) offer(256, 2, 5.63 + end + 0.43 * h->KB / 2);
}

}  // namespace

extern "C" {

int klt_linear_create(const klt_linear_dims* d, const void* w, const float* w_scale,
                      klt_linear** out) {
  if (!out) return KLT_ERR_INVALID_ARG;
  *out = nullptr;
  if (!d || !w || !w_scale) return KLT_ERR_INVALID_ARG;
  const int rc = check_dims(d);
  if (rc) return rc;
  if (!aligned(w_scale, 4)) return KLT_ERR_ALIGN;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return KLT_ERR_CUDA;
  cudaDeviceProp prop;
  if (cudaGetDeviceProperties(&prop, dev) != cudaSuccess) return KLT_ERR_CUDA;
  if (prop.major != 10 || prop.minor != 3) return KLT_ERR_UNSUPPORTED;
  if (!get_encode()) return KLT_ERR_CUDA;
  int max_tiles = 0, clusters[4] = {};
  if (!prepare_linear_narrow(clusters) || !prepare_linear_wide(&max_tiles))
    return KLT_ERR_UNSUPPORTED;

  klt_linear* h = new (std::nothrow) klt_linear();
  if (!h) return KLT_ERR_OOM;
  h->d = *d;
  h->device = dev;
  h->num_sms = prop.multiProcessorCount;
  h->max_tiles = max_tiles;
  for (int i = 0; i < 4; ++i) h->clusters[i] = clusters[i];
  h->NB = (d->N + 127) / 128;
  h->KB = (d->K + 127) / 128;
  const int64_t tiles = static_cast<int64_t>(h->NB) * h->KB;
  if (cudaMalloc(reinterpret_cast<void**>(&h->w), tiles * LIN_TILE_BYTES) != cudaSuccess ||
      cudaMalloc(reinterpret_cast<void**>(&h->ws), (tiles + h->KB) * 4) != cudaSuccess ||
      cudaMalloc(reinterpret_cast<void**>(&h->err), 4) != cudaSuccess) {
    cudaGetLastError();  // the failed allocation is reported here, not to the caller's next call
    free_all(h);
    return KLT_ERR_OOM;
  }
  const int64_t chunks = tiles * (LIN_TILE_BYTES / 16);
  const unsigned blocks =
      static_cast<unsigned>(chunks / 256 < 65536 ? (chunks + 255) / 256 : 65536);
  relayout_kernel<<<blocks, 256>>>(static_cast<const uint8_t*>(w), h->w, d->N, d->K, h->KB,
                                   chunks);
  if (cudaGetLastError() != cudaSuccess ||
      cudaMemsetAsync(h->ws + tiles, 0, h->KB * 4ll, 0) != cudaSuccess ||
      cudaMemcpyAsync(h->ws, w_scale, tiles * 4, cudaMemcpyDeviceToDevice, 0) != cudaSuccess ||
      cudaMemsetAsync(h->err, 0, 4, 0) != cudaSuccess || cudaDeviceSynchronize() != cudaSuccess ||
      !encode_bytes(&h->wmap, h->w, tiles * 128, 128, 128, 128, 128, CU_TENSOR_MAP_SWIZZLE_NONE)) {
    free_all(h);
    return KLT_ERR_CUDA;
  }
  *out = h;
  return KLT_OK;
}

int klt_linear_forward(klt_linear* h, const uint8_t* xq, int64_t ld_xq, const float* xs,
                       int32_t M, void* out, int64_t ld_out, float* out_s,
                       const klt_linear_debug* dbg, void* stream) {
  if (!h || M < 0 || M > (1 << 22)) return KLT_ERR_INVALID_ARG;
  if (dbg && (dbg->stall_after_kblocks < 0 || dbg->timeout_ms < 0 || dbg->force_split < 0))
    return KLT_ERR_INVALID_ARG;
  if (M == 0) return KLT_OK;
  const bool act = h->d.act == KLT_ACT_SWIGLU;
  const int width = act ? h->d.N / 2 : h->d.N;
  const bool codes = h->d.out_dtype == KLT_DT_E4M3;
  if (!xq || !xs || !out || (codes && !out_s)) return KLT_ERR_INVALID_ARG;
  const uintptr_t es = codes ? 1 : h->d.out_dtype == KLT_DT_F32 ? 4 : 2;
  if (!aligned(xq, 16) || ld_xq % 16 || !aligned(xs, 4) || !aligned(out, es) ||
      (codes && !aligned(out_s, 4)))
    return KLT_ERR_ALIGN;
  // 32-bit offsets of the scales: beyond, xq alone would be 256 GB
  if (static_cast<int64_t>(M) * h->KB > 0x7FFFFFFF) return KLT_ERR_UNSUPPORTED;
  if (ld_xq < h->d.K || (M > 1 && ld_out < width)) return KLT_ERR_INVALID_ARG;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return KLT_ERR_CUDA;
  if (dev != h->device) return KLT_ERR_INVALID_ARG;

  int tile, split;
  choose(h, M, &tile, &split);
  if (dbg && (dbg->force_tile || dbg->force_split)) {
    if (dbg->force_tile) {
      tile = dbg->force_tile;
      split = 1;
      if (tile != 16 && tile != 32 && tile != 64 && tile != 128 && tile != 256)
        return KLT_ERR_INVALID_ARG;
      if (act && tile == 128) return KLT_ERR_UNSUPPORTED;
    }
    if (dbg->force_split) split = dbg->force_split;
    if (split != 1 && split != 2 && split != 4 && split != 8) return KLT_ERR_INVALID_ARG;
    if (split > h->KB || (tile == 256 && split > 2)) return KLT_ERR_UNSUPPORTED;
    if (tile < 256 && (M + tile - 1) / tile > 65535) return KLT_ERR_UNSUPPORTED;
  }

  LinParams p = {};
  p.w = h->w;
  p.ws = h->ws;
  p.xs = xs;
  p.out = out;
  p.out_s = out_s;
  p.ld_out = ld_out;
  p.M = M;
  p.KB = h->KB;
  p.NB = h->NB;
  p.width = width;
  p.up = act ? h->NB / 2 : 0;
  p.out_dtype = h->d.out_dtype;
  p.out_wide = aligned(out, 16) && (static_cast<uint64_t>(ld_out) * es) % 16 == 0;
  p.stall = dbg ? dbg->stall_after_kblocks : 0;
  p.err = h->err;
  // SM cycles at about 2 GHz
  p.timeout = static_cast<long long>(dbg && dbg->timeout_ms > 0 ? dbg->timeout_ms : 1000) *
              2000000LL;
  CUtensorMap tok;
  if (!encode_bytes(&tok, xq, M, h->d.K, ld_xq, 128, tile == 256 ? 128 : tile,
                    CU_TENSOR_MAP_SWIZZLE_128B))
    return KLT_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (tile == 256) {
    // 32 rows x 128 bytes (64 of codes) are stored at a time, where the rows allow bulk copies
    CUtensorMap omap = {};
    if (p.out_wide &&
        !encode_bytes(&omap, out, M, width * es, M > 1 ? ld_out * es : (width * es + 15) / 16 * 16,
                      codes ? 64 : 128, 32,
                      codes ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B))
      return KLT_ERR_CUDA;
    e = launch_linear_wide(tok, h->wmap, omap, p, act, split, h->num_sms, s);
  } else {
    e = launch_linear_narrow(tok, p, tile, split, act, s);
  }
  if (e == cudaSuccess) return KLT_OK;
  cudaGetLastError();  // reported here, not to the caller's next call
  return KLT_ERR_CUDA;
}

int klt_linear_tile(const klt_linear* h, int32_t M) {
  if (!h || M < 0) return -KLT_ERR_INVALID_ARG;
  int tile, split;
  choose(h, M, &tile, &split);
  return tile + 1000 * split;
}

int klt_linear_status(klt_linear* h) {
  if (!h) return KLT_ERR_INVALID_ARG;
  int e = 0;
  if (cudaMemcpy(&e, h->err, 4, cudaMemcpyDeviceToHost) != cudaSuccess) return KLT_ERR_CUDA;
  return e & DEV_ERR_TIMEOUT ? KLT_ERR_DEVICE_TIMEOUT : KLT_OK;
}

int klt_linear_destroy(klt_linear* h) {
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
