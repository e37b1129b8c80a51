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

#include <type_traits>


#include "../../include/klt.h"

namespace klt {
namespace {

// ------------------------------------------------------------------ 128 columns of a row
// A half warp holds one group of 128 columns of a row, eight neighbouring ones per lane.
// Where the tensor's rows start on 16 bytes (8 for codes) a lane's eight are one or two vector
// accesses.  Else, and for the short group at a row's end, the half warp moves them element by
// element, neighbouring lanes neighbouring elements (whole sectors), through 512 bytes of shared
// memory.  Plain loads, not the read-only path: the launch may begin while the kernel that
// writes these tensors still runs, and h_out may be h.
struct Half {
  uint32_t mask;  // the lanes of this half warp
  int lane;       // 0 .. 15
  float* buf;     // 128 floats of its own
};
KLT_DEV Half half_warp(float* bufs) {
  const int h = threadIdx.x >> 4;
  return {0xFFFFu << (16 * (h & 1)), static_cast<int>(threadIdx.x & 15),
          bufs ? bufs + h * 128 : nullptr};
}

// This lane's eight values of columns c .. c + 127 (c < C) of the row at element `off`; those
// past C are 0.
KLT_DEV void load8(const Half& hw, const void* base, bool f32, int64_t off, int c, int C, bool wide,
                   float* v) {
  if (wide && c + 128 <= C) {
    off += c + hw.lane * 8;
    if (f32) {
      const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(base) + off);
      const float4 a = p[0], b = p[1];
      v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
      v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    } else {
      const uint4 a =
          *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(base) + off);
      const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
      }
    }
    return;
  }
  if (f32) {
    const float* p = static_cast<const float*>(base) + off + c;
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = c + i * 16 + hw.lane < C ? p[i * 16 + hw.lane] : 0.f;
  } else {
    const __nv_bfloat16* p = static_cast<const __nv_bfloat16*>(base) + off + c;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      v[i] = c + i * 16 + hw.lane < C ? __bfloat162float(p[i * 16 + hw.lane]) : 0.f;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) hw.buf[i * 16 + hw.lane] = v[i];
  __syncwarp(hw.mask);
  const float4 a = reinterpret_cast<const float4*>(hw.buf)[hw.lane * 2];
  const float4 b = reinterpret_cast<const float4*>(hw.buf)[hw.lane * 2 + 1];
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
  v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  __syncwarp(hw.mask);
}
KLT_DEV void store_codes(const Half& hw, uint8_t* q, int64_t off, int c, int C, bool wide,
                         uint2 codes) {
  if (wide && c + 128 <= C) {
    *reinterpret_cast<uint2*>(q + off + c + hw.lane * 8) = codes;
    return;
  }
  reinterpret_cast<uint2*>(hw.buf)[hw.lane] = codes;
  __syncwarp(hw.mask);
  const uint8_t* b = reinterpret_cast<const uint8_t*>(hw.buf);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int e = i * 16 + hw.lane;
    if (c + e < C) q[off + c + e] = b[e];
  }
  __syncwarp(hw.mask);
}

// The largest magnitude of a group, NaN if it holds one.
KLT_DEV float group_amax(const Half& hw, const float* v) {
  float m = max_nan(max_nan(v[0], v[1], v[2]), max_nan(v[3], v[4], v[5]), max_nan(v[6], v[7]));
#pragma unroll
  for (int o = 8; o; o >>= 1) m = max_nan(m, __shfl_xor_sync(hw.mask, m, o));
  return m;
}
// Codes of four or eight values of a group with scale s.
KLT_DEV uint32_t codes4(const float* v, float s) {
  float t[4];
  const float k = rescale(s), inv = __frcp_rn(s);
#pragma unroll
  for (int i = 0; i < 4; ++i) t[i] = v[i];
  if (k != 1.0f) {
#pragma unroll
    for (int i = 0; i < 4; ++i) t[i] *= k;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) t[i] = quot_group(t[i], s, inv);
  return f32x2_to_e4m3x2(t[0], t[1]) | (f32x2_to_e4m3x2(t[2], t[3]) << 16);
}
KLT_DEV uint2 codes8(const float* v, float s) {
  return make_uint2(codes4(v, s), codes4(v + 4, s));
}

// Eight neighbouring values as they lie in memory, of a tensor whose rows are vectors: the
// loads of a whole row are issued before the first value is unpacked.
template <bool F32>
struct Raw8 {
  uint4 w[F32 ? 2 : 1];
  KLT_DEV void load(const void* base, int64_t off) {
    const uint4* p = reinterpret_cast<const uint4*>(static_cast<const char*>(base) +
                                                    off * (F32 ? 4 : 2));
    w[0] = p[0];
    if (F32) w[F32 ? 1 : 0] = p[1];
  }
  KLT_DEV void get(float* v) const {
    if (F32) {
      const uint32_t t[8] = {w[0].x, w[0].y, w[0].z, w[0].w,
                             w[F32].x, w[F32].y, w[F32].z, w[F32].w};
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(t[i]);
    } else {
      const uint32_t t[4] = {w[0].x, w[0].y, w[0].z, w[0].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(t[i] << 16);
        v[2 * i + 1] = __uint_as_float(t[i] & 0xFFFF0000u);
      }
    }
  }
};
template <bool F32>
KLT_DEV void put8(void* base, int64_t off, const float* v) {
  uint4* p = reinterpret_cast<uint4*>(static_cast<char*>(base) + off * (F32 ? 4 : 2));
  uint32_t t[8];
#pragma unroll
  for (int i = 0; i < (F32 ? 8 : 4); ++i) {
    if (F32) {
      t[i] = __float_as_uint(v[i]);
    } else {
      const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      t[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
  }
  p[0] = make_uint4(t[0], t[1], t[2], t[3]);
  if (F32) p[1] = make_uint4(t[4], t[5], t[6], t[7]);
}

// ------------------------------------------------------------------ sixteen values per lane
// The kernels for many rows give a lane 16 neighbouring values, eight lanes a group of 128, and
// compute on pairs: what a group costs beside its values (the scale, the shuffles) is shared
// by more of them, and an instruction does two.
typedef unsigned long long f32x2;

// t[0 .. N-1] = the N words from byte `bytes` (0 .. 15) of t[0 .. N+3] on.
template <int N>
KLT_DEV void shift_words(uint32_t* t, int bytes) {
  if (bytes & 8) {
#pragma unroll
    for (int i = 0; i < N + 2; ++i) t[i] = t[i + 2];
  }
  if (bytes & 4) {
#pragma unroll
    for (int i = 0; i < N + 1; ++i) t[i] = t[i + 1];
  }
#pragma unroll
  for (int i = 0; i < N; ++i) t[i] = __funnelshift_r(t[i], t[i + 1], (bytes & 3) * 8);
}

KLT_DEV int clamp16(int64_t x) { return x < 0 ? 0 : x > 16 ? 16 : static_cast<int>(x); }
// Bytes [first, last) of the aligned vector at v, of elements of two bytes or more; the others
// are 0, and not read.  A front or a back part is read in pieces of 8, 4 and 2 bytes.
KLT_DEV uint4 load_part(const char* v, int first, int last) {
  uint4 q = make_uint4(0, 0, 0, 0);
  if (first >= last) return q;
  if (first == 0) {
    const uint32_t x = last & 4 ? *reinterpret_cast<const uint32_t*>(v + (last & 8)) : 0;
    const uint32_t y = last & 2 ? *reinterpret_cast<const uint16_t*>(v + (last & 12)) : 0;
    const uint32_t a = last & 4 ? x : y, b = last & 4 ? y : 0;
    if (last & 8) {
      const uint2 u = *reinterpret_cast<const uint2*>(v);
      q = make_uint4(u.x, u.y, a, b);
    } else {
      q.x = a, q.y = b;
    }
  } else if (last == 16) {
    const int n = 16 - first;
    const uint32_t x = n & 4 ? *reinterpret_cast<const uint32_t*>(v + 16 - (n & 12)) : 0;
    const uint32_t y = n & 2 ? *reinterpret_cast<const uint16_t*>(v + 16 - (n & 14)) << 16 : 0;
    const uint32_t b = n & 4 ? x : y, a = n & 4 ? y : 0;
    if (n & 8) {
      const uint2 u = *reinterpret_cast<const uint2*>(v + 8);
      q = make_uint4(a, b, u.x, u.y);
    } else {
      q.z = a, q.w = b;
    }
  } else {
    uint32_t t[4] = {0, 0, 0, 0};
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (2 * e >= first && 2 * e < last)
        t[e / 2] |= reinterpret_cast<const uint16_t*>(v)[e] << e % 2 * 16;
    q = make_uint4(t[0], t[1], t[2], t[3]);
  }
  return q;
}
// The same, written; elements of ES bytes.
template <int ES>
KLT_DEV void store_part(char* v, int first, int last, uint4 q) {
  if (first >= last) return;
  if (first == 0) {
    if (last & 8) {
      *reinterpret_cast<uint2*>(v) = make_uint2(q.x, q.y);
      q.x = q.z, q.y = q.w;
    }
    if (last & 4) {
      *reinterpret_cast<uint32_t*>(v + (last & 8)) = q.x;
      q.x = q.y;
    }
    if (ES <= 2 && last & 2) {
      *reinterpret_cast<uint16_t*>(v + (last & 12)) = static_cast<uint16_t>(q.x);
      q.x >>= 16;
    }
    if (ES == 1 && last & 1)
      *reinterpret_cast<uint8_t*>(v + (last & 14)) = static_cast<uint8_t>(q.x);
  } else if (last == 16) {
    const int n = 16 - first;
    if (n & 8) {
      *reinterpret_cast<uint2*>(v + 8) = make_uint2(q.z, q.w);
      q.z = q.x, q.w = q.y;
    }
    if (n & 4) {
      *reinterpret_cast<uint32_t*>(v + 16 - (n & 12)) = q.w;
      q.w = q.z;
    }
    if (ES <= 2 && n & 2) {
      *reinterpret_cast<uint16_t*>(v + 16 - (n & 14)) = static_cast<uint16_t>(q.w >> 16);
      q.w <<= 16;
    }
    if (ES == 1 && n & 1)
      *reinterpret_cast<uint8_t*>(v + 16 - n) = static_cast<uint8_t>(q.w >> 24);
  } else {
    const uint32_t t[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int e = 0; e < 16; ++e)
      if (e >= first && e < last)
        reinterpret_cast<uint8_t*>(v)[e] = static_cast<uint8_t>(t[e / 4] >> e % 4 * 8);
  }
}

template <bool F32>
struct Raw16 {
  uint4 w[F32 ? 4 : 2];
  // WIDE: the rows start on 32 bytes, and a lane's values are one (fp32: two) 32-byte accesses
  template <bool WIDE = false>
  KLT_DEV void load(const void* base, int64_t off) {
    const char* p = static_cast<const char*>(base) + off * (F32 ? 4 : 2);
#pragma unroll
    for (int i = 0; i < (F32 ? 4 : 2); i += 2) {
      if (WIDE) {
        asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(w[i].x), "=r"(w[i].y), "=r"(w[i].z), "=r"(w[i].w),
                       "=r"(w[i + 1].x), "=r"(w[i + 1].y), "=r"(w[i + 1].z), "=r"(w[i + 1].w)
                     : "l"(p + i * 16)
                     : "memory");
      } else {
        w[i] = reinterpret_cast<const uint4*>(p)[i];
        w[i + 1] = reinterpret_cast<const uint4*>(p)[i + 1];
      }
    }
  }
  KLT_DEV void clear() {
#pragma unroll
    for (int i = 0; i < (F32 ? 4 : 2); ++i) w[i] = make_uint4(0, 0, 0, 0);
  }
  // Columns c .. c + 15 of a row of C that starts on any element; those past C are 0.  From
  // the aligned vectors that hold them, of which only what lies inside the row is read.
  KLT_DEV void load_any(const void* row, int c, int C) {
    constexpr int N = F32 ? 16 : 8;  // words
    const char* lo = static_cast<const char*>(row);
    const char *hi = lo + static_cast<int64_t>(C) * (F32 ? 4 : 2), *at = lo + c * (F32 ? 4 : 2);
    const int r = static_cast<int>(reinterpret_cast<uintptr_t>(at) & 15);
    uint32_t t[N + 4];
#pragma unroll
    for (int i = 0; i < N / 4 + 1; ++i) {
      if (i < N / 4 || r) {
        const char* v = at - r + 16 * i;
        const uint4 q = v >= lo && v + 16 <= hi ? *reinterpret_cast<const uint4*>(v)
                                                : load_part(v, clamp16(lo - v), clamp16(hi - v));
        t[4 * i] = q.x, t[4 * i + 1] = q.y, t[4 * i + 2] = q.z, t[4 * i + 3] = q.w;
      }
    }
    if (r) shift_words<N>(t, r);
#pragma unroll
    for (int i = 0; i < N / 4; ++i)
      w[i] = make_uint4(t[4 * i], t[4 * i + 1], t[4 * i + 2], t[4 * i + 3]);
  }
  KLT_DEV f32x2 get(int i) const {  // values 2i and 2i + 1
    if (F32) {
      const uint4& q = w[i >> 1];
      return i & 1 ? pack2(__uint_as_float(q.z), __uint_as_float(q.w))
                   : pack2(__uint_as_float(q.x), __uint_as_float(q.y));
    }
    const uint4& q = w[i >> 2];
    const uint32_t t = (i & 3) == 0 ? q.x : (i & 3) == 1 ? q.y : (i & 3) == 2 ? q.z : q.w;
    return pack2(__uint_as_float(t << 16), __uint_as_float(t & 0xFFFF0000u));
  }
};
// Columns of a row of C that starts on any element, in two steps: load() issues the loads of the
// aligned vectors that hold them; settle(), once all of a row's are in flight, shifts the values
// into place and makes those past C 0 (load_any does both at once: 4000 x 2901 44.4 us, so 41.5).
// A vector may hold bytes of a neighbouring row, but none outside the tensor's span lo .. hi: of
// its first and last only what is in there is read.
template <bool F32>
struct Any16 : Raw16<F32> {
  static constexpr int ES = F32 ? 4 : 2, N = 4 * ES;  // words
  uint32_t t[N + 4];
  int r;
  KLT_DEV void load(const char* lo, const char* hi, int64_t off, int c, int C) {
    const char* at = lo + (off + c) * ES;
    r = static_cast<int>(reinterpret_cast<uintptr_t>(at) & 15);
#pragma unroll
    for (int i = 0; i < N / 4 + 1; ++i) {
      const char* v = at - r + 16 * i;
      uint4 q = make_uint4(0, 0, 0, 0);
      if (16 * i - r < (C - c) * ES && (i < N / 4 || r)) {
        if (v >= lo && v + 16 <= hi)
          q = *reinterpret_cast<const uint4*>(v);
        else
          q = load_part(v, clamp16(lo - v), clamp16(hi - v));
      }
      t[4 * i] = q.x, t[4 * i + 1] = q.y, t[4 * i + 2] = q.z, t[4 * i + 3] = q.w;
    }
  }
  KLT_DEV void settle(int c, int C) {
    if (r) shift_words<N>(t, r);
    if (c + 16 > C) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        if (F32)
          t[i] = c + i < C ? t[i] : 0;
        else
          t[i] = c + 2 * i + 1 < C ? t[i] : c + 2 * i < C ? t[i] & 0xFFFFu : 0;
      }
    }
#pragma unroll
    for (int i = 0; i < N / 4; ++i)
      this->w[i] = make_uint4(t[4 * i], t[4 * i + 1], t[4 * i + 2], t[4 * i + 3]);
  }
};
// The end of `rows` rows of C columns.
template <bool F32>
KLT_DEV const char* span_end(const void* base, int64_t rows, int64_t ld, int C) {
  return static_cast<const char*>(base) + ((rows - 1) * ld + C) * (F32 ? 4 : 2);
}
template <bool F32>
KLT_DEV void put16(void* base, int64_t off, const f32x2* v) {  // rows on 32 bytes
  char* p = static_cast<char*>(base) + off * (F32 ? 4 : 2);
#pragma unroll
  for (int i = 0; i < (F32 ? 2 : 1); ++i) {
    uint32_t t[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float lo, hi;
      if (F32) {
        unpack2(v[4 * i + j / 2], lo, hi);
        t[j] = __float_as_uint(j & 1 ? hi : lo);
      } else {
        unpack2(v[j], lo, hi);
        const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
        t[j] = *reinterpret_cast<const uint32_t*>(&b);
      }
    }
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p + i * 32),
                 "r"(t[0]), "r"(t[1]), "r"(t[2]), "r"(t[3]), "r"(t[4]), "r"(t[5]), "r"(t[6]),
                 "r"(t[7])
                 : "memory");
  }
}
// Columns of a row of C that starts on any element: the whole warp's, NW words (16 elements of
// ES bytes) per lane from column c on; those past C are not written.  Each lane writes the vectors
// that end inside its own words, and takes their fronts from its neighbour; the warp's first and
// last vectors and the row's last are written in part.
template <int NW, int ES>
KLT_DEV void store_any(void* row, int c, int C, const uint32_t* w) {
  const int lane = threadIdx.x & 31;
  char* at = static_cast<char*>(row) + static_cast<int64_t>(c) * ES;
  const int r = static_cast<int>(reinterpret_cast<uintptr_t>(at) & 15);
  // of the vector at `at - r`: the bytes from the warp's first on, to the row's end
  const int first = lane == 0 ? r : 0, end = (C - c) * ES + r;
  char* v = at - r;
  uint32_t t[NW + 4];
#pragma unroll
  for (int i = 0; i < NW; ++i) t[i] = w[i];
  if (r) {
#pragma unroll
    for (int i = 0; i < 4; ++i) t[i] = __shfl_up_sync(0xFFFFFFFFu, w[NW - 4 + i], 1);
#pragma unroll
    for (int i = 0; i < NW; ++i) t[4 + i] = w[i];
    shift_words<NW>(t, 16 - r);
  }
#pragma unroll
  for (int k = 0; k < NW / 4; ++k) {
    const uint4 q = make_uint4(t[4 * k], t[4 * k + 1], t[4 * k + 2], t[4 * k + 3]);
    if ((k > 0 || first == 0) && end >= 16 * k + 16)
      *reinterpret_cast<uint4*>(v + 16 * k) = q;
    else
      store_part<ES>(v + 16 * k, k ? 0 : first, clamp16(end - 16 * k), q);
  }
  if (r && lane == 31) {
    uint32_t z[8] = {w[NW - 4], w[NW - 3], w[NW - 2], w[NW - 1], 0, 0, 0, 0};
    shift_words<4>(z, 16 - r);
    const int last = end - NW * 4;
    store_part<ES>(v + NW * 4, 0, last < r ? last : r, make_uint4(z[0], z[1], z[2], z[3]));
  }
}
template <bool F32>
KLT_DEV void put16_any(void* row, int c, int C, const f32x2* v) {
  uint32_t t[F32 ? 16 : 8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    float lo, hi;
    unpack2(v[j], lo, hi);
    if (F32) {
      t[F32 ? 2 * j : 0] = __float_as_uint(lo);
      t[F32 ? 2 * j + 1 : 0] = __float_as_uint(hi);
    } else {
      const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
      t[j] = *reinterpret_cast<const uint32_t*>(&b);
    }
  }
  store_any<F32 ? 16 : 8, F32 ? 4 : 2>(row, c, C, t);
}
template <bool F32>
KLT_DEV void* byte_offset(const void* p, int64_t elements) {
  return const_cast<char*>(static_cast<const char*>(p)) + elements * (F32 ? 4 : 2);
}
template <bool ANY, bool F32 = false, bool WIDE = false>
KLT_DEV void load16(Raw16<F32>& v, const void* base, int64_t off, int c, int C) {
  if (ANY)
    v.load_any(byte_offset<F32>(base, off), c, C);
  else
    v.template load<WIDE>(base, off + c);
}
// Sixteen codes of a row of C that starts on any byte, from column c on, by this lane alone.
KLT_DEV void store_codes16(uint8_t* row, int c, int C, uint4 codes) {
  uint8_t* at = row + c;
  const int r = static_cast<int>(reinterpret_cast<uintptr_t>(at) & 15);
  char* v = reinterpret_cast<char*>(at - r);
  if (r == 0) {
    if (c + 16 <= C)
      *reinterpret_cast<uint4*>(v) = codes;
    else
      store_part<1>(v, 0, clamp16(C - c), codes);
  } else {
    uint32_t t[12] = {0, 0, 0, 0, codes.x, codes.y, codes.z, codes.w, 0, 0, 0, 0};
    shift_words<8>(t, 16 - r);
    store_part<1>(v, r, clamp16(C - c + r), make_uint4(t[0], t[1], t[2], t[3]));
    store_part<1>(v + 16, 0, min(clamp16(C - c + r - 16), r), make_uint4(t[4], t[5], t[6], t[7]));
  }
}
// The largest magnitude of the group that this lane's eight lanes hold, NaN if it holds one.
KLT_DEV float group_amax16(const f32x2* v) {
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float lo, hi;
    unpack2(v[i], lo, hi);
    m = max_nan(m, lo, hi);
  }
#pragma unroll
  for (int o = 4; o; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
  return m;
}
KLT_DEV uint4 codes16(const f32x2* v, float s) {
  f32x2 t[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) t[i] = v[i];
  const float k = rescale(s), ninv = -__frcp_rn(s);
  if (k != 1.0f) {
#pragma unroll
    for (int i = 0; i < 8; ++i) t[i] = mul2(t[i], pack2(k, k));
  }
  const f32x2 s2 = pack2(s, s), ninv2 = pack2(ninv, ninv);
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float a, b, e, f;
    unpack2(neg_quot_group2(t[2 * i], s2, ninv2), a, b);
    unpack2(neg_quot_group2(t[2 * i + 1], s2, ninv2), e, f);
    c[i] = (f32x2_to_e4m3x2(a, b) | (f32x2_to_e4m3x2(e, f) << 16)) ^ 0x80808080u;
  }
  return make_uint4(c[0], c[1], c[2], c[3]);
}

// ------------------------------------------------------------------ the quantiser
struct QuantParams {
  const void* x;
  uint8_t* q;
  float* s;
  int64_t ld_x, ld_q;
  uint32_t items;  // rows x groups, below 2^31
  uint32_t magic;  // row of item i = (i * magic) >> shift
  int shift, K, G;
  bool f32, wide_x, wide_q;
};

KLT_DEV void quant_item(const QuantParams& p, uint32_t it, uint32_t& row, int& c) {
  row = static_cast<uint32_t>((static_cast<uint64_t>(it) * p.magic) >> p.shift);
  c = static_cast<int>(it - row * p.G) * 128;
}
KLT_DEV void quant_store(const Half& hw, const QuantParams& p, uint32_t it, uint32_t row, int c,
                         const float* v) {
  const float s = group_scale(group_amax(hw, v));
  store_codes(hw, p.q, row * p.ld_q, c, p.K, p.wide_q, codes8(v, s));
  if (hw.lane == 0) p.s[it] = s;
}
// Few groups, any strides and widths: one group of 128 columns per half warp (16 x 3584 1.4 us in
// a captured graph, the hand-off between launches).
__global__ void __launch_bounds__(256) quant_kernel(QuantParams p) {
  __shared__ float bufs[16 * 128];
  pdl_trigger();
  pdl_wait();
  const Half hw = half_warp(bufs);
  const uint32_t it = blockIdx.x * 16u + (threadIdx.x >> 4);
  if (it >= p.items) return;
  uint32_t row;
  int c;
  float v[8];
  quant_item(p, it, row, c);
  load8(hw, p.x, p.f32, row * p.ld_x, c, p.K, p.wide_x, v);
  quant_store(hw, p, it, row, c, v);
}
// Eight lanes per group, U groups each, their loads in flight together.  Vectors throughout (K a
// multiple of 128, aligned rows: 8192 x 7168 27.3 us, 6.5 TB/s), or (ANY) any strides and widths
// (8000 x 5003 24.3 us: instructions, 80 % issue, for the shifts of both sides).
template <int U, bool F32, bool ANY>
__global__ void __launch_bounds__(256) quant_vec_kernel(QuantParams p) {
  pdl_trigger();
  const uint32_t base = blockIdx.x * (32u * U) + (threadIdx.x >> 3);
  const int lane = threadIdx.x & 7;
  Raw16<F32> raw[U];
  uint32_t row[U];
  int c[U];
#pragma unroll
  for (int u = 0; u < U; ++u) quant_item(p, min(base + 32 * u, p.items - 1), row[u], c[u]);
  pdl_wait();
#pragma unroll
  for (int u = 0; u < U; ++u)
    load16<ANY>(raw[u], p.x, row[u] * p.ld_x, c[u] + lane * 16, p.K);
#pragma unroll
  for (int u = 0; u < U; ++u) {
    f32x2 v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = raw[u].get(i);
    const float s = group_scale(group_amax16(v));
    const uint4 codes = codes16(v, s);
    if (base + 32 * u < p.items) {
      uint8_t* q = p.q + row[u] * p.ld_q;
      if (ANY)
        store_codes16(q, c[u] + lane * 16, p.K, codes);
      else
        *reinterpret_cast<uint4*>(q + c[u] + lane * 16) = codes;
      if (lane == 0) p.s[base + 32 * u] = s;
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
  float eps, inv_h, res_scale, branch_scale;
  bool h_f32, y_f32, gate_f32, sigmoid;
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
// 1 / sqrt(sum / H + eps) by the fast reciprocal square root (2 ulp, the same for a whole row).
KLT_DEV float rms_inverse(float sum, float inv_h, float eps) {
  return rsqrtf(fmaf(sum, inv_h, eps));
}
KLT_DEV float gate_value(float g, bool sigmoid) { return sigmoid ? klt::sigmoid(g) : g; }
KLT_DEV float load1(const void* p, bool f32, int64_t i) {
  return f32 ? static_cast<const float*>(p)[i]
             : __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
}

// An element as it lies in memory, 0 where c >= end: without a branch, so that the loads of a
// row are in flight together (where each tensor's loads and conversions stood in branches on its
// type, a row waited for every tensor in turn: 16 x 1016 5.6 us).
template <bool F32>
KLT_DEV uint32_t load_raw(const char* at, int c, int end) {
  uint32_t r;
  if (F32)
    asm volatile(
        "{\n .reg .pred p;\n setp.lt.s32 p, %2, %3;\n mov.b32 %0, 0;\n"
        " @p ld.global.b32 %0, [%1];\n}"
        : "=r"(r)
        : "l"(at), "r"(c), "r"(end)
        : "memory");
  else
    asm volatile(
        "{\n .reg .pred p;\n setp.lt.s32 p, %2, %3;\n mov.b32 %0, 0;\n"
        " @p ld.global.u16 %0, [%1];\n}"
        : "=r"(r)
        : "l"(at), "r"(c), "r"(end)
        : "memory");
  return r;
}
// A row of a tensor.  TYPE: 0 bf16, 1 fp32, 2 either.
template <int TYPE>
struct Row {
  const char* at;
  int end;  // columns to read
  bool f32;
  KLT_DEV Row(const void* base, bool f, int64_t off, int n)
      : at(static_cast<const char*>(base)), end(base ? n : 0), f32(TYPE == 2 ? f : TYPE == 1) {
    at += off * (f32 ? 4 : 2);
  }
  // column c, the i-th element from the row's start
  KLT_DEV uint32_t raw(int c, int64_t i) const {
    if (TYPE == 0) return load_raw<false>(at + i * 2, c, end);
    if (TYPE == 1) return load_raw<true>(at + i * 4, c, end);
    return load_raw<false>(at + i * 2, c, f32 ? 0 : end) |
           load_raw<true>(at + i * 4, c, f32 ? end : 0);
  }
  KLT_DEV float value(uint32_t r) const { return __uint_as_float(f32 ? r : r << 16); }
};
KLT_DEV void store1(void* p, bool f32, int64_t i, float v) {
  if (f32)
    static_cast<float*>(p)[i] = v;
  else
    static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16(v);
}

// Rows of any strides and widths, few of them: one block per row, VPT groups of 128 columns per
// warp, whose lanes hold every 32nd column of a group, so that every access is one element per
// lane and needs no alignment.  TYPE of the residual stream; 2: of y and of a gate across
// channels too, with any stride.  The row's scalars (1/rms and the scales) multiply last: y
// gamma gate is exact up to its final rounding for bf16 tensors, and h' is one multiply-add of
// it.  16 x 2901 in 3.1 us, the latency of one block.
template <int VPT, int TYPE>
__global__ void __launch_bounds__(1024) norm_kernel(NormParams p) {
  constexpr int OTHER = TYPE == 2 ? 2 : 0;
  __shared__ float part[2][32];
  const int64_t row = blockIdx.x;
  const int lane = threadIdx.x & 31;
  const int c0 = static_cast<int>(threadIdx.x >> 5) * 128 + lane;
  const int step = static_cast<int>(blockDim.x) * 4;
  const bool columns = p.gate && p.gate_col != 0;
  const Row<OTHER> yr(p.y, p.y_f32, row * p.ld_y, p.H);
  const Row<TYPE> hr(p.h, p.h_f32, row * p.ld_h, p.H);
  const Row<OTHER> gr(p.gate, p.gate_f32, row * p.gate_row, columns ? p.H : 0);
  const Row<0> post(p.gamma_post, false, 0, p.H), pre(p.gamma_pre, false, 0, p.H);
  uint32_t ur[VPT][4], xr[VPT][4], gate[VPT][4], gpost[VPT][4], gpre[VPT][4];
  pdl_trigger();
  pdl_wait();
#pragma unroll
  for (int i = 0; i < VPT; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int c = c0 + i * step + 32 * j;
      ur[i][j] = yr.raw(c, c);
      xr[i][j] = hr.raw(c, c);
      gpost[i][j] = post.raw(c, c);
      gate[i][j] = gr.raw(c, TYPE == 2 ? c * p.gate_col : c);
      gpre[i][j] = pre.raw(c, c);
    }
  float scale = p.branch_scale;
  if (p.gate && !columns)
    scale *= gate_value(load1(p.gate, p.gate_f32, row * p.gate_row), p.sigmoid);
  if (p.gamma_post) {
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) ss = fmaf(yr.value(ur[i][j]), yr.value(ur[i][j]), ss);
    scale *= rms_inverse(block_sum(ss, part[0]), p.inv_h, p.eps);
  }
  float h[VPT][4], ss = 0.f;
#pragma unroll
  for (int i = 0; i < VPT; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int c = c0 + i * step + 32 * j;
      float u = yr.value(ur[i][j]), v = p.res_scale * hr.value(xr[i][j]);
      if (p.gamma_post) u *= post.value(gpost[i][j]);
      if (columns) u *= gate_value(gr.value(gate[i][j]), p.sigmoid);
      if (p.y) v = fmaf(scale, u, v);
      v = c < p.H ? v : 0.f;  // columns past H stay 0 whatever the scales are
      h[i][j] = v;
      ss = fmaf(v, v, ss);
      if (p.h_out && c < p.H) store1(p.h_out, p.h_f32, row * p.ld_h_out + c, v);
    }
  if (!p.n && !p.q) return;
  const float r = p.gamma_pre ? rms_inverse(block_sum(ss, part[1]), p.inv_h, p.eps) : 1.0f;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = c0 + i * step;
    if (c - lane >= p.H) break;
    if (p.gamma_pre) {
#pragma unroll
      for (int j = 0; j < 4; ++j) h[i][j] *= pre.value(gpre[i][j]);
    }
    if (p.q) {
      // n = t r with t = h' gamma: t against its own largest magnitude, r enters the scale alone
      float m = max_nan(max_nan(h[i][0], h[i][1], h[i][2]), h[i][3]);
#pragma unroll
      for (int o = 16; o; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
      const float d = over_448(m);
      float s = d * r;
      uint32_t codes = codes4(h[i], d == 0.f ? 1.0f : d);
      if (s == 0.f) s = 1.0f, codes = 0;  // n is 0 throughout, or rounds to it
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (c + 32 * j < p.H)
          p.q[row * p.ld_q + c + 32 * j] = static_cast<uint8_t>(codes >> 8 * j);
      if (lane == 0) p.s[row * p.G + c / 128] = s;
    }
    if (p.n) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (c + 32 * j < p.H) store1(p.n, false, row * p.ld_n + c + 32 * j, h[i][j] * r);
    }
  }
}

// The same for rows that are vectors throughout (H a multiple of 128, aligned), of any types: the
// row's loads are in flight together and stay packed until used.  Few rows: 1 x 7168 2.6 us, 16 x
// 7168 of fp32 to codes 3.8 us, the latency of one block and the hand-off between launches; many:
// those of fp32 y or gate (8192 x 7168 of fp32 y to bf16 86 us, 6.8 TB/s; norm_kernel 258).
template <int VPT, bool HF32, bool YF32, bool GF32>
__global__ void __launch_bounds__(VPT == 1 ? 1024 : 512) norm_vec_kernel(NormParams p) {
  __shared__ float part[2][32];
  const Half hw = half_warp(nullptr);
  const int64_t row = blockIdx.x;
  const int c0 = static_cast<int>(threadIdx.x) * 8, step = static_cast<int>(blockDim.x) * 8;
  Raw8<HF32> hr[VPT];
  Raw8<YF32> yr[VPT];
  Raw8<false> g1[VPT], g2[VPT];
  Raw8<GF32> gt[VPT];
  pdl_trigger();
  pdl_wait();
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = c0 + i * step;
    hr[i].w[0] = yr[i].w[0] = make_uint4(0, 0, 0, 0);
    if (HF32) hr[i].w[HF32] = make_uint4(0, 0, 0, 0);
    if (YF32) yr[i].w[YF32] = make_uint4(0, 0, 0, 0);
    if (c < p.H) {
      if (p.y) yr[i].load(p.y, row * p.ld_y + c);
      hr[i].load(p.h, row * p.ld_h + c);
      if (VPT == 1) {  // a short row's weights too
        if (p.gamma_post) g1[i].load(p.gamma_post, c);
        if (p.gamma_pre) g2[i].load(p.gamma_pre, c);
        if (p.gate && p.gate_col != 0) gt[i].load(p.gate, row * p.gate_row + c);
      }
    }
  }
  const float token =
      p.gate && p.gate_col == 0 ? load1(p.gate, p.gate_f32, row * p.gate_row) : 0.f;
  float scale = p.branch_scale;
  if (p.gamma_post) {
    float ss = 0.f, v[8];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      yr[i].get(v);
#pragma unroll
      for (int j = 0; j < 8; ++j) ss = fmaf(v[j], v[j], ss);
    }
    scale *= rms_inverse(block_sum(ss, part[0]), p.inv_h, p.eps);
  }
  if (p.gate && p.gate_col == 0)
    scale *= gate_value(token, p.sigmoid);
  float h[VPT][8], ss = 0.f;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = c0 + i * step;
    float u[8], g[8];
    hr[i].get(h[i]);
    if (c < p.H) {
      if (p.y) {
        yr[i].get(u);
        if (p.gamma_post) {
          if (VPT > 1) g1[i].load(p.gamma_post, c);
          g1[i].get(g);
#pragma unroll
          for (int j = 0; j < 8; ++j) u[j] *= g[j];
        }
        if (p.gate && p.gate_col != 0) {
          if (VPT > 1) gt[i].load(p.gate, row * p.gate_row + c);
          gt[i].get(g);
          if (p.sigmoid) {
#pragma unroll
            for (int j = 0; j < 8; ++j) g[j] = gate_value(g[j], true);
          }
#pragma unroll
          for (int j = 0; j < 8; ++j) u[j] *= g[j];
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) h[i][j] = fmaf(scale, u[j], p.res_scale * h[i][j]);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) h[i][j] *= p.res_scale;
      }
      if (p.h_out) put8<HF32>(p.h_out, row * p.ld_h_out + c, h[i]);
#pragma unroll
      for (int j = 0; j < 8; ++j) ss = fmaf(h[i][j], h[i][j], ss);
    }
  }
  if (!p.n && !p.q) return;
  const float r =
      p.gamma_pre ? rms_inverse(block_sum(ss, part[1]), p.inv_h, p.eps) : 1.0f;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = c0 + i * step;
    if (c < p.H) {
      if (p.gamma_pre) {
        float g[8];
        if (VPT > 1) g2[i].load(p.gamma_pre, c);
        g2[i].get(g);
#pragma unroll
        for (int j = 0; j < 8; ++j) h[i][j] *= g[j];
      }
      if (p.q) {  // as norm_kernel
        const float d = over_448(group_amax(hw, h[i]));
        float s = d * r;
        uint2 codes = codes8(h[i], d == 0.f ? 1.0f : d);
        if (s == 0.f) s = 1.0f, codes = make_uint2(0, 0);
        *reinterpret_cast<uint2*>(p.q + row * p.ld_q + c) = codes;
        if (hw.lane == 0) p.s[row * p.G + c / 128] = s;
      }
      if (p.n) {
#pragma unroll
        for (int j = 0; j < 8; ++j) h[i][j] *= r;
        put8<false>(p.n, row * p.ld_n + c, h[i]);
      }
    }
  }
}

// Many rows: one block per row, VPT times 16 columns per thread, pairs throughout.  Of vectors
// that start on 32 bytes (8192 x 7168 to bf16 72 us, 6.5 TB/s; to codes with a gate 86, 4.8 TB/s,
// with a sigmoid gate 101: occupancy, as registers limit an SM to three rows, 52 % issue), or (ANY)
// of any start and length (1021 x 2901 11.2 us).
template <int VPT, bool HF32, bool ANY>
KLT_DEV void norm_many_row(const NormParams& p) {
  __shared__ float part[2][32];
  const int64_t row = blockIdx.x;
  const int c0 = static_cast<int>(threadIdx.x) * 16, step = static_cast<int>(blockDim.x) * 16;
  typename std::conditional<ANY, Any16<HF32>, Raw16<HF32>>::type hr[VPT];
  typename std::conditional<ANY, Any16<false>, Raw16<false>>::type yr[VPT];
  // One set of columns per thread: the weights' loads go out with the row's (8192 x 2048 25.1 us,
  // so 23.1; with two sets their registers cost more than that saves: 8192 x 7168 88 and 107 us).
  // Else the gate's go with the weight's where there are registers (88 and 86.4; fp32 rows 117
  // and 135).
  constexpr bool EARLY = VPT == 1 && !ANY, TOGETHER = !HF32 && !ANY;
  Raw16<false> post, other, g;
  Raw16<false>& gate = EARLY || TOGETHER ? other : post;
  const bool columns = p.gate && p.gate_col != 0;
  pdl_trigger();
  pdl_wait();
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = c0 + i * step;
    hr[i].clear();
    yr[i].clear();
    if (c < p.H) {
      if constexpr (ANY) {
        if (p.y)
          yr[i].load(static_cast<const char*>(p.y), span_end<false>(p.y, gridDim.x, p.ld_y, p.H),
                     row * p.ld_y, c, p.H);
        hr[i].load(static_cast<const char*>(p.h), span_end<HF32>(p.h, gridDim.x, p.ld_h, p.H),
                   row * p.ld_h, c, p.H);
      } else {
        if (p.y) yr[i].template load<true>(p.y, row * p.ld_y + c);
        hr[i].template load<true>(p.h, row * p.ld_h + c);
      }
      if (EARLY) {
        if (p.gamma_post) load16<ANY>(post, p.gamma_post, 0, c, p.H);
        if (columns) load16<ANY>(gate, p.gate, row * p.gate_row, c, p.H);
      }
    }
  }
  if constexpr (ANY) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = c0 + i * step;
      if (c < p.H) {
        if (p.y) yr[i].settle(c, p.H);
        hr[i].settle(c, p.H);
      }
    }
  }
  float lo, hi, scale = p.branch_scale;
  if (p.gamma_post) {
    f32x2 ss = 0;
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const f32x2 v = yr[i].get(j);
        ss = fmaf2(v, v, ss);
      }
    unpack2(ss, lo, hi);
    scale *= rms_inverse(block_sum(lo + hi, part[0]), p.inv_h, p.eps);
  }
  if (p.gate && p.gate_col == 0)
    scale *= gate_value(load1(p.gate, p.gate_f32, row * p.gate_row), p.sigmoid);
  const f32x2 scale2 = pack2(scale, scale), res2 = pack2(p.res_scale, p.res_scale);
  f32x2 h[VPT][8], ss = 0;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = c0 + i * step;
#pragma unroll
    for (int j = 0; j < 8; ++j) h[i][j] = 0;
    if (c < p.H) {
#pragma unroll
      for (int j = 0; j < 8; ++j) h[i][j] = mul2(hr[i].get(j), res2);
      if (p.y) {
        f32x2 u[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) u[j] = yr[i].get(j);
        if (!EARLY) {
          if (p.gamma_post) load16<ANY>(post, p.gamma_post, 0, c, p.H);
          if (columns && TOGETHER) load16<ANY>(gate, p.gate, row * p.gate_row, c, p.H);
        }
        if (p.gamma_post) {
#pragma unroll
          for (int j = 0; j < 8; ++j) u[j] = mul2(u[j], post.get(j));
        }
        if (columns) {
          if (!EARLY && !TOGETHER) load16<ANY>(gate, p.gate, row * p.gate_row, c, p.H);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            f32x2 w = gate.get(j);
            if (p.sigmoid) {
              unpack2(w, lo, hi);
              w = pack2(gate_value(lo, true), gate_value(hi, true));
            }
            u[j] = mul2(u[j], w);
          }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) h[i][j] = fmaf2(scale2, u[j], h[i][j]);
      }
      if (ANY && c + 16 > p.H) {  // columns past H stay 0 whatever the scales are
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          unpack2(h[i][j], lo, hi);
          h[i][j] = pack2(c + 2 * j < p.H ? lo : 0.f, c + 2 * j + 1 < p.H ? hi : 0.f);
        }
      }
      if (!ANY && p.h_out) put16<HF32>(p.h_out, row * p.ld_h_out + c, h[i]);
#pragma unroll
      for (int j = 0; j < 8; ++j) ss = fmaf2(h[i][j], h[i][j], ss);
    }
    if (ANY && p.h_out)
      put16_any<HF32>(byte_offset<HF32>(p.h_out, row * p.ld_h_out), c, p.H, h[i]);
  }
  if (!p.n && !p.q) return;
  float r = 1.0f;
  if (p.gamma_pre) {
    unpack2(ss, lo, hi);
    r = rms_inverse(block_sum(lo + hi, part[1]), p.inv_h, p.eps);
  }
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = c0 + i * step;
    if (p.gamma_pre && c < p.H) {
      load16<ANY>(g, p.gamma_pre, 0, c, p.H);
#pragma unroll
      for (int j = 0; j < 8; ++j) h[i][j] = mul2(h[i][j], g.get(j));
    }
    if (p.q) {  // as norm_kernel
      const float d = over_448(group_amax16(h[i]));
      float s = d * r;
      uint4 codes = codes16(h[i], d == 0.f ? 1.0f : d);
      if (s == 0.f) s = 1.0f, codes = make_uint4(0, 0, 0, 0);
      if (ANY) {
        const uint32_t t[4] = {codes.x, codes.y, codes.z, codes.w};
        store_any<4, 1>(p.q + row * p.ld_q, c, p.H, t);
      } else if (c < p.H) {
        *reinterpret_cast<uint4*>(p.q + row * p.ld_q + c) = codes;
      }
      if (c < p.H && (threadIdx.x & 7) == 0) p.s[row * p.G + c / 128] = s;
    }
    if (p.n && (ANY || c < p.H)) {
#pragma unroll
      for (int j = 0; j < 8; ++j) h[i][j] = mul2(h[i][j], pack2(r, r));
      if (ANY)
        put16_any<false>(byte_offset<false>(p.n, row * p.ld_n), c, p.H, h[i]);
      else
        put16<false>(p.n, row * p.ld_n + c, h[i]);
    }
  }
}

template <int VPT, bool HF32, bool ANY>
__global__ void __launch_bounds__(512) norm_many_kernel(NormParams p) {
  norm_many_row<VPT, HF32, ANY>(p);
}
// Long bf16 rows: with one register more an SM takes two rows instead of three (8192 x 7168 to
// codes 112 us, so 86).
__global__ void __maxnreg__(80) norm_long_kernel(NormParams p) { norm_many_row<2, false, false>(p); }

template <typename Kernel, typename... Params>
cudaError_t launch_pdl(Kernel k, unsigned grid, unsigned block, cudaStream_t s,
                       const Params&... p) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k, p...);
}

template <int TYPE>
cudaError_t launch_row(unsigned grid, cudaStream_t st, const NormParams& p) {
  const int groups = p.G <= 32 ? 1 : p.G <= 64 ? 2 : 4;
  const unsigned lanes = (p.G + groups - 1) / groups * 32;
  return groups == 1   ? launch_pdl(norm_kernel<1, TYPE>, grid, lanes, st, p)
         : groups == 2 ? launch_pdl(norm_kernel<2, TYPE>, grid, lanes, st, p)
                       : launch_pdl(norm_kernel<4, TYPE>, grid, lanes, st, p);
}

template <bool HF32, bool YF32, bool GF32>
cudaError_t launch_vec(int vpt, unsigned grid, unsigned threads, cudaStream_t st,
                       const NormParams& p) {
  switch (vpt) {
    case 1: return launch_pdl(norm_vec_kernel<1, HF32, YF32, GF32>, grid, threads, st, p);
    case 2: return launch_pdl(norm_vec_kernel<2, HF32, YF32, GF32>, grid, threads, st, p);
    default: return launch_pdl(norm_vec_kernel<4, HF32, YF32, GF32>, grid, threads, st, p);
  }
}

template <bool HF32, bool ANY>
cudaError_t launch_many(bool twice, unsigned grid, unsigned lanes, cudaStream_t st,
                        const NormParams& p) {
  if (!twice) return launch_pdl(norm_many_kernel<1, HF32, ANY>, grid, lanes, st, p);
  if constexpr (!HF32 && !ANY)
    return launch_pdl(norm_long_kernel, grid, lanes, st, p);
  else
    return launch_pdl(norm_many_kernel<2, HF32, ANY>, grid, lanes, st, p);
}

int status_of(cudaError_t e) {
  if (e == cudaSuccess) return KLT_OK;
  cudaGetLastError();  // reported here, not to the caller's next call
  return KLT_ERR_CUDA;
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
  // offsets within a row are 32 bits
  if (!known(x_dtype) || K > (1 << 28)) return KLT_ERR_UNSUPPORTED;
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
  const int64_t items = static_cast<int64_t>(M) * p.G;
  if (items > 0x7FFFFF00) return KLT_ERR_UNSUPPORTED;
  p.items = static_cast<uint32_t>(items);
  // i / G for i < 2^31 by multiplication: magic = ceil(2^(31 + l) / G), l = ceil(log2 G)
  int l = 0;
  while ((1ll << l) < p.G) ++l;
  p.shift = 31 + l;
  p.magic = static_cast<uint32_t>(((1ull << p.shift) + p.G - 1) / p.G);
  p.f32 = x_dtype == KLT_DT_F32;
  p.wide_x = wide(x, ld_x, esize(x_dtype), 16);
  p.wide_q = wide(q, ld_q, 1, 8);
  // 16 values per lane once there are enough groups to fill the device: vectors throughout, two
  // groups in flight, from four groups per half warp on (8192 x 7168 27.6 us, one group per half
  // warp 38); other rows from 4096 groups on (8000 x 5003 24.8 and 47.1 us, 300 x 5003 3.1 and
  // 3.6, 1021 x 301 even; two groups in flight 29.4).  Else one group per half warp, spread over
  // more SMs.
  const bool vectors = K % 128 == 0 && p.wide_x && wide(q, ld_q, 1, 16);
  const bool many = items >= (vectors ? 4 * 16 * 152 * 4 : 4096);
  const int per = many ? vectors ? 64 : 32 : 16;
  const unsigned grid = static_cast<unsigned>((items + per - 1) / per);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (!many)
    e = launch_pdl(quant_kernel, grid, 256, st, p);
  else if (vectors)
    e = p.f32 ? launch_pdl(quant_vec_kernel<2, true, false>, grid, 256, st, p)
              : launch_pdl(quant_vec_kernel<2, false, false>, grid, 256, st, p);
  else
    e = p.f32 ? launch_pdl(quant_vec_kernel<1, true, true>, grid, 256, st, p)
              : launch_pdl(quant_vec_kernel<1, false, true>, grid, 256, st, p);
  return status_of(e);
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
  p.inv_h = 1.0f / static_cast<float>(H);
  p.res_scale = a->res_scale;
  p.branch_scale = a->branch_scale;
  p.h_f32 = a->h_dtype == KLT_DT_F32;
  p.y_f32 = a->y_dtype == KLT_DT_F32;
  p.gate_f32 = a->gate_dtype == KLT_DT_F32;
  p.sigmoid = a->gate_sigmoid != 0;
  // One group per half warp, the shortest path through a row (2000 x 1024 5.4 us, two groups 6.8);
  // of many long rows as many as leave 8 warps a block (8000 x 7168 four groups 107, two 128,
  // one 193; 4000 x 2944 two groups 27.9, one 31, four 29.9)
  int vpt = 1;
  while (vpt < 4 && (p.G > vpt * (vpt == 1 ? 64 : 32) || (M > 8 * 152 && p.G > vpt * 16)))
    vpt *= 2;
  const int threads = ((p.G + vpt - 1) / vpt * 16 + 31) / 32 * 32;
  const unsigned grid = static_cast<unsigned>(M);
  const bool vectors = H % 128 == 0 && wide(a->h, a->ld_h, he, 16) &&
                       (!a->y || wide(a->y, a->ld_y, ye, 16)) &&
                       (!a->gate || a->gate_col != 1 || wide(a->gate, a->gate_row, ge, 16)) &&
                       aligned(a->gamma_post, 16) && aligned(a->gamma_pre, 16) &&
                       (!a->h_out || wide(a->h_out, a->ld_h_out, he, 16)) &&
                       (!a->n || wide(a->n, a->ld_n, 2, 16)) &&
                       (!a->q || wide(a->q, a->ld_q, 1, 8));
  // stride of a gate across channels, 0 if there is none: neighbouring columns, or any
  const int64_t columns = a->gate ? a->gate_col : 0;
  // types and strides that only some of the kernels take
  const bool plain = (a->y && p.y_f32) || columns > 1 || (columns == 1 && p.gate_f32);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  // Enough values to fill the device (160 x 7168: 3.6 us, eight per thread 4.6; 400 x 2048: 3.3
  // and 2.9 us), in rows that start on 32 bytes: 16 per thread, and twice that for many long rows
  // of bf16 (8192 x 7168 to codes 86.8 and 96.6 us; 8192 x 2048 25.9 and 23.1, fp32 rows of 7168
  // 117 either way), but with a gate of their own (8192 x 7168 119 and 108).
  const bool many = M > 152 && static_cast<int64_t>(M) * H > 1 << 20 && vectors && !plain &&
                    wide(a->h, a->ld_h, he, 32) &&
                    (!a->y || wide(a->y, a->ld_y, ye, 32)) &&
                    (!a->h_out || wide(a->h_out, a->ld_h_out, he, 32)) &&
                    (!a->n || wide(a->n, a->ld_n, 2, 32)) && (!a->q || wide(a->q, a->ld_q, 1, 16));
  // Rows of any start and length: the same with 16 per thread from about a million values on
  // (1021 x 2901 11.2 us, norm_kernel 18.2; 1000 x 7001 31 and 38; 300 x 7001 8.2 and 9.8; but
  // 1000 x 1016 8.0 and 5.8, 16 x 2901 6.3 and 3.1); 32 per thread took 150 us for 4000 x 7001,
  // 16 per thread 89.
  const bool any = !vectors && !plain && static_cast<int64_t>(M) * H > 5 << 18;
  if (many) {
    const bool full = a->gate && a->gate_col != 0 && a->gate_row != 0;
    const bool twice = H > 8192 || (M > 8 * 152 && H > 4096 && !p.h_f32 && !full);
    const int per = twice ? 32 : 16;
    const unsigned lanes = ((H + per - 1) / per + 31) / 32 * 32;
    e = p.h_f32 ? launch_many<true, false>(twice, grid, lanes, st, p)
                : launch_many<false, false>(twice, grid, lanes, st, p);
  } else if (any) {
    const bool twice = H > 8192;
    const unsigned lanes = ((H + (twice ? 31 : 15)) / (twice ? 32 : 16) + 31) / 32 * 32;
    e = p.h_f32 ? launch_many<true, true>(twice, grid, lanes, st, p)
                : launch_many<false, true>(twice, grid, lanes, st, p);
  } else if (!vectors || columns > 1) {
    e = plain ? launch_row<2>(grid, st, p) : p.h_f32 ? launch_row<1>(grid, st, p)
                                                     : launch_row<0>(grid, st, p);
  } else {
    const bool yf = a->y && p.y_f32, gf = columns == 1 && p.gate_f32;
    auto vec = [&](auto hf32) {
      constexpr bool H32 = decltype(hf32)::value;
      if (yf && gf) return launch_vec<H32, true, true>(vpt, grid, threads, st, p);
      if (yf) return launch_vec<H32, true, false>(vpt, grid, threads, st, p);
      if (gf) return launch_vec<H32, false, true>(vpt, grid, threads, st, p);
      return launch_vec<H32, false, false>(vpt, grid, threads, st, p);
    };
    e = p.h_f32 ? vec(std::true_type()) : vec(std::false_type());
  }
  return status_of(e);
}
