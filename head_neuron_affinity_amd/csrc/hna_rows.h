// Device helpers of the row kernels (norms and 8-bit rows): 8-element loads and
// stores in fp32, sums and maxima over the lanes that hold one row, and the
// rounding of a row to 8-bit integers.
#pragma once

#include "hna_internal.h"

namespace hna {
namespace rows {

// ---- the elements of a row over its lanes ----
// NT lanes hold a row in chunks of 8 NT elements, 8 to a lane: in two halves of 4
// that follow each other, or (SPLIT) lie NT 4 elements apart.  SPLIT is for rows
// that are fp32 on one side: a load or store of 16 bytes a lane then covers whole
// lines, where 8 consecutive fp32 elements a lane would take every other 16 bytes.
template <int NT, bool SPLIT>
struct Lane {
  int lane;
  __device__ inline int at(int c, int h) const {
    return SPLIT ? c * NT * 8 + h * NT * 4 + lane * 4 : (c * NT + lane) * 8 + h * 4;
  }
};

typedef float f32x4v __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4v __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2v __attribute__((ext_vector_type(2)));
// NTEMP: past the caches (a stream that they could not hold)
template <bool NTEMP, typename V>
__device__ inline V load_v(const void* p) {
  const V* v = static_cast<const V*>(p);
  if constexpr (NTEMP) return __builtin_nontemporal_load(v);
  else return *v;
}
template <bool NTEMP, typename V>
__device__ inline void store_v(void* p, V x) {
  V* v = static_cast<V*>(p);
  if constexpr (NTEMP) __builtin_nontemporal_store(x, v);
  else *v = x;
}

// A lane's 8 elements of a chunk as they lie in memory; halves from C on are zeros
template <typename T, bool SPLIT>
struct Raw8;
template <bool SPLIT>
struct Raw8<__bf16, SPLIT> {
  u32x2v q[2];
  template <bool NTEMP, int NT>
  __device__ inline void load(const __bf16* row, Lane<NT, SPLIT> l, int c, int C, bool live) {
    q[0] = q[1] = u32x2v{0u, 0u};
    if constexpr (SPLIT) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if (live && l.at(c, h) < C) q[h] = load_v<NTEMP, u32x2v>(row + l.at(c, h));
    } else if (live && l.at(c, 0) < C) {
      const u32x4v v = load_v<NTEMP, u32x4v>(row + l.at(c, 0));
      q[0] = u32x2v{v.x, v.y};
      q[1] = u32x2v{v.z, v.w};
    }
  }
  __device__ inline void get(float (&v)[8]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t w = i & 1 ? q[i >> 1].y : q[i >> 1].x;
      v[2 * i] = __uint_as_float(w << 16);
      v[2 * i + 1] = __uint_as_float(w & 0xffff0000u);
    }
  }
};
template <bool SPLIT>
struct Raw8<float, SPLIT> {
  f32x4v q[2];
  template <bool NTEMP, int NT>
  __device__ inline void load(const float* row, Lane<NT, SPLIT> l, int c, int C, bool live) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      q[h] = f32x4v{0.f, 0.f, 0.f, 0.f};
      if (live && l.at(c, h) < C) q[h] = load_v<NTEMP, f32x4v>(row + l.at(c, h));
    }
  }
  __device__ inline void get(float (&v)[8]) const {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      v[4 * h] = q[h].x;
      v[4 * h + 1] = q[h].y;
      v[4 * h + 2] = q[h].z;
      v[4 * h + 3] = q[h].w;
    }
  }
};
template <bool NTEMP, int NT, bool SPLIT>
__device__ inline void store8(__bf16* row, Lane<NT, SPLIT> l, int c, int C, const float (&v)[8]) {
  const u32x2v a = {pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])}, b = {pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])};
  if constexpr (SPLIT) {
    if (l.at(c, 0) < C) store_v<NTEMP, u32x2v>(row + l.at(c, 0), a);
    if (l.at(c, 1) < C) store_v<NTEMP, u32x2v>(row + l.at(c, 1), b);
  } else {
    if (l.at(c, 0) < C) store_v<NTEMP, u32x4v>(row + l.at(c, 0), u32x4v{a.x, a.y, b.x, b.y});
  }
}
template <bool NTEMP, int NT, bool SPLIT>
__device__ inline void store8(float* row, Lane<NT, SPLIT> l, int c, int C, const float (&v)[8]) {
#pragma unroll
  for (int h = 0; h < 2; ++h)
    if (l.at(c, h) < C) store_v<NTEMP, f32x4v>(row + l.at(c, h), f32x4v{v[4 * h], v[4 * h + 1], v[4 * h + 2], v[4 * h + 3]});
}
// 8 floats of a gain row, 1 from C on
template <int NT, bool SPLIT>
__device__ inline void load_gain(const float* row, Lane<NT, SPLIT> l, int c, int C, float (&v)[8]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    f32x4v q = {1.f, 1.f, 1.f, 1.f};
    if (l.at(c, h) < C) q = *reinterpret_cast<const f32x4v*>(row + l.at(c, h));
    v[4 * h] = q.x;
    v[4 * h + 1] = q.y;
    v[4 * h + 2] = q.z;
    v[4 * h + 3] = q.w;
  }
}
// v as it will be read back from a tensor of type R
template <typename R>
__device__ inline float as_stored(float v) {
  if constexpr (sizeof(R) == 2) return __uint_as_float(pack_bf16x2(v, 0.f) << 16);
  return v;
}

// ---- one value per lane combined over the 64 lanes of a wave; every lane gets
// the same bits (each step combines the same two values in both lanes) ----
template <int CTRL>
__device__ inline uint32_t dpp(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xf, 0xf, true);
}
template <typename F>
__device__ inline uint32_t wave_all(uint32_t v, F f) {
  v = f(v, dpp<0xB1>(v));    // lane ^ 1
  v = f(v, dpp<0x4E>(v));    // lane ^ 2
  v = f(v, dpp<0x141>(v));   // the other four of eight
  v = f(v, dpp<0x140>(v));   // the other eight of sixteen
  const auto a = __builtin_amdgcn_permlane16_swap(v, v, false, false);
  v = f(a[0], a[1]);
  const auto b = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  return f(b[0], b[1]);
}
__device__ inline uint32_t add_bits(uint32_t a, uint32_t b) {
  return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
}
__device__ inline uint32_t max_bits(uint32_t a, uint32_t b) { return a > b ? a : b; }

// The same over the NT lanes that hold one row (whole waves), NT / 64 partials
// through LDS.  `box` holds 2 x (workgroup waves) words and `phase` alternates
// between its halves: a half is written again only after the barrier of the
// other half, which every wave reaches after its reads of this one, so one
// barrier per call is enough.  Every thread of the workgroup must call it.
template <int NT, int WG, typename F>
__device__ inline uint32_t row_all(uint32_t v, uint32_t* box, int& phase, F f) {
  v = wave_all(v, f);
  if constexpr (NT > 64) {
    uint32_t* b = box + phase * (WG / 64);
    phase ^= 1;
    const int w = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) b[w] = v;
    __syncthreads();
    const int w0 = w & ~(NT / 64 - 1);
    v = b[w0];
#pragma unroll
    for (int i = 1; i < NT / 64; ++i) v = f(v, b[w0 + i]);
  }
  return v;
}
template <int NT, int WG>
__device__ inline float row_sum(float v, uint32_t* box, int& phase) {
  return __uint_as_float(row_all<NT, WG>(__float_as_uint(v), box, phase, add_bits));
}
// Largest |v| of a row as bits: the order of the bits of |v| is that of |v|,
// with infinity and every NaN above the finite values
template <int NT, int WG>
__device__ inline uint32_t row_max_bits(uint32_t v, uint32_t* box, int& phase) {
  return row_all<NT, WG>(v, box, phase, max_bits);
}

// ---- a row as 8-bit integers ----
// q = the integer nearest to 127 v / top, top = max|v| of the row, ties to even,
// exactly: v * (127 / top) is within 2e-5 of the quotient (two roundings, at most
// 127), so its nearest integer is right unless it lies that close to a half;
// there the sign of 254 |v| - (2 k + 1) top decides, k the integer below.  With
// b + bl = (2 k + 1) top exactly (b rounded, bl the remainder), 254 |v| - b is
// a difference of close numbers of at most 32 bits and comes out exactly, so
// the sign of its difference with bl is exact too.
// `pre` is a power of two that keeps top within 2^-100 .. 2^100, so that
// neither 127 / top nor the products leave the range of fp32; 1 for nearly
// every row.
struct RowScale {
  float scale;   // what one step of q stands for: top / 127 (NaN for a row with a NaN or an infinity)
  float inv;     // 127 / (top pre), 0 where every q is 0
  float top;     // top pre
  float pre;
};
__device__ inline RowScale row_scale(uint32_t top_bits) {
  RowScale s;
  const float top = __uint_as_float(top_bits);
  const bool finite = top_bits < 0x7f800000u;
  s.pre = top < 0x1p-100f ? 0x1p100f : (top > 0x1p100f ? 0x1p-100f : 1.f);
  s.top = top * s.pre;
  s.scale = finite ? top / 127.f : __uint_as_float(0x7fc00000u);
  s.inv = finite && top > 0.f ? 127.f / s.top : 0.f;
  return s;
}
__device__ inline float quant_exact(float v, float t, const RowScale& s) {
  const float av = fabsf(v), k = floorf(fabsf(t)), odd = 2.f * k + 1.f;
  const float b = odd * s.top, bl = fmaf(odd, s.top, -b);
  const float d = fmaf(254.f, av, -b) - bl;
  const float q = k + ((d > 0.f || (d == 0.f && ((int)k & 1))) ? 1.f : 0.f);
  return copysignf(q, v);
}
// 8 elements to 8 bytes.  Adding 1.5 * 2^23 rounds to an integer, whose low
// byte is the sum's.
__device__ inline uint2 quant8(const float (&x)[8], const RowScale& s) {
  if (s.inv == 0.f) return make_uint2(0u, 0u);
  constexpr float kInt = 12582912.f;
  float v[8], r[8], off[8], worst = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = x[e];
  if (s.pre != 1.f) {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] *= s.pre;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    r[e] = fmaf(v[e], s.inv, kInt);
    off[e] = fabsf(fmaf(v[e], s.inv, kInt - r[e]));
    worst = fmaxf(worst, off[e]);
  }
  if (worst > 0.4999f) {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (off[e] > 0.4999f) r[e] = kInt + quant_exact(v[e], v[e] * s.inv, s);
  }
  uint32_t w[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t lo = __builtin_amdgcn_perm(__float_as_uint(r[4 * h + 1]), __float_as_uint(r[4 * h]), 0x0c0c0400u);
    const uint32_t hi = __builtin_amdgcn_perm(__float_as_uint(r[4 * h + 3]), __float_as_uint(r[4 * h + 2]), 0x04000c0cu);
    w[h] = lo | hi;
  }
  return make_uint2(w[0], w[1]);
}

template <int NT, bool SPLIT>
__device__ inline void store_quant8(int8_t* row, Lane<NT, SPLIT> l, int c, int pitch, uint2 q) {
  if constexpr (SPLIT) {
    if (l.at(c, 0) < pitch) *reinterpret_cast<uint32_t*>(row + l.at(c, 0)) = q.x;
    if (l.at(c, 1) < pitch) *reinterpret_cast<uint32_t*>(row + l.at(c, 1)) = q.y;
  } else {
    if (l.at(c, 0) < pitch) *reinterpret_cast<uint2*>(row + l.at(c, 0)) = q;
  }
}

}  // namespace rows
}  // namespace hna
