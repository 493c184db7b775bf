// Device helpers of the kernels that multiply operands of either type on the
// matrix cores from 16-byte fragments (gfx950): the products of a fragment pair,
// fragments of operands whose rows run along the product's sum, and the address
// of a k-major tile's 16-byte chunks in LDS.
#pragma once

#include "hna_hot.h"

namespace hna {
namespace mm {

using hot::lds_ptr;
using hot::u32x4;

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4* lds_s16x4;

// c += a b over one 16-byte fragment of k a lane: bf16 16 elements (lane l holds
// k = 8 (l / 32) + e), fp32 8 elements (k = 4 (l / 32) + e)
template <typename T>
__device__ inline void mma16(f32x16& c, const uint4& a, const uint4& b) {
  if constexpr (sizeof(T) == 2) {
    c = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  } else {
    c = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(a.x), __uint_as_float(b.x), c, 0, 0, 0);
    c = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(a.y), __uint_as_float(b.y), c, 0, 0, 0);
    c = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(a.z), __uint_as_float(b.z), c, 0, 0, 0);
    c = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(a.w), __uint_as_float(b.w), c, 0, 0, 0);
  }
}

// 4 x 4 elements of 16 bits transposed among 16 lanes: lane i of the 16 gives the
// address of row i / 4, columns 4 (i % 4) .. + 3, and gets column i of the 4 rows
__device__ inline uint2 read_tr16(const unsigned char* p) {
  const s16x4 v = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)(lds_ptr)const_cast<unsigned char*>(p));
  return __builtin_bit_cast(uint2, v);
}

// A tile whose LDS rows run along k, each PITCH bytes of the other dimension.
// XOR applied to the 16-byte chunk index of row k: the four rows that 16 lanes
// read at once (64 bytes of each for the two sixteens of a fragment) lie in
// different banks.  fp32 rows are read 4 bytes a lane and need none.
template <typename T, int PITCH>
__device__ inline int ksw(int k) {
  if constexpr (sizeof(T) == 4 || PITCH <= 64) return 0;
  else if constexpr (PITCH == 128) return ((k >> 1) & 1) << 2;
  else return (k & 3) << 2;
}
// the lane's part of a fragment's address in such a tile (fragment of 32 columns
// from column 0, k from 0), to be XORed with 64 f for columns 32 f of bf16
template <typename T, int PITCH>
__device__ inline int klane(int l) {
  if constexpr (sizeof(T) == 2) {
    const int r = (l & 15) >> 2;
    return (8 * (l >> 5) + r) * PITCH + ((ksw<T, PITCH>(r) ^ (2 * ((l >> 4) & 1) + ((l & 3) >> 1))) << 4) + (l & 1) * 8;
  } else {
    return 4 * (l >> 5) * PITCH + (l & 31) * 4;
  }
}
// fragment of 32 columns 32 f .. of 16 (bf16) or 8 (fp32) rows k from the h-th such step on
template <typename T, int PITCH>
__device__ inline uint4 kfrag(const unsigned char* tile, int lane_part, int f, int h) {
  if constexpr (sizeof(T) == 2) {
    const unsigned char* q = tile + (PITCH >= 128 ? (lane_part ^ (64 * (f & 3))) + 256 * (f >> 2) : lane_part) + 16 * h * PITCH;
    const uint2 lo = read_tr16(q), hi = read_tr16(q + 4 * PITCH);
    return make_uint4(lo.x, lo.y, hi.x, hi.y);
  } else {
    const unsigned char* q = tile + lane_part + 128 * f + 8 * h * PITCH;
    return make_uint4(*reinterpret_cast<const uint32_t*>(q), *reinterpret_cast<const uint32_t*>(q + PITCH),
                      *reinterpret_cast<const uint32_t*>(q + 2 * PITCH), *reinterpret_cast<const uint32_t*>(q + 3 * PITCH));
  }
}

// 4 floats as T
template <typename T>
struct Four;
template <>
struct Four<__bf16> {
  typedef uint2 type;
  __device__ static inline uint2 of(float a, float b, float c, float d) { return make_uint2(pack_bf16x2(a, b), pack_bf16x2(c, d)); }
};
template <>
struct Four<float> {
  typedef float4 type;
  __device__ static inline float4 of(float a, float b, float c, float d) { return make_float4(a, b, c, d); }
};

template <typename T>
__device__ inline T to_type(float f) {
  if constexpr (sizeof(T) == 2) return __builtin_bit_cast(T, (uint16_t)pack_bf16x2(f, 0.f));
  else return f;
}

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;

// 1 / (1 + exp(-x)); 0 where exp(-x) passes fp32's range
__device__ inline float sigmoid(float x) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-kLog2e * x));
}

}  // namespace mm
}  // namespace hna
