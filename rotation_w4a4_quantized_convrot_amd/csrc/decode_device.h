// Device helpers shared by the decoding operators (w4a16.hip, rotary.hip, kv8.hip): loads of
// 16 values, the regular Hadamard rotation of values held 16 to a lane, bf16 rounding.
#pragma once

#include "convrot_internal.h"

namespace convrot {
namespace {

typedef _Float16 half8 __attribute__((ext_vector_type(8)));
typedef _Float16 half2_t __attribute__((ext_vector_type(2)));
typedef float float4_t __attribute__((ext_vector_type(4)));
typedef uint32_t uint4_t __attribute__((ext_vector_type(4)));
typedef uint32_t uint2_t __attribute__((ext_vector_type(2)));

__device__ __forceinline__ float bf16_to_f32(uint16_t b) { return __uint_as_float(uint32_t(b) << 16); }

// Round to nearest even; NaN stays NaN.
__device__ __forceinline__ uint16_t f32_to_bf16(float f) {
  const uint32_t u = __float_as_uint(f);
  if ((u & 0x7FFFFFFFu) > 0x7F800000u) return uint16_t((u >> 16) | 0x40u);
  return uint16_t((u + 0x7FFFu + ((u >> 16) & 1u)) >> 16);
}

template <typename T> __device__ __forceinline__ float load_one(const T* p);
template <> __device__ __forceinline__ float load_one<float>(const float* p) { return *p; }
template <> __device__ __forceinline__ float load_one<uint16_t>(const uint16_t* p) { return bf16_to_f32(*p); }

// Sixteen consecutive values, the first `left` of them there (left <= 0: none) and the rest
// zero.  `wide`: the address is a multiple of 16 bytes.
template <typename T>
__device__ __forceinline__ void load16(const T* p, int64_t left, bool wide, float (&v)[16]) {
  if (left >= 16 && wide) {
    constexpr int kPer = 16 / sizeof(T);
#pragma unroll
    for (int i = 0; i < 16 / kPer; ++i) {
      const uint4_t w = reinterpret_cast<const uint4_t*>(p)[i];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (sizeof(T) == 4) {
          v[4 * i + j] = __uint_as_float(w[j]);
        } else {
          v[8 * i + 2 * j] = __uint_as_float(w[j] << 16);
          v[8 * i + 2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
        }
      }
    }
  } else {
#pragma unroll
    for (int e = 0; e < 16; ++e) v[e] = e < left ? load_one<T>(p + e) : 0.0f;
  }
}

template <int CTRL>
__device__ __forceinline__ float lane_dpp(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xF, 0xF, false));
}
template <int CTRL>
__device__ __forceinline__ uint32_t lane_dpp_u(uint32_t v) {
  return uint32_t(__builtin_amdgcn_update_dpp(0, int(v), CTRL, 0xF, 0xF, false));
}
constexpr int kQuadXor1 = 0xB1, kQuadXor2 = 0x4E, kRowRor4 = 0x124, kRowRor8 = 0x128;

// One radix-4 digit of H_g / sqrt(g): each factor is (J - 2I) / 2, so a value becomes half the
// sum of its four less itself.
__device__ __forceinline__ void digit_in_lane(float& a, float& b, float& c, float& d) {
  const float h = 0.5f * ((a + b) + (c + d));
  a = h - a;
  b = h - b;
  c = h - c;
  d = h - d;
}

// Rotates values held 16 to a lane, element 16 * lane + e, in windows of g = 4^digits (digits
// 2 to 5, the windows starting at lanes that are multiples of g / 16; 0: nothing).  Digits 0
// and 1 are in a lane's registers; digit 2 is lane bits 0-1, digit 3 bits 2-3 (both by DPP: a
// sum over two rotations of a row of 16 by 8 and 4 is the sum over the four lanes of equal bits
// 0-1), digit 4 bits 4-5.  At most 13 VALU operations an element, no LDS before digit 4.
__device__ __forceinline__ void rotate16(float (&v)[16], int digits) {
  if (digits < 2) return;
#pragma unroll
  for (int i = 0; i < 4; ++i) digit_in_lane(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
#pragma unroll
  for (int i = 0; i < 4; ++i) digit_in_lane(v[i], v[4 + i], v[8 + i], v[12 + i]);
  if (digits >= 3) {
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      float s = v[e] + lane_dpp<kQuadXor1>(v[e]);
      s += lane_dpp<kQuadXor2>(s);
      v[e] = 0.5f * s - v[e];
    }
  }
  if (digits >= 4) {
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      float s = v[e] + lane_dpp<kRowRor8>(v[e]);
      s += lane_dpp<kRowRor4>(s);
      v[e] = 0.5f * s - v[e];
    }
  }
  if (digits >= 5) {
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      float s = v[e] + __shfl_xor(v[e], 16);
      s += __shfl_xor(s, 32);
      v[e] = 0.5f * s - v[e];
    }
  }
}

// Largest |v[e]| as the bits of a non-negative float: they order as integers, a NaN above Inf.
__device__ __forceinline__ uint32_t abs_max16(const float (&v)[16]) {
  uint32_t m = 0;
#pragma unroll
  for (int e = 0; e < 16; ++e) m = max(m, __float_as_uint(v[e]) & 0x7FFFFFFFu);
  return m;
}

// Maximum over a row of 16 lanes.
__device__ __forceinline__ uint32_t row_max(uint32_t m) {
  m = max(m, lane_dpp_u<kQuadXor1>(m));
  m = max(m, lane_dpp_u<kQuadXor2>(m));
  m = max(m, lane_dpp_u<kRowRor4>(m));
  return max(m, lane_dpp_u<kRowRor8>(m));
}

// Maximum over a row of 16 lanes, or over the wave where a window of 1024 spans it.
__device__ __forceinline__ uint32_t unit_max(uint32_t m, int digits) {
  m = row_max(m);
  if (digits >= 5) {
    m = max(m, uint32_t(__shfl_xor(int(m), 16)));
    m = max(m, uint32_t(__shfl_xor(int(m), 32)));
  }
  return m;
}

// An exact power of two that takes values of largest magnitude `bits`, times `growth` = 2^grow
// at most, to at most 2^15 (fp16 holds 65504), and its inverse.  A zero row gives 1; a row that
// holds an Inf or a NaN gives an inverse of NaN, which the caller multiplies the row's result
// with.  Where the exact power would leave fp32's normal range it is clamped: rows below
// 2^-110 then use less of fp16's range.
__device__ __forceinline__ void half_range(uint32_t bits, int grow, float* to_half, float* back) {
  int e = int(bits >> 23) - 127 + 1 + grow;           // magnitude * growth < 2^e
  e = min(max(e, -110), 126 + 15);
  const int up = 15 - e;                              // in [-126, 125]
  *to_half = bits == 0 ? 1.0f : __uint_as_float(uint32_t(127 + up) << 23);
  *back = bits == 0 ? 1.0f
          : bits >= 0x7F800000u ? __uint_as_float(0x7FC00000u)
                                : __uint_as_float(uint32_t(127 - up) << 23);
}

// A barrier for what is in LDS: loads from memory may still be on their way.
__device__ __forceinline__ void lds_barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

__host__ __device__ __forceinline__ int digits_of(int g) {
  return g == 16 ? 2 : g == 64 ? 3 : g == 256 ? 4 : g == 1024 ? 5 : 0;
}

}  // namespace
}  // namespace convrot
