// csa_element.cuh -- element types of the head norm, the rotation and the paged cache:
// loads and stores of bf16, fp16 and fp32 as fp32, and the cache's 8- and 4-bit codes.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "csa_compressor.h"
#include "csa_device.cuh"

namespace csa {

template <int DTYPE>
struct Element;

template <>
struct Element<CSA_DTYPE_BF16> {
  using T = uint16_t;
  static __device__ __forceinline__ float to_float(T v) { return __uint_as_float(static_cast<uint32_t>(v) << 16); }
  static __device__ __forceinline__ T from_float(float v) {
    return __bfloat16_as_ushort(__float2bfloat16_rn(v));
  }
};
template <>
struct Element<CSA_DTYPE_FP16> {
  using T = uint16_t;
  static __device__ __forceinline__ float to_float(T v) { return __half2float(__ushort_as_half(v)); }
  static __device__ __forceinline__ T from_float(float v) {
    return __half_as_ushort(__float2half_rn(v));
  }
};
template <>
struct Element<CSA_DTYPE_FP32> {
  using T = float;
  static __device__ __forceinline__ float to_float(T v) { return v; }
  static __device__ __forceinline__ T from_float(float v) { return v; }
};

__host__ __device__ constexpr int dtype_size(int dtype) { return dtype == CSA_DTYPE_FP32 ? 4 : 2; }

// Calls f with the element type as a compile-time constant.
template <typename F>
auto by_dtype(int dtype, F f) {
  return dtype == CSA_DTYPE_BF16   ? f(std::integral_constant<int, CSA_DTYPE_BF16>{})
         : dtype == CSA_DTYPE_FP16 ? f(std::integral_constant<int, CSA_DTYPE_FP16>{})
                                   : f(std::integral_constant<int, CSA_DTYPE_FP32>{});
}

// Whether an output [rows, heads, d] with these strides writes every element to a place of its
// own: the heads of a row (or the rows of a head) side by side, d columns each, and these
// groups one behind another.
inline bool separate(int64_t rows, int64_t heads, int64_t d, int64_t row_stride, int64_t head_stride) {
  struct Axis {
    int64_t n, stride;
  } inner{heads, head_stride}, outer{rows, row_stride};
  if (rows < 1) return true;
  if (outer.n > 1 && (inner.n == 1 || outer.stride < inner.stride)) {
    const Axis t = inner;
    inner = outer;
    outer = t;
  }
  if (inner.n > 1 && inner.stride < d) return false;
  const __int128 span = static_cast<__int128>(inner.n - 1) * inner.stride + d;
  return outer.n <= 1 || outer.stride >= span;
}

inline bool is_aligned(const void* p, uintptr_t a) {
  return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0;
}

// 8 consecutive columns, 16-byte aligned: as they lie in memory, and as fp32.
template <int DTYPE>
struct Eight {
  static constexpr int kWords = dtype_size(DTYPE) / 2;  // 16-byte words
  uint4 w[kWords];
  __device__ __forceinline__ void load(const void* p) {
    const uint4* q = static_cast<const uint4*>(p);
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      asm volatile("ld.global.cs.v4.u32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(w[i].x), "=r"(w[i].y), "=r"(w[i].z), "=r"(w[i].w)
                   : "l"(q + i));
    }
  }
  __device__ __forceinline__ void store(void* p) const {
    uint4* q = static_cast<uint4*>(p);
#pragma unroll
    for (int i = 0; i < kWords; ++i) q[i] = w[i];
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (DTYPE == CSA_DTYPE_FP32) {
        v[2 * i] = __uint_as_float(i < 2 ? (i == 0 ? w[0].x : w[0].z) : (i == 2 ? w[kWords - 1].x : w[kWords - 1].z));
        v[2 * i + 1] = __uint_as_float(i < 2 ? (i == 0 ? w[0].y : w[0].w) : (i == 2 ? w[kWords - 1].y : w[kWords - 1].w));
      } else {
        const uint32_t x = i == 0 ? w[0].x : i == 1 ? w[0].y : i == 2 ? w[0].z : w[0].w;
        if constexpr (DTYPE == CSA_DTYPE_BF16) {
          v[2 * i] = bf16_lo(x);
          v[2 * i + 1] = bf16_hi(x);
        } else {
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&x));
          v[2 * i] = f.x;
          v[2 * i + 1] = f.y;
        }
      }
    }
  }
  static __device__ __forceinline__ uint32_t two(float a, float b) {
    if constexpr (DTYPE == CSA_DTYPE_BF16) return pack_bf16x2(a, b);
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  __device__ __forceinline__ void set(const float (&v)[8]) {
    if constexpr (DTYPE == CSA_DTYPE_FP32) {
      w[0] = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
      w[kWords - 1] = make_uint4(__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]), __float_as_uint(v[7]));
    } else {
      w[0] = make_uint4(two(v[0], v[1]), two(v[2], v[3]), two(v[4], v[5]), two(v[6], v[7]));
    }
  }
};

// ---------------------------------------------------------------------------------
// Cache codes. Two e4m3 codes to two fp32 values (both exact in fp16), four e2m1 codes
// likewise, and back, rounding to nearest even.
// ---------------------------------------------------------------------------------
__device__ __forceinline__ float2 e4m3x2_to_float2(uint16_t c) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(c));
  return __half22float2(*reinterpret_cast<__half2*>(&h));
}
__device__ __forceinline__ uint16_t float2_to_e4m3x2(float lo, float hi) {
  uint16_t c;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(c) : "f"(hi), "f"(lo));
  return c;
}
__device__ __forceinline__ float2 e2m1x2_to_float2(uint32_t c) {
  uint32_t h;
  asm("{\n\t.reg .b8 b;\n\tcvt.u8.u32 b, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, b;\n\t}"
      : "=r"(h)
      : "r"(c & 0xFFu));
  return __half22float2(*reinterpret_cast<__half2*>(&h));
}
__device__ __forceinline__ uint32_t float2_to_e2m1x2(float lo, float hi) {
  uint32_t c;
  asm("{\n\t.reg .b8 b;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %1, %2;\n\tcvt.u32.u8 %0, b;\n\t}"
      : "=r"(c)
      : "f"(hi), "f"(lo));
  return c;
}

// Scale byte of a group with largest magnitude `amax`, given the magnitude's bits: the smallest k
// in [0, 254] with amax <= most * 2^(k - 127), most = 1.75 * 2^8 (e4m3) or 1.5 * 2^2 (e2m1):
// amax's exponent less 8 or 2, one more where its mantissa is above most's. A non-finite
// amax gives 255. (Finite ones end at 253.)
template <int FORMAT>
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax_bits) {
  constexpr int kEmax = FORMAT == CSA_CACHE_E4M3 ? 8 : 2;
  constexpr uint32_t kMant = FORMAT == CSA_CACHE_E4M3 ? 0x600000u : 0x400000u;
  const int ex = static_cast<int>(amax_bits >> 23);
  if (ex == 255) return 255u;
  const int k = ex - kEmax + ((amax_bits & 0x7FFFFFu) > kMant ? 1 : 0);
  return k < 0 ? 0u : static_cast<uint32_t>(k);
}
// 2^(k - 127); byte 0 is the subnormal 2^-127, byte 255 a NaN.
__device__ __forceinline__ float scale_value(uint32_t k) {
  return k == 0 ? __uint_as_float(0x00400000u)
                : (k == 255 ? __uint_as_float(0x7FC00000u) : __uint_as_float(k << 23));
}
// 2^(127 - k), exact for the bytes that scale_byte gives to finite groups (0..253): the
// reciprocal of a power of two, so value * inverse is the exact quotient.
__device__ __forceinline__ float scale_inverse(uint32_t k) { return __uint_as_float((254u - k) << 23); }

}  // namespace csa
