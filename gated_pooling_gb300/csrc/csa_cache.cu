// csa_cache.cu -- rows into the paged cache (bf16, or e4m3 / e2m1 codes with one power-of-two
// scale per 32 columns) and back; formats and rules are in csa_compressor.h.
//
// Both are bound by HBM bytes: every value is read once and written once.
//
// The scale is a power of two because these codes have exponents of their own: a finer
// scale would only move values within a binade, and with a power of two value / scale and
// code * scale are exact, so each value is rounded once, to its nearest code, and the
// quotient needs no division.
#include <climits>
#include <cstdint>
#include <type_traits>

#include "csa_compressor.h"
#include "csa_element.cuh"
#include "csa_internal.h"

namespace csa {
namespace {

constexpr int kCacheThreads = 256;

// Division of numbers below 2^31 by n: floor(x m / 2^(31 + l)) with l = ceil(log2 n) and m =
// floor(2^(31 + l) / n) + 1 < 2^32 is exact there (Granlund and Montgomery 1994).
struct FastDivisor {
  uint32_t n = 1, m = 0, shift = 31;
  FastDivisor() = default;
  explicit FastDivisor(uint32_t d) : n(d) {
    uint32_t l = 0;
    while ((1ull << l) < d) ++l;
    shift = 31 + l;
    m = static_cast<uint32_t>((1ull << shift) / d + (d == 1 ? 0 : 1));
  }
  __device__ __forceinline__ uint32_t quotient(uint32_t x) const {
    return static_cast<uint32_t>((static_cast<uint64_t>(x) * m) >> shift);
  }
};

struct CacheParams {
  const void* x;  // rows: read by the write kernels
  void* out;      // rows: written by the read kernels
  uint8_t* data;
  uint8_t* scales;
  const int64_t* slots;
  int32_t* dev_error;
  int64_t rows, num_slots, row_stride, head_stride;
  int heads, d;
  FastDivisor pieces, by_heads;  // vector kernels: pieces of a row's head, heads
};

// Slot of a row, or -1 where the row is left out; reports slots past the pool's end.
__device__ __forceinline__ int64_t row_slot(const CacheParams& p, int64_t row) {
  const int64_t s = __ldg(p.slots + row);
  if (s < p.num_slots) return s < 0 ? -1 : s;
  if (p.dev_error != nullptr) *p.dev_error = CSA_DEVERR_SLOT;
  return -1;
}

// Scalar kernels, any alignment: a warp per 32 consecutive columns of a row's head (the last
// ones of a bf16 cache's head may be fewer), a lane per column.
template <int DTYPE, int FORMAT>
__global__ void __launch_bounds__(kCacheThreads) cache_write_scalar_kernel(CacheParams p) {
  using E = Element<DTYPE>;
  const int lane = threadIdx.x & 31;
  const int groups = (p.d + 31) / 32;
  pdl_wait();
  const int64_t n = p.rows * p.heads * groups;
  for (int64_t u = (static_cast<int64_t>(blockIdx.x) * kCacheThreads + threadIdx.x) / 32; u < n;
       u += static_cast<int64_t>(gridDim.x) * (kCacheThreads / 32)) {
    const int64_t rh = u / groups, row = rh / p.heads;
    const int g = static_cast<int>(u - rh * groups), head = static_cast<int>(rh - row * p.heads);
    const int64_t slot = row_slot(p, row);
    if (slot < 0) continue;
    const int col = g * 32 + lane;
    const typename E::T* x = static_cast<const typename E::T*>(p.x) + row * p.row_stride + head * p.head_stride;
    const float v = col < p.d ? E::to_float(x[col]) : 0.f;
    const int64_t entry = slot * p.heads + head;
    if constexpr (FORMAT == CSA_CACHE_BF16) {
      if (col < p.d)
        reinterpret_cast<uint16_t*>(p.data)[entry * p.d + col] = Element<CSA_DTYPE_BF16>::from_float(v);
    } else {
      const uint32_t top = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(v) & 0x7FFFFFFFu);
      const uint32_t k = scale_byte<FORMAT>(top);
      const float q = v * scale_inverse(k == 255u ? 127u : k);
      if (lane == 0) p.scales[entry * groups + g] = static_cast<uint8_t>(k);
      if constexpr (FORMAT == CSA_CACHE_E4M3) {
        p.data[entry * p.d + col] = static_cast<uint8_t>(float2_to_e4m3x2(q, 0.f) & 0xFFu);
      } else {
        const float hi = __shfl_down_sync(0xFFFFFFFFu, q, 1);
        if (lane % 2 == 0) p.data[entry * (p.d / 2) + col / 2] = static_cast<uint8_t>(float2_to_e2m1x2(q, hi));
      }
    }
  }
}

template <int DTYPE, int FORMAT>
__global__ void __launch_bounds__(kCacheThreads) cache_read_scalar_kernel(CacheParams p) {
  using E = Element<DTYPE>;
  const int lane = threadIdx.x & 31;
  const int groups = (p.d + 31) / 32;
  pdl_wait();
  const int64_t n = p.rows * p.heads * groups;
  for (int64_t u = (static_cast<int64_t>(blockIdx.x) * kCacheThreads + threadIdx.x) / 32; u < n;
       u += static_cast<int64_t>(gridDim.x) * (kCacheThreads / 32)) {
    const int64_t rh = u / groups, row = rh / p.heads;
    const int g = static_cast<int>(u - rh * groups), head = static_cast<int>(rh - row * p.heads);
    const int64_t slot = row_slot(p, row);
    if (slot < 0) continue;
    const int col = g * 32 + lane;
    if (col >= p.d) continue;
    const int64_t entry = slot * p.heads + head;
    float v;
    if constexpr (FORMAT == CSA_CACHE_BF16) {
      v = Element<CSA_DTYPE_BF16>::to_float(reinterpret_cast<const uint16_t*>(p.data)[entry * p.d + col]);
    } else {
      const float s = scale_value(p.scales[entry * groups + g]);
      if constexpr (FORMAT == CSA_CACHE_E4M3) {
        v = e4m3x2_to_float2(p.data[entry * p.d + col]).x * s;
      } else {
        const float2 two = e2m1x2_to_float2(p.data[entry * (p.d / 2) + col / 2]);
        v = (lane % 2 == 0 ? two.x : two.y) * s;
      }
    }
    typename E::T* out = static_cast<typename E::T*>(p.out) + row * p.row_stride + head * p.head_stride;
    out[col] = E::from_float(v);
  }
}

// Vector kernels: a thread takes 16 consecutive columns of a row's head (8 of a bf16 cache), two
// neighbouring threads share a scale; 16-byte accesses (8 bytes of e2m1). What is left beside
// the bytes is finding a thread's place, so its two divisions are products with reciprocals
// (items below 2^31), and 8 columns a thread, with twice the places, was slower: 24571 entries
// of 512 written and read back took 25.4 us instead of 14.9 (5.1 TB/s).
// One item a thread: with 2 or 4 under way the same took 16.0 or 19.4 us instead of 14.9.
constexpr int kItems = 1;
template <int FORMAT>
struct CachePiece {
  static constexpr int kCols = FORMAT == CSA_CACHE_BF16 ? 8 : 16;
};

// Row, head and first column of a thread's item.
struct ItemAt {
  int row, head, col;
  __device__ __forceinline__ ItemAt(const CacheParams& p, uint32_t item, int cols) {
    const uint32_t rh = p.pieces.quotient(item), r = p.by_heads.quotient(rh);
    col = static_cast<int>(item - rh * p.pieces.n) * cols;
    row = static_cast<int>(r);
    head = static_cast<int>(rh - r * p.by_heads.n);
  }
};

template <int DTYPE, int FORMAT>
__global__ void __launch_bounds__(kCacheThreads) cache_write_vec_kernel(CacheParams p) {
  using T = typename Element<DTYPE>::T;
  constexpr int kCols = CachePiece<FORMAT>::kCols, kEights = kCols / 8;
  pdl_wait();
  const uint32_t items = static_cast<uint32_t>(p.rows) * p.heads * p.pieces.n;
  const uint32_t i0 = blockIdx.x * (kCacheThreads * kItems) + threadIdx.x;
  Eight<DTYPE> v[kItems][kEights];
  int64_t entry[kItems];  // -1: left out
  int cols[kItems];
#pragma unroll
  for (int k = 0; k < kItems; ++k) {
    const uint32_t i = i0 + k * kCacheThreads;
    entry[k] = -1;
    cols[k] = 0;
    if (i < items) {
      const ItemAt at(p, i, kCols);
      cols[k] = at.col;
      const int64_t slot = row_slot(p, at.row);
      if (slot >= 0) entry[k] = slot * p.heads + at.head;
      const T* x = static_cast<const T*>(p.x) + static_cast<int64_t>(at.row) * p.row_stride + at.head * p.head_stride + at.col;
#pragma unroll
      for (int e = 0; e < kEights; ++e) v[k][e].load(x + 8 * e);
    }
  }
#pragma unroll
  for (int k = 0; k < kItems; ++k) {
    const int col = cols[k];
    float f[kEights][8];
#pragma unroll
    for (int e = 0; e < kEights; ++e) v[k][e].get(f[e]);
    if constexpr (FORMAT == CSA_CACHE_BF16) {
      Eight<CSA_DTYPE_BF16> out;
      out.set(f[0]);
      if (entry[k] >= 0) out.store(reinterpret_cast<uint16_t*>(p.data) + entry[k] * p.d + col);
    } else {
      // the group's largest magnitude, as bits: an infinity or NaN is above every number
      uint32_t top = 0;
#pragma unroll
      for (int e = 0; e < kEights; ++e)
#pragma unroll
        for (int c = 0; c < 8; ++c) top = max(top, __float_as_uint(f[e][c]) & 0x7FFFFFFFu);
      top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
      const uint32_t b = scale_byte<FORMAT>(top);
      const float inv = scale_inverse(b == 255u ? 127u : b);
      if (entry[k] >= 0) {
        uint32_t w[4];
        if constexpr (FORMAT == CSA_CACHE_E4M3) {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const float* g = &f[q / 2][(q % 2) * 4];
            w[q] = float2_to_e4m3x2(g[0] * inv, g[1] * inv) |
                   (static_cast<uint32_t>(float2_to_e4m3x2(g[2] * inv, g[3] * inv)) << 16);
          }
          *reinterpret_cast<uint4*>(p.data + entry[k] * p.d + col) = make_uint4(w[0], w[1], w[2], w[3]);
        } else {
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            const float* g = f[q];
            w[q] = float2_to_e2m1x2(g[0] * inv, g[1] * inv) | (float2_to_e2m1x2(g[2] * inv, g[3] * inv) << 8) |
                   (float2_to_e2m1x2(g[4] * inv, g[5] * inv) << 16) | (float2_to_e2m1x2(g[6] * inv, g[7] * inv) << 24);
          }
          *reinterpret_cast<uint2*>(p.data + entry[k] * (p.d / 2) + col / 2) = make_uint2(w[0], w[1]);
        }
        if ((col & 16) == 0) p.scales[entry[k] * (p.d / CSA_CACHE_GROUP) + col / CSA_CACHE_GROUP] = static_cast<uint8_t>(b);
      }
    }
  }
}

template <int DTYPE, int FORMAT>
__global__ void __launch_bounds__(kCacheThreads) cache_read_vec_kernel(CacheParams p) {
  using T = typename Element<DTYPE>::T;
  constexpr int kCols = CachePiece<FORMAT>::kCols, kEights = kCols / 8;
  pdl_wait();
  const uint32_t items = static_cast<uint32_t>(p.rows) * p.heads * p.pieces.n;
  const uint32_t i0 = blockIdx.x * (kCacheThreads * kItems) + threadIdx.x;
  uint4 v[kItems];
  uint32_t b[kItems];
  T* to[kItems];  // null: left out
#pragma unroll
  for (int k = 0; k < kItems; ++k) {
    const uint32_t i = i0 + k * kCacheThreads;
    to[k] = nullptr;
    if (i < items) {
      const ItemAt at(p, i, kCols);
      const int64_t slot = row_slot(p, at.row);
      if (slot >= 0) {
        to[k] = static_cast<T*>(p.out) + static_cast<int64_t>(at.row) * p.row_stride + at.head * p.head_stride + at.col;
        const int64_t entry = slot * p.heads + at.head;
        if constexpr (FORMAT == CSA_CACHE_BF16) {
          v[k] = __ldg(reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(p.data) + entry * p.d + at.col));
        } else {
          b[k] = __ldg(p.scales + entry * (p.d / CSA_CACHE_GROUP) + at.col / CSA_CACHE_GROUP);
          if constexpr (FORMAT == CSA_CACHE_E4M3) {
            v[k] = __ldg(reinterpret_cast<const uint4*>(p.data + entry * p.d + at.col));
          } else {
            const uint2 w = __ldg(reinterpret_cast<const uint2*>(p.data + entry * (p.d / 2) + at.col / 2));
            v[k].x = w.x;
            v[k].y = w.y;
          }
        }
      }
    }
  }
#pragma unroll
  for (int k = 0; k < kItems; ++k) {
    if (to[k] == nullptr) continue;
    float f[kEights][8];
    if constexpr (FORMAT == CSA_CACHE_BF16) {
      Eight<CSA_DTYPE_BF16> e;
      e.w[0] = v[k];
      e.get(f[0]);
    } else {
      const float s = scale_value(b[k]);
      const uint32_t w[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const float2 two = FORMAT == CSA_CACHE_E4M3 ? e4m3x2_to_float2((w[q / 2] >> (16 * (q % 2))) & 0xFFFFu)
                                                   : e2m1x2_to_float2(w[q / 4] >> (8 * (q % 4)));
        f[q / 4][(q % 4) * 2] = two.x * s;
        f[q / 4][(q % 4) * 2 + 1] = two.y * s;
      }
    }
#pragma unroll
    for (int e = 0; e < kEights; ++e) {
      Eight<DTYPE> o;
      o.set(f[e]);
      o.store(to[k] + 8 * e);
    }
  }
}

// Calls f with the cache format as a compile-time constant.
template <typename F>
auto by_format(int format, F f) {
  return format == CSA_CACHE_BF16   ? f(std::integral_constant<int, CSA_CACHE_BF16>{})
         : format == CSA_CACHE_E4M3 ? f(std::integral_constant<int, CSA_CACHE_E4M3>{})
                                    : f(std::integral_constant<int, CSA_CACHE_E2M1>{});
}

csa_status_t check_cache(const void* x, int32_t dtype, int64_t rows, int32_t heads, int32_t d,
                         int64_t row_stride, int64_t head_stride, const int64_t* slots,
                         int64_t num_slots, int32_t format, const void* data, const void* scales,
                         const int32_t* dev_error) {
  if (rows < 0 || heads < 1 || d < 1 || num_slots < 0 || row_stride < 0 || head_stride < 0)
    return CSA_ERR_INVALID_VALUE;
  if (dtype < CSA_DTYPE_BF16 || dtype > CSA_DTYPE_FP32 || format < CSA_CACHE_BF16 ||
      format > CSA_CACHE_E2M1)
    return CSA_ERR_UNSUPPORTED;
  if (format != CSA_CACHE_BF16 && d % CSA_CACHE_GROUP != 0) return CSA_ERR_UNSUPPORTED;
  if (d > INT_MAX / heads || rows > INT64_MAX / 64 / (static_cast<int64_t>(heads) * d) ||
      num_slots > INT64_MAX / 64 / (static_cast<int64_t>(heads) * d))
    return CSA_ERR_UNSUPPORTED;
  if (!is_aligned(x, dtype_size(dtype)) || !is_aligned(slots, 8) || !is_aligned(dev_error, 4) ||
      (format == CSA_CACHE_BF16 && !is_aligned(data, 2)))
    return CSA_ERR_INVALID_VALUE;
  if (rows > 0 && (x == nullptr || slots == nullptr)) return CSA_ERR_INVALID_VALUE;
  if (num_slots > 0 && (data == nullptr || (format != CSA_CACHE_BF16 && scales == nullptr)))
    return CSA_ERR_INVALID_VALUE;
  return CSA_OK;
}

// Whether a call's shapes and pointers suit the vector kernels.
bool vector_call(CacheParams& p, const void* x, int format) {
  const int cols = format == CSA_CACHE_BF16 ? 8 : 16;
  if (p.d % 8 != 0 || p.row_stride % 8 != 0 || p.head_stride % 8 != 0 || !is_aligned(x, 16) ||
      !is_aligned(p.data, 16))
    return false;
  const int64_t items = p.rows * p.heads * (p.d / cols);
  if (items > INT_MAX - kCacheThreads * kItems) return false;
  p.pieces = FastDivisor(static_cast<uint32_t>(p.d / cols));
  p.by_heads = FastDivisor(static_cast<uint32_t>(p.heads));
  return true;
}

csa_status_t launch_cache(const void* k, bool vec, CacheParams& p, csa_stream_t stream) {
  int64_t blocks;
  if (vec) {
    blocks = (p.rows * p.heads * p.pieces.n + kCacheThreads * kItems - 1) / (kCacheThreads * kItems);
  } else {
    int dev = 0, sms = 0;
    if (note(cudaGetDevice(&dev)) != cudaSuccess || device_sms(dev, &sms) != cudaSuccess)
      return CSA_ERR_CUDA;
    const int64_t warps = p.rows * p.heads * ((p.d + 31) / 32);
    const int64_t want = (warps + kCacheThreads / 32 - 1) / (kCacheThreads / 32);
    const int64_t most = 64 * static_cast<int64_t>(sms);
    blocks = want < most ? want : most;
  }
  void* args[] = {&p};
  return launch_pdl(k, dim3(static_cast<unsigned>(blocks)), dim3(kCacheThreads), 0,
                    reinterpret_cast<cudaStream_t>(stream), args) == cudaSuccess
             ? CSA_OK
             : CSA_ERR_CUDA;
}

}  // namespace
}  // namespace csa

using namespace csa;

extern "C" csa_status_t csa_cache_write(const void* x, int32_t dtype, int64_t rows, int32_t heads,
                                        int32_t d, int64_t x_row_stride, int64_t x_head_stride,
                                        const int64_t* slots, int64_t num_slots, int32_t format,
                                        void* data, uint8_t* scales, int32_t* dev_error,
                                        csa_stream_t stream) {
  const csa_status_t st = check_cache(x, dtype, rows, heads, d, x_row_stride, x_head_stride, slots,
                                      num_slots, format, data, scales, dev_error);
  if (st != CSA_OK || rows == 0) return st;
  CacheParams p{};
  p.x = x;
  p.data = static_cast<uint8_t*>(data);
  p.scales = scales;
  p.slots = slots;
  p.dev_error = dev_error;
  p.rows = rows;
  p.num_slots = num_slots;
  p.row_stride = x_row_stride;
  p.head_stride = x_head_stride;
  p.heads = heads;
  p.d = d;
  const bool vec = vector_call(p, x, format);
  const void* k = by_dtype(dtype, [&](auto t) {
    return by_format(format, [&](auto f) {
      constexpr int T = decltype(t)::value, F = decltype(f)::value;
      return vec ? reinterpret_cast<const void*>(cache_write_vec_kernel<T, F>)
                 : reinterpret_cast<const void*>(cache_write_scalar_kernel<T, F>);
    });
  });
  return launch_cache(k, vec, p, stream);
}

extern "C" csa_status_t csa_cache_read(const void* data, const uint8_t* scales, int32_t format,
                                       const int64_t* slots, int64_t rows, int64_t num_slots,
                                       int32_t heads, int32_t d, void* out, int32_t dtype,
                                       int64_t out_row_stride, int64_t out_head_stride,
                                       int32_t* dev_error, csa_stream_t stream) {
  const csa_status_t st = check_cache(out, dtype, rows, heads, d, out_row_stride, out_head_stride,
                                      slots, num_slots, format, data, scales, dev_error);
  if (st != CSA_OK || rows == 0) return st;
  if (!separate(rows, heads, d, out_row_stride, out_head_stride)) return CSA_ERR_INVALID_VALUE;
  CacheParams p{};
  p.out = out;
  p.data = static_cast<uint8_t*>(const_cast<void*>(data));
  p.scales = const_cast<uint8_t*>(scales);
  p.slots = slots;
  p.dev_error = dev_error;
  p.rows = rows;
  p.num_slots = num_slots;
  p.row_stride = out_row_stride;
  p.head_stride = out_head_stride;
  p.heads = heads;
  p.d = d;
  const bool vec = vector_call(p, out, format);
  const void* k = by_dtype(dtype, [&](auto t) {
    return by_format(format, [&](auto f) {
      constexpr int T = decltype(t)::value, F = decltype(f)::value;
      return vec ? reinterpret_cast<const void*>(cache_read_vec_kernel<T, F>)
                 : reinterpret_cast<const void*>(cache_read_scalar_kernel<T, F>);
    });
  });
  return launch_cache(k, vec, p, stream);
}
