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

struct CacheParams {
  const void* x;  // rows: read by the write kernels
  void* out;      // rows: written by the read kernels
  uint8_t* data;
  uint8_t* scales;
  const int64_t* slots;
  int32_t* dev_error;
  int64_t rows, num_slots, row_stride, head_stride;
  int heads, d;
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

csa_status_t launch_scalar(const void* k, CacheParams& p, csa_stream_t stream) {
  int dev = 0, sms = 0;
  if (note(cudaGetDevice(&dev)) != cudaSuccess || device_sms(dev, &sms) != cudaSuccess)
    return CSA_ERR_CUDA;
  const int64_t warps = p.rows * p.heads * ((p.d + 31) / 32);
  const int64_t want = (warps + kCacheThreads / 32 - 1) / (kCacheThreads / 32);
  const int64_t most = 64 * static_cast<int64_t>(sms);
  void* args[] = {&p};
  return launch_pdl(k, dim3(static_cast<unsigned>(want < most ? want : most)), dim3(kCacheThreads), 0,
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
  const void* k = by_dtype(dtype, [&](auto t) {
    return by_format(format, [](auto f) {
      return reinterpret_cast<const void*>(cache_write_scalar_kernel<decltype(t)::value, decltype(f)::value>);
    });
  });
  return launch_scalar(k, p, stream);
}

extern "C" csa_status_t csa_cache_read(const void* data, const uint8_t* scales, int32_t format,
                                       const int64_t* slots, int64_t rows, int64_t num_slots,
                                       int32_t heads, int32_t d, void* out, int32_t dtype,
                                       int64_t out_row_stride, int64_t out_head_stride,
                                       int32_t* dev_error, csa_stream_t stream) {
  const csa_status_t st = check_cache(out, dtype, rows, heads, d, out_row_stride, out_head_stride,
                                      slots, num_slots, format, data, scales, dev_error);
  if (st != CSA_OK || rows == 0) return st;
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
  const void* k = by_dtype(dtype, [&](auto t) {
    return by_format(format, [](auto f) {
      return reinterpret_cast<const void*>(cache_read_scalar_kernel<decltype(t)::value, decltype(f)::value>);
    });
  });
  return launch_scalar(k, p, stream);
}
