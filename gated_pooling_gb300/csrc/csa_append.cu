// csa_append.cu -- rows normed, turned to their positions and put into slots of the paged cache in one
// pass (the interface is in csa_compressor.h; norm and rotation as in csa_rope.cu, formats as in
// csa_cache.cu).
//
// What lies between reading x and writing the codes stays in registers, so a value is rounded once, to
// its code, where a norm and rotation followed by a cache write round twice and pass the row through
// memory in between. Bound by HBM bytes: x once, codes and scales once.
//
// Angles and roots are taken as for fp32 results whatever x's type: a code's border may be anywhere, and
// what fp32 rounding leaves is what a code may be off by.
#include <climits>
#include <cstdint>
#include <type_traits>

#include "csa_compressor.h"
#include "csa_element.cuh"
#include "csa_internal.h"
#include "csa_rope.cuh"

namespace csa {
namespace {

struct AppendParams {
  RopeParams r;
  uint8_t* data;
  uint8_t* scales;
  const int64_t* slots;
  int64_t num_slots;
  int32_t* dev_error;
  int each, more;  // vector kernel: heads of a warp, and the first warps that have one more
};

// A row's slot, -1 where the row is left out (a negative position or slot, or one past the pool, which is
// reported).
__device__ __forceinline__ int64_t append_slot(const AppendParams& p, int64_t row, int32_t pos) {
  const int64_t s = __ldg(p.slots + row);
  if (pos < 0 || s < 0) return -1;
  if (s < p.num_slots) return s;
  if (p.dev_error != nullptr) *p.dev_error = CSA_DEVERR_SLOT;
  return -1;
}

// cos and sin of a turn, times amp, without a branch: the nearest quarter of a turn is taken off the 32-bit fraction
// exactly, what is left, at most pi / 4 either way, goes through Taylor's series (the next terms are below 2e-9 and
// 3e-8), and the quarter swaps them and sets their signs.
__device__ __forceinline__ void quarter_cos_sin(int32_t pos, uint64_t per, float amp, float& c, float& s) {
  const uint64_t t = static_cast<uint64_t>(static_cast<int64_t>(pos)) * per;
  const uint32_t whole = static_cast<uint32_t>(t >> 32), q = (whole + 0x20000000u) >> 30;
  const float x = static_cast<float>(static_cast<int32_t>(whole - (q << 30))) * 1.46291807926715968105e-9f;  // pi 2^-31
  const float y = x * x;
  float a = fmaf(y, 1.f / 362880.f, -1.f / 5040.f);
  a = fmaf(y, a, 1.f / 120.f);
  a = fmaf(y, a, -1.f / 6.f);
  a = fmaf(x * y, a, x);
  float b = fmaf(y, 1.f / 40320.f, -1.f / 720.f);
  b = fmaf(y, b, 1.f / 24.f);
  b = fmaf(y, b, -0.5f);
  b = fmaf(y, b, 1.f);
  const bool odd = (q & 1u) != 0;
  c = (odd ? a : b) * __uint_as_float(__float_as_uint(amp) ^ (((q + 1u) & 2u) << 30));
  s = (odd ? b : a) * __uint_as_float(__float_as_uint(amp) ^ ((q & 2u) << 30));
}

// The largest magnitude of three, NaN if one is.
__device__ __forceinline__ float max_magnitude(float a, float b, float c) {
  float d;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// Scalar kernel, any d, rotation and alignment: a warp per row and head, which leaves the finished row in shared
// memory and then takes it 32 columns, a scale's, at a time. Four of everything side by side: few rows take as
// long as one, a chain of loads, angles and sums over lanes.
template <int DTYPE, int FORMAT>
__global__ void __launch_bounds__(kRopeThreads) append_scalar_kernel(const __grid_constant__ AppendParams q) {
  using E = Element<DTYPE>;
  using T = typename E::T;
  extern __shared__ float s_rows[];  // [warps][d]
  const RopeParams& p = q.r;
  const int lane = threadIdx.x & 31, groups = (p.d + 31) / 32;
  float* n = s_rows + (threadIdx.x >> 5) * p.d;
  pdl_wait();
  for (int64_t u = static_cast<int64_t>(blockIdx.x) * kRopeWarps + (threadIdx.x >> 5); u < p.units;
       u += static_cast<int64_t>(gridDim.x) * kRopeWarps) {
    const int64_t row = static_cast<int>(u) / p.heads, head = u - row * p.heads;  // (units below 2^31)
    const int32_t pos = p.pos != nullptr ? __ldg(p.pos + row) : 0;
    const int64_t slot = append_slot(q, row, pos);
    const T* x = static_cast<const T*>(p.x) + row * p.x_row + head * p.x_head;
    float ss = 0.f;
    for (int c0 = lane; c0 < p.d; c0 += 256) {
      T v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (c0 + 32 * i < p.d) v[i] = x[c0 + 32 * i];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (c0 + 32 * i < p.d) {
          const float f = E::to_float(v[i]);
          n[c0 + 32 * i] = f;
          ss = fmaf(f, f, ss);
        }
    }
    if (slot < 0) {
      __syncwarp();
      continue;
    }
    if (p.norm) {
      const float r = rsqrtf(warp_sum(ss) / static_cast<float>(p.d) + p.eps);
      for (int c0 = lane; c0 < p.d; c0 += 256) {
        float w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = p.weight != nullptr && c0 + 32 * i < p.d ? __ldg(p.weight + c0 + 32 * i) : 1.f;
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (c0 + 32 * i < p.d) n[c0 + 32 * i] = n[c0 + 32 * i] * r * w[i];
      }
    }
    __syncwarp();
    for (int i0 = lane; i0 < p.rot / 2; i0 += 128) {
      uint64_t per[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) per[k] = i0 + 32 * k < p.rot / 2 ? __ldg(p.turns + i0 + 32 * k) : 0;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        float cs, sn;
        quarter_cos_sin(pos, per[k], p.amp, cs, sn);
        if (i0 + 32 * k < p.rot / 2) {
          int a, b;
          pair_columns(p, i0 + 32 * k, a, b);
          const float va = n[a], vb = n[b];
          n[a] = va * cs - vb * sn;
          n[b] = va * sn + vb * cs;
        }
      }
    }
    __syncwarp();
    const int64_t entry = slot * p.heads + head;
    for (int g0 = 0; g0 < groups; g0 += 4) {
      float v[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = (g0 + k) * 32 + lane < p.d ? n[(g0 + k) * 32 + lane] : 0.f;
      if constexpr (FORMAT == CSA_CACHE_BF16) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int col = (g0 + k) * 32 + lane;
          if (col < p.d) reinterpret_cast<uint16_t*>(q.data)[entry * p.d + col] = Element<CSA_DTYPE_BF16>::from_float(v[k]);
        }
      } else {
        uint32_t top[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) top[k] = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(v[k]) & 0x7FFFFFFFu);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int g = g0 + k, col = g * 32 + lane;
          const uint32_t s = scale_byte<FORMAT>(top[k]);
          const float c = v[k] * scale_inverse(s == 255u ? 127u : s), hi = __shfl_down_sync(0xFFFFFFFFu, c, 1);
          if (g >= groups) continue;
          if (lane == 0) q.scales[entry * groups + g] = static_cast<uint8_t>(s);
          if constexpr (FORMAT == CSA_CACHE_E4M3) {
            q.data[entry * p.d + col] = static_cast<uint8_t>(float2_to_e4m3x2(c, 0.f) & 0xFFu);
          } else {
            if (lane % 2 == 0) q.data[entry * (p.d / 2) + col / 2] = static_cast<uint8_t>(float2_to_e2m1x2(c, hi));
          }
        }
      }
    }
    __syncwarp();
  }
}

// A warp's run of heads (of less than 2^31, as RopeRun; counted without a sign, since the last step may pass that): this
// lane's row and head, and where its x begins, moving on by the warp's groups with additions alone.
template <typename T>
struct AppendRun {
  unsigned u, end, row, head;  // unit of this lane's group, end of the warp's run
  const T* x;
  int groups, step_rows, step_heads;
  int64_t step, wrap;
  __device__ __forceinline__ AppendRun(const AppendParams& q, int group, int n) : groups(n) {
    const RopeParams& p = q.r;
    const int w = blockIdx.x * kRopeWarps + (threadIdx.x >> 5);
    u = static_cast<unsigned>(w * q.each + min(w, q.more));
    end = u + q.each + (w < q.more ? 1 : 0);
    u += group;
    row = p.heads == 1 ? u : u / p.heads;
    head = u - row * p.heads;
    step_rows = p.heads == 1 ? groups : groups / p.heads;
    step_heads = groups - step_rows * p.heads;
    x = static_cast<const T*>(p.x) + row * p.x_row + head * p.x_head;
    step = step_rows * p.x_row + step_heads * p.x_head;
    wrap = p.x_row - p.heads * p.x_head;
  }
  __device__ __forceinline__ void next(const RopeParams& p) {
    u += groups;
    row += step_rows;
    head += step_heads;
    x += step;
    if (head >= static_cast<unsigned>(p.heads)) {
      head -= p.heads;
      ++row;
      x += wrap;
    }
  }
};

// Vector kernel: lanes, pieces and runs as in the norm and rotation's. A scale belongs to four
// pieces of 8 columns, which the rotation's pairing leaves with any lanes; the pieces' largest
// magnitudes meet in shared memory, 4 bytes a piece, and each lane reads its group's four at once.
// Bound by instructions (24571 entries of 512 into e4m3), so what a lane has is told apart as little as can be: FULL,
// every lane has all its pieces.
template <int DTYPE, int PP, int FORMAT, bool FULL>
__global__ void __launch_bounds__(kRopeThreads, PP == 1 && DTYPE != CSA_DTYPE_FP32 ? 3 : 2)
    append_vec_kernel(const __grid_constant__ AppendParams q) {
  using T = typename Element<DTYPE>::T;
  __shared__ __align__(16) float s_w[CSA_MAX_HEAD_DIM];
  __shared__ __align__(16) uint32_t s_top[kRopeWarps][64 * PP];
  __shared__ __align__(16) float2 s_turn[kRopeWarps][256 * PP];  // cos and sin of each group's row, pair by pair
  const RopeParams& p = q.r;
  RopeLane<DTYPE, PP> L(p);
  uint32_t* const top = s_top[threadIdx.x >> 5] + L.group * (p.d / 8);
  pdl_wait();
  stage_weight(p, s_w);
  const float inv_d = 1.f / static_cast<float>(p.d);
  AppendRun<T> run(q, L.group, L.groups);
  unsigned base = run.u - L.group;  // the warp's first unit: all its lanes leave the loop together
  RopePieces<DTYPE, PP> cur{}, nxt{};  // (pieces that a lane does not have stay 0)
  int32_t pos = -1, pos_n = -1;
  int64_t slot = -1, slot_n = -1;
  auto fetch = [&](RopePieces<DTYPE, PP>& v, int32_t& ps, int64_t& at) {
    ps = -1;
    at = -1;
    if (run.u < run.end) {
      ps = p.pos != nullptr ? __ldg(p.pos + run.row) : 0;
      at = __ldg(q.slots + run.row);
#pragma unroll
      for (int s = 0; s < PP; ++s) {
        if (FULL || L.a[s] >= 0) v.a[s].load(run.x + L.a[s]);
        if (FULL || L.b[s] >= 0) v.b[s].load(run.x + L.b[s]);
      }
    }
  };
  fetch(cur, pos, slot);
  unsigned turned = ~0u;
  for (; base < run.end; base += L.groups) {
    const unsigned row = run.row, head = run.head;
    run.next(p);
    fetch(nxt, pos_n, slot_n);
    const bool live = pos >= 0 && static_cast<uint64_t>(slot) < static_cast<uint64_t>(q.num_slots);
    if (pos >= 0 && slot >= q.num_slots && q.dev_error != nullptr) *q.dev_error = CSA_DEVERR_SLOT;
    float xa[PP][8], xb[PP][8];
    float ss = 0.f;
#pragma unroll
    for (int s = 0; s < PP; ++s) {
      cur.a[s].get(xa[s]);
      cur.b[s].get(xb[s]);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        ss = fmaf(xa[s][i], xa[s][i], ss);
        ss = fmaf(xb[s][i], xb[s][i], ss);
      }
    }
    // A row's angles are worked out by all lanes of its heads in the warp, whichever turn columns by them (with 64 of
    // 512 columns turned, four at a time in eight lanes took as long as the rest; 22706 rows of 2 heads of 128,
    // put in and read back: 12.8 us, 14.1 where each head's lanes worked out all of them).
    if (p.rot > 0 && __any_sync(0xFFFFFFFFu, live && row != turned)) {
      const int h = static_cast<int>(head), g0 = max(0, L.group - h), g1 = L.group + min(L.groups - L.group, p.heads - h);
      const int32_t at = __shfl_sync(0xFFFFFFFFu, pos, g0 * p.lanes);  // (the first of them is there if any is)
      float2* turn = s_turn[threadIdx.x >> 5] + g0 * (p.rot / 2);
      for (int i = L.lane - g0 * p.lanes; i < p.rot / 2; i += (g1 - g0) * p.lanes) {
        float c, n;
        quarter_cos_sin(at, __ldg(p.turns + i), p.amp, c, n);
        turn[i] = make_float2(c, n);
      }
      __syncwarp();
      L.read_turns(p, turn);
      turned = row;
      __syncwarp();
    }
    if (p.norm) {
      const float r = rsqrtf(fmaf(L.sum(p, ss), inv_d, p.eps));
#pragma unroll
      for (int s = 0; s < PP; ++s) {
        float w[8];
        read_weight(s_w, FULL ? L.a[s] : max(L.a[s], 0), w);
#pragma unroll
        for (int i = 0; i < 8; ++i) xa[s][i] = xa[s][i] * r * w[i];
        read_weight(s_w, FULL ? L.b[s] : max(L.b[s], 0), w);
#pragma unroll
        for (int i = 0; i < 8; ++i) xb[s][i] = xb[s][i] * r * w[i];
      }
    }
#pragma unroll
    for (int s = 0; s < PP; ++s) {
      auto turn_pair = [](float& u, float& v, float c, float n) {
        const float w = u * c - v * n;
        v = u * n + v * c;
        u = w;
      };
      if (!p.interleaved) {
        if (L.ia[s] >= 0)
#pragma unroll
          for (int i = 0; i < 8; ++i) turn_pair(xa[s][i], xb[s][i], L.cs[s][i], L.sn[s][i]);
        continue;
      }
      if (L.ia[s] >= 0)
#pragma unroll
        for (int i = 0; i < 4; ++i) turn_pair(xa[s][2 * i], xa[s][2 * i + 1], L.cs[s][i], L.sn[s][i]);
      if (L.ib[s] >= 0)
#pragma unroll
        for (int i = 0; i < 4; ++i) turn_pair(xb[s][2 * i], xb[s][2 * i + 1], L.cs[s][4 + i], L.sn[s][4 + i]);
    }
    const int64_t entry = slot * p.heads + head;
    if constexpr (FORMAT == CSA_CACHE_BF16) {
      uint16_t* y = reinterpret_cast<uint16_t*>(q.data) + entry * p.d;
#pragma unroll
      for (int s = 0; s < PP; ++s) {
        Eight<CSA_DTYPE_BF16> o;
        o.set(xa[s]);
        if (live && (FULL || L.a[s] >= 0)) o.store(y + L.a[s]);
        o.set(xb[s]);
        if (live && (FULL || L.b[s] >= 0)) o.store(y + L.b[s]);
      }
    } else {
      auto largest = [](const float (&v)[8]) {  // (NaN if one is)
        const float a = max_magnitude(v[0], v[1], v[2]), b = max_magnitude(v[3], v[4], v[5]);
        return __float_as_uint(max_magnitude(max_magnitude(a, b, v[6]), v[7], v[7])) & 0x7FFFFFFFu;
      };
#pragma unroll
      for (int s = 0; s < PP; ++s) {
        if (FULL || L.a[s] >= 0) top[L.a[s] >> 3] = largest(xa[s]);
        if (FULL || L.b[s] >= 0) top[L.b[s] >> 3] = largest(xb[s]);
      }
      __syncwarp();
      uint8_t* const data = q.data + entry * (FORMAT == CSA_CACHE_E4M3 ? p.d : p.d / 2);
      uint8_t* const scales = q.scales + entry * (p.d / CSA_CACHE_GROUP);
      auto put = [&](int col, const float (&v)[8]) {
        if (!FULL && col < 0) return;
        const uint4 g = *reinterpret_cast<const uint4*>(top + (col >> 5) * 4);
        const uint32_t k = scale_byte<FORMAT>(max(max(g.x, g.y), max(g.z, g.w)));
        const float inv = scale_inverse(k == 255u ? 127u : k);
        if constexpr (FORMAT == CSA_CACHE_E4M3) {
          uint2 w;
          w.x = float2_to_e4m3x2(v[0] * inv, v[1] * inv) | (static_cast<uint32_t>(float2_to_e4m3x2(v[2] * inv, v[3] * inv)) << 16);
          w.y = float2_to_e4m3x2(v[4] * inv, v[5] * inv) | (static_cast<uint32_t>(float2_to_e4m3x2(v[6] * inv, v[7] * inv)) << 16);
          if (live) *reinterpret_cast<uint2*>(data + col) = w;
        } else {
          const uint32_t w = float2_to_e2m1x2(v[0] * inv, v[1] * inv) | (float2_to_e2m1x2(v[2] * inv, v[3] * inv) << 8) |
                             (float2_to_e2m1x2(v[4] * inv, v[5] * inv) << 16) | (float2_to_e2m1x2(v[6] * inv, v[7] * inv) << 24);
          if (live) *reinterpret_cast<uint32_t*>(data + col / 2) = w;
        }
        if (live && (col & 31) == 0) scales[col >> 5] = static_cast<uint8_t>(k);
      };
#pragma unroll
      for (int s = 0; s < PP; ++s) {
        put(L.a[s], xa[s]);
        put(L.b[s], xb[s]);
      }
      __syncwarp();
    }
    cur = nxt;
    pos = pos_n;
    slot = slot_n;
  }
}

template <typename F>
auto by_format(int format, F f) {
  return format == CSA_CACHE_BF16   ? f(std::integral_constant<int, CSA_CACHE_BF16>{})
         : format == CSA_CACHE_E4M3 ? f(std::integral_constant<int, CSA_CACHE_E4M3>{})
                                    : f(std::integral_constant<int, CSA_CACHE_E2M1>{});
}

}  // namespace
}  // namespace csa

using namespace csa;

extern "C" csa_status_t csa_cache_append(const void* x, int32_t dtype, int64_t rows, int32_t heads,
                                         int32_t d, int64_t x_row_stride, int64_t x_head_stride,
                                         const float* weight, int32_t norm, float eps,
                                         const int32_t* positions, const uint64_t* turns,
                                         int32_t rot_dim, int32_t rot_start, int32_t layout,
                                         float amplitude, const int64_t* slots, int64_t num_slots,
                                         int32_t format, void* data, uint8_t* scales,
                                         int32_t* dev_error, csa_stream_t stream) {
  const csa_status_t st = check_rope(dtype, rows, heads, d, weight, norm, eps, positions, turns, rot_dim,
                                     rot_start, layout);
  if (st != CSA_OK) return st;
  if (x_row_stride < 0 || x_head_stride < 0 || num_slots < 0) return CSA_ERR_INVALID_VALUE;
  if (format < CSA_CACHE_BF16 || format > CSA_CACHE_E2M1) return CSA_ERR_UNSUPPORTED;
  if (format != CSA_CACHE_BF16 && d % CSA_CACHE_GROUP != 0) return CSA_ERR_UNSUPPORTED;
  if (num_slots > INT64_MAX / 64 / (static_cast<int64_t>(heads) * d)) return CSA_ERR_UNSUPPORTED;
  if (!is_aligned(x, dtype_size(dtype)) || !is_aligned(slots, 8) || !is_aligned(dev_error, 4) ||
      (format == CSA_CACHE_BF16 && !is_aligned(data, 2)))
    return CSA_ERR_INVALID_VALUE;
  if (rows > 0 && (x == nullptr || slots == nullptr)) return CSA_ERR_INVALID_VALUE;
  if (num_slots > 0 && (data == nullptr || (format != CSA_CACHE_BF16 && scales == nullptr)))
    return CSA_ERR_INVALID_VALUE;
  if (rows == 0) return CSA_OK;
  AppendParams p{};
  p.r = rope_params(rows, heads, d, weight, norm, eps, positions, turns, rot_dim, rot_start, layout, amplitude);
  p.r.x = x;
  p.r.x_row = x_row_stride;
  p.r.x_head = x_head_stride;
  p.r.lanes = vector_lanes(p.r, dtype, x, data, nullptr);
  p.data = static_cast<uint8_t*>(data);
  p.scales = scales;
  p.slots = slots;
  p.num_slots = num_slots;
  p.dev_error = dev_error;
  const bool wide = vector_pairs(p.r) == 2, full = d / 8 == 2 * p.r.lanes;
  const void* k = by_dtype(dtype, [&](auto t) {
    return by_format(format, [&](auto f) {
      constexpr int T = decltype(t)::value, F = decltype(f)::value;
      return p.r.lanes == 0 ? reinterpret_cast<const void*>(append_scalar_kernel<T, F>)
             : wide         ? reinterpret_cast<const void*>(append_vec_kernel<T, 2, F, false>)
             : full         ? reinterpret_cast<const void*>(append_vec_kernel<T, 1, F, true>)
                            : reinterpret_cast<const void*>(append_vec_kernel<T, 1, F, false>);
    });
  });
  // one run of heads a resident warp
  const size_t smem = p.r.lanes == 0 ? sizeof(float) * kRopeWarps * d : 0;
  int dev = 0, sms = 0, bps = 0;
  if (note(cudaGetDevice(&dev)) != cudaSuccess || device_sms(dev, &sms) != cudaSuccess ||
      blocks_per_sm(dev, k, kRopeThreads, smem, &bps) != cudaSuccess)
    return CSA_ERR_CUDA;
  const int64_t per = kRopeWarps * (p.r.lanes == 0 ? 1 : 32 / p.r.lanes), most = static_cast<int64_t>(sms) * bps;
  int64_t blocks = (p.r.units + per - 1) / per;
  if (blocks > most) blocks = most;
  p.each = static_cast<int>(p.r.units / (blocks * kRopeWarps));
  p.more = static_cast<int>(p.r.units - p.each * blocks * kRopeWarps);
  void* args[] = {&p};
  return launch_pdl(k, dim3(static_cast<unsigned>(blocks)), dim3(kRopeThreads), smem,
                    reinterpret_cast<cudaStream_t>(stream), args) == cudaSuccess
             ? CSA_OK
             : CSA_ERR_CUDA;
}
