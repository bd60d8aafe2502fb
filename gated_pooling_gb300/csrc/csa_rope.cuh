// csa_rope.cuh -- what the kernels of the head norm and rotation share with those that go on from its
// result: the call's parameters and checks, angles, and a lane's pieces of a head.
//
// Angles: a pair turns by positions[r] * turns[i] in units of 2^-64 of a full turn, an
// integer product modulo 2^64. Its upper 32 bits, taken as a signed number, are the angle
// within half a turn either way, to 2^-32 of a turn, whatever the position (turns[i] is the nearest
// whole number, so a position below 2^31 is off by 2^-34 of a turn from it); only then does
// it become a float. No position loses precision, and no 64-bit floating point is needed.
#pragma once

#include <climits>
#include <cmath>
#include <cstdint>

#include "csa_compressor.h"
#include "csa_element.cuh"

namespace csa {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeWarps = kRopeThreads / 32;

struct RopeParams {
  const void* x;
  const void* dy;  // backward
  void* y;         // backward: dx
  const float* weight;
  const int32_t* pos;
  const uint64_t* turns;
  float* partial;  // backward: [gridDim.x, d]
  int64_t x_row, x_head, dy_row, dy_head, y_row, y_head;
  int64_t units;  // rows * heads
  int heads, d, rot, start;
  int norm, interleaved;
  int lanes;  // vector kernels: lanes of a row's head (a power of two)
  float eps, amp;
};

// cos and sin of a turn, times amp.
__device__ __forceinline__ void turn_cos_sin(int32_t pos, uint64_t per, float amp, float& c, float& s) {
  const uint64_t t = static_cast<uint64_t>(static_cast<int64_t>(pos)) * per;
  const float half_turns = static_cast<float>(static_cast<int32_t>(t >> 32)) * 0x1p-31f;
  sincospif(half_turns, &s, &c);
  c *= amp;
  s *= amp;
}

// 16-bit types take cos and sin from the hardware approximation (within 2^-21 of the value at
// an angle already brought to half a turn either way: 2^-9 and 2^-12 of a result are
// rounded away behind it); fp32 from CUDA's functions.
template <int DTYPE>
__device__ __forceinline__ void cos_sin(int32_t pos, uint64_t per, float amp, float& c, float& s) {
  if constexpr (DTYPE == CSA_DTYPE_FP32) {
    turn_cos_sin(pos, per, amp, c, s);
  } else {
    const uint64_t t = static_cast<uint64_t>(static_cast<int64_t>(pos)) * per;
    const float x = static_cast<float>(static_cast<int32_t>(t >> 32)) * 1.46291807926715968105e-9f;  // pi 2^-31
    c = __cosf(x) * amp;
    s = __sinf(x) * amp;
  }
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

// Columns of pair i of the rotated part.
__device__ __forceinline__ void pair_columns(const RopeParams& p, int i, int& a, int& b) {
  a = p.start + (p.interleaved ? 2 * i : i);
  b = a + (p.interleaved ? 1 : p.rot / 2);
}
// Column of the j-th column outside the rotated part.
__device__ __forceinline__ int other_column(const RopeParams& p, int j) {
  return j < p.start ? j : j + p.rot;
}

// ---------------------------------------------------------------------------------
// Vector kernels: d, strides and the rotated part in pieces of 8 columns.
//
// A lane owns PP pairs of pieces: with the half layout a rotated pair's two pieces hold the
// members of 8 column pairs, so no value changes lanes; all other pieces are paired by
// distance, so that neighbouring lanes read neighbouring pieces. `lanes` (up to 32) lanes
// share a row's head, 32 / lanes heads go through a warp at once, and a warp takes a run of
// consecutive heads and rows, so the angles of a row serve all its heads. The next head's
// pieces are loaded while one is computed. Three blocks an SM forward (two or four: 57.6 or
// 55.3 us instead of 51.5 for 8192 rows of 64 heads of 128, 5.2 TB/s), two backward (one:
// 67.9 us instead of 48.1 for 32 heads, 4.2 TB/s).
// ---------------------------------------------------------------------------------
template <int DTYPE, int PP>
struct RopeLane {
  int a[PP], b[PP];        // first columns of the pair's pieces, -1: none
  int ia[PP], ib[PP];      // first turns of their 8 (half) or 4 + 4 (interleaved) pairs, -1: not rotated
  float cs[PP][8], sn[PP][8];
  int lane, sub, group, groups;

  __device__ __forceinline__ explicit RopeLane(const RopeParams& p) {
    lane = threadIdx.x & 31;
    sub = lane & (p.lanes - 1);
    group = lane / p.lanes;
    groups = 32 / p.lanes;
    const int n = p.d / 8, s0 = p.start / 8, nr = p.rot / 8;
#pragma unroll
    for (int s = 0; s < PP; ++s) {
      const int k = sub + 32 * s;
      ia[s] = ib[s] = -1;
      int ca, cb;
      if (p.interleaved) {
        const int h = (n + 1) / 2;
        ca = k < h ? k : -1;
        cb = k < h && k + h < n ? k + h : -1;
        if (ca >= s0 && ca < s0 + nr) ia[s] = (ca - s0) * 4;
        if (cb >= s0 && cb < s0 + nr) ib[s] = (cb - s0) * 4;
      } else if (k < nr / 2) {
        ca = s0 + k;
        cb = ca + nr / 2;
        ia[s] = k * 8;
      } else {
        const int m = n - nr, h = (m + 1) / 2, j = k - nr / 2;
        ca = j < h ? j : -1;
        cb = j < h && j + h < m ? j + h : -1;
        if (ca >= s0) ca += nr;
        if (cb >= s0) cb += nr;
      }
      a[s] = ca < 0 ? -1 : ca * 8;
      b[s] = cb < 0 ? -1 : cb * 8;
    }
  }

  // the angles of a row
  __device__ __forceinline__ void turn_to(const RopeParams& p, int32_t pos) {
#pragma unroll
    for (int s = 0; s < PP; ++s) {
      if (ia[s] < 0 && ib[s] < 0) continue;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int i0 = h == 0 ? ia[s] : (p.interleaved ? ib[s] : ia[s] + 4);
        if (i0 < 0) continue;
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
          const ulonglong2 per = __ldg(reinterpret_cast<const ulonglong2*>(p.turns + i0 + i));
          cos_sin<DTYPE>(pos, per.x, p.amp, cs[s][4 * h + i], sn[s][4 * h + i]);
          cos_sin<DTYPE>(pos, per.y, p.amp, cs[s][4 * h + i + 1], sn[s][4 * h + i + 1]);
        }
      }
    }
  }
  // the same from a list of each pair's cos and sin
  __device__ __forceinline__ void read_turns(const RopeParams& p, const float2* list) {
#pragma unroll
    for (int s = 0; s < PP; ++s) {
      if (ia[s] < 0 && ib[s] < 0) continue;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int i0 = h == 0 ? ia[s] : (p.interleaved ? ib[s] : ia[s] + 4);
        if (i0 < 0) continue;
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
          const float4 v = *reinterpret_cast<const float4*>(list + i0 + i);
          cs[s][4 * h + i] = v.x;
          sn[s][4 * h + i] = v.y;
          cs[s][4 * h + i + 1] = v.z;
          sn[s][4 * h + i + 1] = v.w;
        }
      }
    }
  }
  // the pair's values turned, or turned back
  template <bool BACK>
  __device__ __forceinline__ void turn(const RopeParams& p, int s, float (&x)[8], float (&y)[8]) const {
    auto two = [&](float& u, float& v, float c, float n) {
      if (BACK) n = -n;
      const float w = u * c - v * n;
      v = u * n + v * c;
      u = w;
    };
    if (p.interleaved) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (ia[s] >= 0) two(x[2 * i], x[2 * i + 1], cs[s][i], sn[s][i]);
        if (ib[s] >= 0) two(y[2 * i], y[2 * i + 1], cs[s][4 + i], sn[s][4 + i]);
      }
    } else if (ia[s] >= 0) {
#pragma unroll
      for (int i = 0; i < 8; ++i) two(x[i], y[i], cs[s][i], sn[s][i]);
    }
  }
  // sum over the head's lanes
  __device__ __forceinline__ float sum(const RopeParams& p, float v) const {
    for (int o = p.lanes / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
  }
};

// A warp's run of heads: this lane's row and head, moving on by the warp's groups.
struct RopeRun {
  int64_t u, end;  // unit of this lane's group, end of the warp's run
  int64_t row;
  int head, step_rows, step_heads;
  __device__ __forceinline__ RopeRun(const RopeParams& p, int group, int groups) {
    const int64_t warps = static_cast<int64_t>(gridDim.x) * kRopeWarps;
    const int64_t w = static_cast<int64_t>(blockIdx.x) * kRopeWarps + (threadIdx.x >> 5);
    u = p.units * w / warps;
    end = p.units * (w + 1) / warps;
    u += group;
    row = u / p.heads;
    head = static_cast<int>(u - row * p.heads);
    step_rows = groups / p.heads;
    step_heads = groups - step_rows * p.heads;
  }
  __device__ __forceinline__ bool valid() const { return u < end; }
  __device__ __forceinline__ void next(const RopeParams& p, int groups) {
    u += groups;
    row += step_rows;
    head += step_heads;
    if (head >= p.heads) {
      head -= p.heads;
      ++row;
    }
  }
};

// This lane's pieces of a row's head.
template <int DTYPE, int PP>
struct RopePieces {
  Eight<DTYPE> a[PP], b[PP];
  __device__ __forceinline__ void load(const RopeLane<DTYPE, PP>& L, const void* x, int64_t at) {
    const typename Element<DTYPE>::T* q = static_cast<const typename Element<DTYPE>::T*>(x) + at;
#pragma unroll
    for (int s = 0; s < PP; ++s) {
      if (L.a[s] >= 0) a[s].load(q + L.a[s]);
      if (L.b[s] >= 0) b[s].load(q + L.b[s]);
    }
  }
};

// The weight in shared memory (ones without one): kept there rather than in a lane's registers,
// which hold the heads on their way.
__device__ __forceinline__ void stage_weight(const RopeParams& p, float* s_w) {
  if (!p.norm) return;
  for (int c = threadIdx.x; c < p.d; c += kRopeThreads) s_w[c] = p.weight != nullptr ? __ldg(p.weight + c) : 1.f;
  __syncthreads();
}
__device__ __forceinline__ void read_weight(const float* s_w, int col, float (&w)[8]) {
  const float4 u = *reinterpret_cast<const float4*>(s_w + col), v = *reinterpret_cast<const float4*>(s_w + col + 4);
  w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w;
  w[4] = v.x, w[5] = v.y, w[6] = v.z, w[7] = v.w;
}

// Lanes of a row's head, or 0 where the vector kernels do not take the call.
inline int vector_lanes(const RopeParams& p, int dtype, const void* x, const void* y, const void* z) {
  const bool fits = p.d % 8 == 0 && p.start % 8 == 0 && p.rot % (p.interleaved ? 8 : 16) == 0 &&
                    p.x_row % 8 == 0 && p.x_head % 8 == 0 && p.y_row % 8 == 0 && p.y_head % 8 == 0 &&
                    p.dy_row % 8 == 0 && p.dy_head % 8 == 0 && is_aligned(x, 16) && is_aligned(y, 16) &&
                    is_aligned(z, 16) && is_aligned(p.weight, 16) && is_aligned(p.turns, 16);
  if (!fits) return 0;
  const int n = p.d / 8;
  // pairs of pieces: the half layout's rotated pieces pair among themselves
  const int pairs = p.interleaved ? (n + 1) / 2 : p.rot / 16 + (n - p.rot / 8 + 1) / 2;
  int lanes = 1;
  while (lanes < 32 && lanes < pairs) lanes *= 2;
  return lanes;
}
// Pairs of pieces a lane holds: one up to d = 512.
inline int vector_pairs(const RopeParams& p) {
  const int n = p.d / 8;
  const int pairs = p.interleaved ? (n + 1) / 2 : p.rot / 16 + (n - p.rot / 8 + 1) / 2;
  return pairs <= 32 ? 1 : 2;
}

inline csa_status_t check_rope(int32_t dtype, int64_t rows, int32_t heads, int32_t d,
                        const float* weight, int32_t norm, float eps, const int32_t* positions,
                        const uint64_t* turns, int32_t rot_dim, int32_t rot_start, int32_t layout) {
  if (rows < 0 || heads < 1 || d < 1 || (norm != 0 && norm != 1) || rot_dim < 0 ||
      rot_dim % 2 != 0 || rot_start < 0 || !(eps >= 0.f) || std::isinf(eps))
    return CSA_ERR_INVALID_VALUE;
  if (d > CSA_MAX_HEAD_DIM || rows > INT_MAX / heads) return CSA_ERR_UNSUPPORTED;
  if (dtype < CSA_DTYPE_BF16 || dtype > CSA_DTYPE_FP32 ||
      (layout != CSA_ROPE_HALF && layout != CSA_ROPE_INTERLEAVED))
    return CSA_ERR_UNSUPPORTED;
  if (rot_dim > d || rot_start > d - rot_dim) return CSA_ERR_INVALID_VALUE;
  if (norm == 0 && weight != nullptr) return CSA_ERR_INVALID_VALUE;
  if (rot_dim > 0 && rows > 0 && (positions == nullptr || turns == nullptr))
    return CSA_ERR_INVALID_VALUE;
  if (!is_aligned(weight, 4) || !is_aligned(positions, 4) || !is_aligned(turns, 8))
    return CSA_ERR_INVALID_VALUE;
  return CSA_OK;
}

inline RopeParams rope_params(int64_t rows, int32_t heads, int32_t d, const float* weight, int32_t norm,
                       float eps, const int32_t* positions, const uint64_t* turns, int32_t rot_dim,
                       int32_t rot_start, int32_t layout, float amplitude) {
  RopeParams p{};
  p.weight = weight;
  p.pos = positions;
  p.turns = turns;
  p.units = rows * heads;
  p.heads = heads;
  p.d = d;
  p.rot = rot_dim;
  p.start = rot_start;
  p.norm = norm;
  p.interleaved = layout == CSA_ROPE_INTERLEAVED;
  p.eps = eps;
  p.amp = amplitude;
  return p;
}

}  // namespace
}  // namespace csa
