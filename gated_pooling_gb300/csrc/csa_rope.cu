// csa_rope.cu -- head norm and rotation in one pass, forward and backward (the interface and
// the formulas are in csa_compressor.h).
//
// A row's head is read once, its mean square taken in fp32, and the columns written back
// normed and turned; backward, x and dy are read once and dx written. Bound by HBM bytes.
//
// Angles: a pair turns by positions[r] * turns[i] in units of 2^-64 of a full turn, an
// integer product modulo 2^64. Its upper 32 bits, taken as a signed number, are the angle
// within half a turn either way, to 2^-32 of a turn, whatever the position (turns[i] is the nearest
// whole number, so a position below 2^31 is off by 2^-34 of a turn from it); only then does
// it become a float. No position loses precision, and no 64-bit floating point is needed.
#include <cmath>
#include <climits>
#include <cstdint>
#include <type_traits>

#include "csa_compressor.h"
#include "csa_element.cuh"
#include "csa_internal.h"

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

// Scalar kernel, any d and alignment: a warp per row and head. Each lane takes whole pairs
// and the columns outside the rotated part, reads both of a pair before it writes them (so
// y may be x), and the backward's dweight sums stay with the lane that owns the column.
template <int DTYPE>
__global__ void __launch_bounds__(kRopeThreads) rope_scalar_kernel(RopeParams p) {
  using E = Element<DTYPE>;
  using T = typename E::T;
  const int lane = threadIdx.x & 31;
  pdl_wait();
  for (int64_t u = static_cast<int64_t>(blockIdx.x) * kRopeWarps + (threadIdx.x >> 5); u < p.units;
       u += static_cast<int64_t>(gridDim.x) * kRopeWarps) {
    const int64_t row = static_cast<int>(u) / p.heads, head = u - row * p.heads;  // (units below 2^31)
    // (the position, the row and the first angle load side by side)
    const int32_t pos = p.pos != nullptr ? __ldg(p.pos + row) : 0;
    const uint64_t per0 = lane < p.rot / 2 ? __ldg(p.turns + lane) : 0;
    const T* x = static_cast<const T*>(p.x) + row * p.x_row + head * p.x_head;
    T* y = static_cast<T*>(p.y) + row * p.y_row + head * p.y_head;
    float r = 1.f;
    if (p.norm) {
      float ss = 0.f;
      for (int c = lane; c < p.d; c += 32) {
        const float v = E::to_float(x[c]);
        ss = fmaf(v, v, ss);
      }
      r = 1.f / sqrtf(warp_sum(ss) / static_cast<float>(p.d) + p.eps);
    }
    if (pos < 0) continue;
    auto normed = [&](int c) {
      const float v = E::to_float(x[c]);
      return p.norm ? (p.weight != nullptr ? v * r * p.weight[c] : v * r) : v;
    };
    for (int i = lane; i < p.rot / 2; i += 32) {
      int a, b;
      pair_columns(p, i, a, b);
      float cs, sn;
      cos_sin<DTYPE>(pos, i == lane ? per0 : __ldg(p.turns + i), p.amp, cs, sn);
      const float va = normed(a), vb = normed(b);
      y[a] = E::from_float(va * cs - vb * sn);
      y[b] = E::from_float(va * sn + vb * cs);
    }
    for (int j = lane; j < p.d - p.rot; j += 32) {
      const int c = other_column(p, j);
      y[c] = E::from_float(normed(c));
    }
  }
}

// Backward of the same. dweight: a warp adds its units' terms per column in shared memory
// (compensated fp32 sums), then the block adds its warps in order and writes one partial
// row; csa_api.cu's fixed-order reduction adds the rows.
template <int DTYPE>
__global__ void __launch_bounds__(kRopeThreads) rope_scalar_bwd_kernel(RopeParams p) {
  using E = Element<DTYPE>;
  using T = typename E::T;
  extern __shared__ float s_dw[];  // [warps][2][d]: sums and their compensation
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float* sum = s_dw + static_cast<size_t>(warp) * 2 * p.d;
  float* cmp = sum + p.d;
  if (p.partial != nullptr) {
    for (int c = threadIdx.x; c < kRopeWarps * 2 * p.d; c += kRopeThreads) s_dw[c] = 0.f;
    __syncthreads();
  }
  pdl_wait();
  for (int64_t u = static_cast<int64_t>(blockIdx.x) * kRopeWarps + warp; u < p.units;
       u += static_cast<int64_t>(gridDim.x) * kRopeWarps) {
    const int64_t row = static_cast<int>(u) / p.heads, head = u - row * p.heads;  // (units below 2^31)
    const int32_t pos = p.pos != nullptr ? p.pos[row] : 0;
    if (pos < 0) continue;
    const T* x = static_cast<const T*>(p.x) + row * p.x_row + head * p.x_head;
    const T* dy = static_cast<const T*>(p.dy) + row * p.dy_row + head * p.dy_head;
    T* dx = static_cast<T*>(p.y) + row * p.y_row + head * p.y_head;
    // f(column, gradient of n) for every column the lane owns; both of a pair are read
    // before either is handed on
    auto each = [&](auto f) {
      for (int i = lane; i < p.rot / 2; i += 32) {
        int a, b;
        pair_columns(p, i, a, b);
        float cs, sn;
        cos_sin<DTYPE>(pos, __ldg(p.turns + i), p.amp, cs, sn);
        const float ga = E::to_float(dy[a]), gb = E::to_float(dy[b]);
        f(a, ga * cs + gb * sn);
        f(b, gb * cs - ga * sn);
      }
      for (int j = lane; j < p.d - p.rot; j += 32) {
        const int c = other_column(p, j);
        f(c, E::to_float(dy[c]));
      }
    };
    if (!p.norm) {
      each([&](int c, float g) { dx[c] = E::from_float(g); });
      continue;
    }
    float ss = 0.f, dot = 0.f;
    each([&](int c, float g) {
      const float v = E::to_float(x[c]);
      ss = fmaf(v, v, ss);
      dot = fmaf(p.weight != nullptr ? g * p.weight[c] : g, v, dot);
    });
    const float n = static_cast<float>(p.d);
    const float r = 1.f / sqrtf(warp_sum(ss) / n + p.eps);
    const float k = warp_sum(dot) / n * r * r;  // mean(dn w xhat) * r
    each([&](int c, float g) {
      const float v = E::to_float(x[c]);
      if (p.partial != nullptr) {
        float s = sum[c], e = cmp[c];
        neumaier_add(s, e, g * (v * r));
        sum[c] = s;
        cmp[c] = e;
      }
      dx[c] = E::from_float(r * ((p.weight != nullptr ? g * p.weight[c] : g) - v * k));
    });
  }
  if (p.partial == nullptr) return;
  __syncthreads();
  for (int c = threadIdx.x; c < p.d; c += kRopeThreads) {
    float s = 0.f, e = 0.f;
    for (int w = 0; w < kRopeWarps; ++w) {
      neumaier_add(s, e, s_dw[static_cast<size_t>(w) * 2 * p.d + c]);
      neumaier_add(s, e, s_dw[static_cast<size_t>(w) * 2 * p.d + p.d + c]);
    }
    p.partial[static_cast<int64_t>(blockIdx.x) * p.d + c] = s + e;
  }
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

template <int DTYPE, int PP>
__global__ void __launch_bounds__(kRopeThreads, PP == 1 && DTYPE != CSA_DTYPE_FP32 ? 3 : 2)
    rope_vec_kernel(RopeParams p) {
  using T = typename Element<DTYPE>::T;
  __shared__ __align__(16) float s_w[CSA_MAX_HEAD_DIM];
  RopeLane<DTYPE, PP> L(p);
  pdl_wait();
  stage_weight(p, s_w);
  const float inv_d = 1.f / static_cast<float>(p.d);
  RopeRun run(p, L.group, L.groups);
  int64_t base = run.u - L.group;  // the warp's first unit: all its lanes leave the loop together
  RopePieces<DTYPE, PP> cur, nxt;
  int32_t pos = -1, pos_n = -1;
  auto fetch = [&](RopePieces<DTYPE, PP>& v, int32_t& ps) {
    ps = -1;
    if (run.valid()) {
      ps = p.pos != nullptr ? __ldg(p.pos + run.row) : 0;
      v.load(L, p.x, run.row * p.x_row + run.head * p.x_head);
    }
  };
  fetch(cur, pos);
  int64_t turned = -1;
  for (; base < run.end; base += L.groups) {
    const int64_t row = run.row;
    const int head = run.head;
    run.next(p, L.groups);
    fetch(nxt, pos_n);
    float xa[PP][8], xb[PP][8];
    float r = 1.f;
    float ss = 0.f;
#pragma unroll
    for (int s = 0; s < PP; ++s) {
      cur.a[s].get(xa[s]);
      cur.b[s].get(xb[s]);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (L.a[s] >= 0) ss = fmaf(xa[s][i], xa[s][i], ss);
        if (L.b[s] >= 0) ss = fmaf(xb[s][i], xb[s][i], ss);
      }
    }
    if (p.norm) r = rsqrtf(fmaf(L.sum(p, ss), inv_d, p.eps));
    if (pos >= 0) {
      if (row != turned) {
        L.turn_to(p, pos);
        turned = row;
      }
      T* y = static_cast<T*>(p.y) + row * p.y_row + head * p.y_head;
#pragma unroll
      for (int s = 0; s < PP; ++s) {
        if (p.norm) {
          float w[8];
          if (L.a[s] >= 0) {
            read_weight(s_w, L.a[s], w);
#pragma unroll
            for (int i = 0; i < 8; ++i) xa[s][i] = xa[s][i] * r * w[i];
          }
          if (L.b[s] >= 0) {
            read_weight(s_w, L.b[s], w);
#pragma unroll
            for (int i = 0; i < 8; ++i) xb[s][i] = xb[s][i] * r * w[i];
          }
        }
        L.template turn<false>(p, s, xa[s], xb[s]);
        Eight<DTYPE> o;
        if (L.a[s] >= 0) {
          o.set(xa[s]);
          o.store(y + L.a[s]);
        }
        if (L.b[s] >= 0) {
          o.set(xb[s]);
          o.store(y + L.b[s]);
        }
      }
    }
    cur = nxt;
    pos = pos_n;
  }
}

// Backward. dweight: a lane sums its columns over at most kDwRun heads in registers, then the
// warp's groups join them and add them to the warp's sums in shared memory; the block adds
// its warps in order and writes one partial row. No chain of plain additions is longer than
// kDwRun, or a warp's heads / (kDwRun * groups).
constexpr int kDwRun = 16;
template <int DTYPE, int PP>
__global__ void __launch_bounds__(kRopeThreads, PP == 1 ? 2 : 1) rope_vec_bwd_kernel(RopeParams p) {
  using T = typename Element<DTYPE>::T;
  extern __shared__ float s_dw[];  // [warps][d]
  __shared__ __align__(16) float s_w[CSA_MAX_HEAD_DIM];
  RopeLane<DTYPE, PP> L(p);
  float* sums = s_dw + (threadIdx.x >> 5) * p.d;
  if (p.partial != nullptr)
    for (int c = L.lane; c < p.d; c += 32) sums[c] = 0.f;
  __syncwarp();
  pdl_wait();
  stage_weight(p, s_w);
  float da[PP][8], db[PP][8];
#pragma unroll
  for (int s = 0; s < PP; ++s)
#pragma unroll
    for (int i = 0; i < 8; ++i) da[s][i] = db[s][i] = 0.f;
  auto flush = [&]() {
#pragma unroll
    for (int s = 0; s < PP; ++s)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float va = da[s][i], vb = db[s][i];
        for (int o = p.lanes; o < 32; o <<= 1) {
          va += __shfl_xor_sync(0xFFFFFFFFu, va, o);
          vb += __shfl_xor_sync(0xFFFFFFFFu, vb, o);
        }
        if (L.group == 0) {
          if (L.a[s] >= 0) sums[L.a[s] + i] += va;
          if (L.b[s] >= 0) sums[L.b[s] + i] += vb;
        }
        da[s][i] = db[s][i] = 0.f;
      }
  };
  const float inv_d = 1.f / static_cast<float>(p.d);
  RopeRun run(p, L.group, L.groups);
  int64_t base = run.u - L.group;
  RopePieces<DTYPE, PP> cx, cg, nx, ng;
  int32_t pos = -1, pos_n = -1;
  auto fetch = [&](RopePieces<DTYPE, PP>& vx, RopePieces<DTYPE, PP>& vg, int32_t& ps) {
    ps = -1;
    if (run.valid()) {
      ps = p.pos != nullptr ? __ldg(p.pos + run.row) : 0;
      if (p.norm) vx.load(L, p.x, run.row * p.x_row + run.head * p.x_head);
      vg.load(L, p.dy, run.row * p.dy_row + run.head * p.dy_head);
    }
  };
  fetch(cx, cg, pos);
  int64_t turned = -1;
  int since = 0;
  for (; base < run.end; base += L.groups) {
    const int64_t row = run.row;
    const int head = run.head;
    run.next(p, L.groups);
    fetch(nx, ng, pos_n);
    if (pos >= 0 && row != turned) {
      L.turn_to(p, pos);
      turned = row;
    }
    float ga[PP][8], gb[PP][8], xa[PP][8], xb[PP][8];
    float ss = 0.f, dot = 0.f;
#pragma unroll
    for (int s = 0; s < PP; ++s) {
      cg.a[s].get(ga[s]);
      cg.b[s].get(gb[s]);
      if (pos >= 0) L.template turn<true>(p, s, ga[s], gb[s]);
      if (p.norm) {
        cx.a[s].get(xa[s]);
        cx.b[s].get(xb[s]);
        float w[8];
        if (L.a[s] >= 0) {
          read_weight(s_w, L.a[s], w);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            ss = fmaf(xa[s][i], xa[s][i], ss);
            dot = fmaf(ga[s][i] * w[i], xa[s][i], dot);
          }
        }
        if (L.b[s] >= 0) {
          read_weight(s_w, L.b[s], w);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            ss = fmaf(xb[s][i], xb[s][i], ss);
            dot = fmaf(gb[s][i] * w[i], xb[s][i], dot);
          }
        }
      }
    }
    if (p.norm) {
      const float r = rsqrtf(fmaf(L.sum(p, ss), inv_d, p.eps));
      const float k = L.sum(p, dot) * inv_d * r * r;
      if (pos >= 0) {
#pragma unroll
        for (int s = 0; s < PP; ++s) {
          float w[8];
          if (L.a[s] >= 0) {
            read_weight(s_w, L.a[s], w);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              da[s][i] = fmaf(ga[s][i], xa[s][i] * r, da[s][i]);
              ga[s][i] = r * (ga[s][i] * w[i] - xa[s][i] * k);
            }
          }
          if (L.b[s] >= 0) {
            read_weight(s_w, L.b[s], w);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              db[s][i] = fmaf(gb[s][i], xb[s][i] * r, db[s][i]);
              gb[s][i] = r * (gb[s][i] * w[i] - xb[s][i] * k);
            }
          }
        }
      }
    }
    if (pos >= 0) {
      T* dx = static_cast<T*>(p.y) + row * p.y_row + head * p.y_head;
#pragma unroll
      for (int s = 0; s < PP; ++s) {
        Eight<DTYPE> o;
        if (L.a[s] >= 0) {
          o.set(ga[s]);
          o.store(dx + L.a[s]);
        }
        if (L.b[s] >= 0) {
          o.set(gb[s]);
          o.store(dx + L.b[s]);
        }
      }
    }
    cx = nx;
    cg = ng;
    pos = pos_n;
    if (p.partial != nullptr && ++since == kDwRun) {
      flush();
      since = 0;
    }
  }
  if (p.partial == nullptr) return;
  flush();
  __syncthreads();
  for (int c = threadIdx.x; c < p.d; c += kRopeThreads) {
    float s = 0.f, e = 0.f;
    for (int w = 0; w < kRopeWarps; ++w) neumaier_add(s, e, s_dw[w * p.d + c]);
    p.partial[static_cast<int64_t>(blockIdx.x) * p.d + c] = s + e;
  }
}

// Lanes of a row's head, or 0 where the vector kernels do not take the call.
int vector_lanes(const RopeParams& p, int dtype, const void* x, const void* y, const void* z) {
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
int vector_pairs(const RopeParams& p) {
  const int n = p.d / 8;
  const int pairs = p.interleaved ? (n + 1) / 2 : p.rot / 16 + (n - p.rot / 8 + 1) / 2;
  return pairs <= 32 ? 1 : 2;
}

// Blocks of the backward (= partial rows): enough to fill the GPU, at most one per warp's worth
// of units.
int64_t bwd_blocks(int64_t units, int sms) {
  const int64_t want = (units + kRopeWarps - 1) / kRopeWarps, most = 2 * static_cast<int64_t>(sms);
  return want < 1 ? 1 : (want < most ? want : most);
}

csa_status_t check_rope(int32_t dtype, int64_t rows, int32_t heads, int32_t d,
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

RopeParams rope_params(int64_t rows, int32_t heads, int32_t d, const float* weight, int32_t norm,
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

// Numbers as the unevaluated sum of two doubles, |lo| at most half a step of hi, for the table on the
// host: 64 bits of a turn are more than a double holds. Sums and products with the errors of their
// roundings as in Dekker (1971) and Knuth; each operation is within a few 2^-104. (volatile: no sum is
// contracted with the product before it, whatever the compiler's default.)
struct Twofold {
  double hi, lo;
};
constexpr Twofold kInvTwoPi{0x1.45f306dc9c883p-3, -0x1.6b01ec5417056p-57};
constexpr Twofold kLnTwo{0x1.62e42fefa39efp-1, 0x1.abc9e3b39803fp-56};
Twofold sum_of(double a, double b) {
  const volatile double s = a + b, v = s - a, u = s - v;
  const volatile double x = a - u, y = b - v;
  return {s, x + y};
}
Twofold plus(Twofold a, Twofold b) {
  const Twofold s = sum_of(a.hi, b.hi);
  const volatile double low = a.lo + b.lo;
  const Twofold t = sum_of(s.hi, s.lo + low);
  return t;
}
Twofold times(Twofold a, Twofold b) {
  const volatile double p = a.hi * b.hi, x = a.hi * b.lo, y = a.lo * b.hi;
  const volatile double e = std::fma(a.hi, b.hi, -p), c = x + y;
  return sum_of(p, e + c);
}
Twofold over(Twofold a, double b) {
  const volatile double q = a.hi / b;
  const Twofold back = times({q, 0.0}, {b, 0.0});
  const Twofold rest = plus(a, {-back.hi, -back.lo});
  return sum_of(q, rest.hi / b);
}
// e^x = the result times 2^*e: Taylor's series of the remainder's 256th part, squared eight times.
Twofold exp_of(Twofold x, int* e) {
  const double k = std::nearbyint(x.hi / kLnTwo.hi);
  const Twofold r = plus(x, times(kLnTwo, {-k, 0.0}));
  const Twofold y{r.hi / 256, r.lo / 256};
  Twofold s{1.0, 0.0};
  for (int n = 16; n > 0; --n) s = plus({1.0, 0.0}, times(over(y, n), s));
  for (int n = 0; n < 8; ++n) s = times(s, s);
  *e = static_cast<int>(k);
  return s;
}
// ln x of a double above 0: one step of Newton's method from the double's.
Twofold log_of(double x) {
  int e, k;
  const double m = std::frexp(x, &e), y = std::log(m);
  Twofold b = exp_of({-y, 0.0}, &k);
  b = {std::ldexp(b.hi, k), std::ldexp(b.lo, k)};
  const Twofold rest = plus(times(b, {m, 0.0}), {-1.0, 0.0});
  return plus(times(kLnTwo, {static_cast<double>(e), 0.0}), plus({y, 0.0}, rest));
}
// x 2^e, between 0 and 2^63, to the nearest whole number.
uint64_t nearest(Twofold x, int e) {
  const double hi = std::ldexp(x.hi, e), whole = std::nearbyint(hi);
  const volatile double left = hi - whole;
  return static_cast<uint64_t>(static_cast<int64_t>(whole) +
                               static_cast<int64_t>(std::nearbyint(left + std::ldexp(x.lo, e))));
}

}  // namespace
}  // namespace csa

using namespace csa;

extern "C" csa_status_t csa_rope_table(int32_t rot_dim, double base, int32_t scaling, double factor,
                                       double original_length, double beta_fast, double beta_slow,
                                       uint64_t* turns_host, float* amplitude) {
  if (rot_dim < 0 || rot_dim % 2 != 0 || !(base > 1.0) || std::isinf(base) ||
      (rot_dim > 0 && turns_host == nullptr))
    return CSA_ERR_INVALID_VALUE;
  if (rot_dim > CSA_MAX_HEAD_DIM || scaling < CSA_ROPE_PLAIN || scaling > CSA_ROPE_YARN)
    return CSA_ERR_UNSUPPORTED;
  if (scaling != CSA_ROPE_PLAIN && (!(factor >= 1.0) || std::isinf(factor))) return CSA_ERR_INVALID_VALUE;
  if (scaling == CSA_ROPE_YARN &&
      (!(original_length >= 1.0) || std::isinf(original_length) || !(beta_fast > 0.0) ||
       !(beta_slow > 0.0) || std::isinf(beta_fast) || std::isinf(beta_slow)))
    return CSA_ERR_INVALID_VALUE;
  const double two_pi = 6.283185307179586476925286766559;
  double lo = 0.0, span = 1.0;
  if (scaling == CSA_ROPE_YARN && rot_dim > 0) {
    auto at = [&](double beta) {
      return rot_dim * std::log(original_length / (two_pi * beta)) / (2.0 * std::log(base));
    };
    const double last = rot_dim - 1;
    lo = std::fmin(std::fmax(std::floor(at(beta_fast)), 0.0), last);
    const double hi = std::fmin(std::fmax(std::ceil(at(beta_slow)), 0.0), last);
    span = std::fmax(hi - lo, 0.001);
  }
  const Twofold one{1.0, 0.0}, log_base = log_of(base);
  for (int32_t i = 0; i < rot_dim / 2; ++i) {
    int e;
    Twofold f = exp_of(times(over(log_base, rot_dim), {-2.0 * i, 0.0}), &e);
    if (scaling == CSA_ROPE_LINEAR) f = over(f, factor);
    if (scaling == CSA_ROPE_YARN) {
      const Twofold m = i <= lo ? Twofold{0.0, 0.0} : i - lo >= span ? one : over({i - lo, 0.0}, span);
      f = plus(times(over(f, factor), m), times(f, plus(one, {-m.hi, -m.lo})));
    }
    turns_host[i] = nearest(times(f, kInvTwoPi), e + 64);
  }
  if (amplitude != nullptr)
    *amplitude = scaling == CSA_ROPE_YARN ? static_cast<float>(0.1 * std::log(factor) + 1.0) : 1.f;
  return CSA_OK;
}

extern "C" csa_status_t csa_norm_rope_fwd(const void* x, int32_t dtype, int64_t rows, int32_t heads,
                                          int32_t d, int64_t x_row_stride, int64_t x_head_stride,
                                          const float* weight, int32_t norm, float eps,
                                          const int32_t* positions, const uint64_t* turns,
                                          int32_t rot_dim, int32_t rot_start, int32_t layout,
                                          float amplitude, void* y, int64_t y_row_stride,
                                          int64_t y_head_stride, csa_stream_t stream) {
  csa_status_t st = check_rope(dtype, rows, heads, d, weight, norm, eps, positions, turns, rot_dim,
                               rot_start, layout);
  if (st != CSA_OK) return st;
  if (x_row_stride < 0 || x_head_stride < 0 || y_row_stride < 0 || y_head_stride < 0)
    return CSA_ERR_INVALID_VALUE;
  const uintptr_t size = dtype_size(dtype);
  if (!is_aligned(x, size) || !is_aligned(y, size)) return CSA_ERR_INVALID_VALUE;
  if (rows == 0) return CSA_OK;
  if (x == nullptr || y == nullptr || !separate(rows, heads, d, y_row_stride, y_head_stride))
    return CSA_ERR_INVALID_VALUE;
  RopeParams p = rope_params(rows, heads, d, weight, norm, eps, positions, turns, rot_dim, rot_start,
                             layout, amplitude);
  p.x = x;
  p.y = y;
  p.x_row = x_row_stride;
  p.x_head = x_head_stride;
  p.y_row = y_row_stride;
  p.y_head = y_head_stride;
  p.lanes = vector_lanes(p, dtype, x, y, nullptr);
  const bool wide = vector_pairs(p) == 2;
  const void* k = by_dtype(dtype, [&](auto t) {
    constexpr int T = decltype(t)::value;
    return p.lanes == 0 ? reinterpret_cast<const void*>(rope_scalar_kernel<T>)
           : wide       ? reinterpret_cast<const void*>(rope_vec_kernel<T, 2>)
                        : reinterpret_cast<const void*>(rope_vec_kernel<T, 1>);
  });
  int64_t blocks = (p.units + kRopeWarps - 1) / kRopeWarps;
  if (p.lanes != 0) {
    // one run of heads a resident warp
    int dev = 0, sms = 0, bps = 0;
    if (note(cudaGetDevice(&dev)) != cudaSuccess || device_sms(dev, &sms) != cudaSuccess ||
        blocks_per_sm(dev, k, kRopeThreads, 0, &bps) != cudaSuccess)
      return CSA_ERR_CUDA;
    const int64_t per = kRopeWarps * (32 / p.lanes), most = static_cast<int64_t>(sms) * bps;
    blocks = (p.units + per - 1) / per;
    if (blocks > most) blocks = most;
  }
  void* args[] = {&p};
  if (launch_pdl(k, dim3(static_cast<unsigned>(blocks)), dim3(kRopeThreads), 0,
                 reinterpret_cast<cudaStream_t>(stream), args) != cudaSuccess)
    return CSA_ERR_CUDA;
  return CSA_OK;
}

extern "C" size_t csa_norm_rope_bwd_workspace_bytes(int64_t rows, int32_t heads, int32_t d) {
  if (rows < 0 || heads < 1 || d < 1 || d > CSA_MAX_HEAD_DIM || rows > INT_MAX / heads) return 0;
  int dev = 0, sms = 0;
  if (note(cudaGetDevice(&dev)) != cudaSuccess || device_sms(dev, &sms) != cudaSuccess) return 0;
  return (static_cast<size_t>(bwd_blocks(rows * heads, sms)) * d * sizeof(float) + 15) &
         ~static_cast<size_t>(15);
}

extern "C" csa_status_t csa_norm_rope_bwd(
    const void* x, const void* dy, int32_t dtype, int64_t rows, int32_t heads, int32_t d,
    int64_t x_row_stride, int64_t x_head_stride, int64_t dy_row_stride, int64_t dy_head_stride,
    const float* weight, int32_t norm, float eps, const int32_t* positions, const uint64_t* turns,
    int32_t rot_dim, int32_t rot_start, int32_t layout, float amplitude, void* dx,
    int64_t dx_row_stride, int64_t dx_head_stride, float* dweight, int32_t accumulate_dweight,
    void* workspace, size_t workspace_bytes, csa_stream_t stream) {
  csa_status_t st = check_rope(dtype, rows, heads, d, weight, norm, eps, positions, turns, rot_dim,
                               rot_start, layout);
  if (st != CSA_OK) return st;
  if (x_row_stride < 0 || x_head_stride < 0 || dy_row_stride < 0 || dy_head_stride < 0 ||
      dx_row_stride < 0 || dx_head_stride < 0)
    return CSA_ERR_INVALID_VALUE;
  if (norm == 0 && dweight != nullptr) return CSA_ERR_INVALID_VALUE;
  const uintptr_t size = dtype_size(dtype);
  if (!is_aligned(x, size) || !is_aligned(dy, size) || !is_aligned(dx, size) ||
      !is_aligned(dweight, 4) || !is_aligned(workspace, 16))
    return CSA_ERR_INVALID_VALUE;
  if (rows > 0 && ((norm != 0 && x == nullptr) || dy == nullptr || dx == nullptr ||
                   !separate(rows, heads, d, dx_row_stride, dx_head_stride)))
    return CSA_ERR_INVALID_VALUE;
  if (rows == 0 && (dweight == nullptr || accumulate_dweight != 0)) return CSA_OK;
  // the smallest partial is one row: refused before the device is asked
  if (dweight != nullptr && (workspace == nullptr || workspace_bytes < sizeof(float) * d))
    return CSA_ERR_WORKSPACE;
  int dev = 0, sms = 0;
  if (note(cudaGetDevice(&dev)) != cudaSuccess || device_sms(dev, &sms) != cudaSuccess)
    return CSA_ERR_CUDA;
  RopeParams p = rope_params(rows, heads, d, weight, norm, eps, positions, turns, rot_dim, rot_start,
                             layout, amplitude);
  const int64_t blocks = bwd_blocks(p.units, sms);
  if (dweight != nullptr && workspace_bytes < static_cast<size_t>(blocks) * d * sizeof(float))
    return CSA_ERR_WORKSPACE;
  p.x = x;
  p.dy = dy;
  p.y = dx;
  p.x_row = x_row_stride;
  p.x_head = x_head_stride;
  p.dy_row = dy_row_stride;
  p.dy_head = dy_head_stride;
  p.y_row = dx_row_stride;
  p.y_head = dx_head_stride;
  p.partial = dweight != nullptr ? static_cast<float*>(workspace) : nullptr;
  p.lanes = vector_lanes(p, dtype, norm != 0 ? x : nullptr, dx, dy);
  const bool wide = vector_pairs(p) == 2;
  const void* k = by_dtype(dtype, [&](auto t) {
    constexpr int T = decltype(t)::value;
    return p.lanes == 0 ? reinterpret_cast<const void*>(rope_scalar_bwd_kernel<T>)
           : wide       ? reinterpret_cast<const void*>(rope_vec_bwd_kernel<T, 2>)
                        : reinterpret_cast<const void*>(rope_vec_bwd_kernel<T, 1>);
  });
  const size_t smem = dweight != nullptr ? sizeof(float) * kRopeWarps * (p.lanes == 0 ? 2 : 1) * d : 0;
  int bps = 0;
  if (blocks_per_sm(dev, k, kRopeThreads, smem, &bps) != cudaSuccess) return CSA_ERR_CUDA;
  if (bps < 1) return CSA_ERR_UNSUPPORTED;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  void* args[] = {&p};
  if (launch_pdl(k, dim3(static_cast<unsigned>(blocks)), dim3(kRopeThreads), smem, s, args) !=
      cudaSuccess)
    return CSA_ERR_CUDA;
  if (dweight == nullptr) return CSA_OK;
  return launch_partial_reduce(p.partial, static_cast<int>(blocks), d, dweight,
                               accumulate_dweight != 0, nullptr, s) == cudaSuccess
             ? CSA_OK
             : CSA_ERR_CUDA;
}
