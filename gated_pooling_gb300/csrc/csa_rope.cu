// csa_rope.cu -- head norm and rotation in one pass, forward and backward (the interface and
// the formulas are in csa_compressor.h).
//
// A row's head is read once, its mean square taken in fp32, and the columns written back
// normed and turned; backward, x and dy are read once and dx written. Bound by HBM bytes.
// Angles are taken as csa_rope.cuh says.
#include <cmath>
#include <climits>
#include <cstdint>
#include <type_traits>

#include "csa_compressor.h"
#include "csa_element.cuh"
#include "csa_internal.h"
#include "csa_rope.cuh"

namespace csa {
namespace {

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

// Blocks of the backward (= partial rows): enough to fill the GPU, at most one per warp's worth
// of units.
int64_t bwd_blocks(int64_t units, int sms) {
  const int64_t want = (units + kRopeWarps - 1) / kRopeWarps, most = 2 * static_cast<int64_t>(sms);
  return want < 1 ? 1 : (want < most ? want : most);
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
