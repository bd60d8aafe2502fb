// csa_step.cu -- the pooling of csa_compressor_fwd continued over calls: new tokens of each sequence go on
// from a state that holds the tokens whose block, or whose next block, is not complete yet (the
// interface is in csa_compressor.h).
//
// Every kv and score that a window reads is read once and by one block; bound by HBM bytes for chunks
// of many tokens, by the launch for single ones.
//
// A window's tokens lie among the call's, in the state, or both; a thread finds each by its position. The
// blocks whose windows reach into the state (the first `coff` of a sequence at most) and the state's new
// contents belong to one CTA per sequence and slice of columns, which reads before it writes; all other
// blocks read new tokens alone and are spread over the grid.
#include <climits>
#include <cmath>
#include <cstdint>

#include "csa_compressor.h"
#include "csa_element.cuh"
#include "csa_internal.h"

namespace csa {
namespace {

constexpr int kStepThreads = 256;
constexpr int kStepFlight = 8;  // (kv, score) pieces that a thread loads at a time

struct StepParams {
  const uint16_t* kv;
  const uint16_t* score;
  const float* ape;
  const int32_t* cu;
  const int32_t* first;
  const int32_t* source;
  const int32_t* target;
  uint16_t* kv_state;
  uint16_t* score_state;
  uint16_t* out;
  const int32_t* base;
  const int32_t* table;
  int32_t* positions;
  int64_t* slots;
  int32_t* entries;
  int32_t* dev_error;
  int64_t capacity, out_rows, num_states;
  int S, ratio, coff, d, C, W;
  int max_pages, page_size, offset;
  int R;       // CTAs of a column slice
  int CL;      // pieces of a slice
  int PG;      // threads that share a window's positions
  int RS;      // windows that a CTA works on at once
  int chunks;  // pieces of a row
};

// VEC consecutive bf16 values (4: 8 bytes, aligned), read once.
template <int VEC>
struct Piece;
template <>
struct Piece<4> {
  uint2 w;
  __device__ __forceinline__ void load(const uint16_t* p) {
    asm volatile("ld.global.cs.v2.u32 {%0, %1}, [%2];" : "=r"(w.x), "=r"(w.y) : "l"(p));
  }
  __device__ __forceinline__ void store(uint16_t* p) const { *reinterpret_cast<uint2*>(p) = w; }
  __device__ __forceinline__ void clear() { w = make_uint2(0, 0); }
  __device__ __forceinline__ float get(int i) const {
    const uint32_t x = i < 2 ? w.x : w.y;
    return i % 2 == 0 ? bf16_lo(x) : bf16_hi(x);
  }
};
template <>
struct Piece<1> {
  uint16_t w;
  __device__ __forceinline__ void load(const uint16_t* p) {
    asm volatile("ld.global.cs.u16 %0, [%1];" : "=h"(w) : "l"(p));
  }
  __device__ __forceinline__ void store(uint16_t* p) const { *p = w; }
  __device__ __forceinline__ void clear() { w = 0; }
  __device__ __forceinline__ float get(int) const { return __uint_as_float(static_cast<uint32_t>(w) << 16); }
};
template <int VEC>
__device__ __forceinline__ void load_embedding(float (&a)[VEC], const float* p) {
  if constexpr (VEC == 2) {
    const float2 t = __ldg(reinterpret_cast<const float2*>(p));
    a[0] = t.x;
    a[1] = t.y;
  } else {
    a[0] = __ldg(p);
  }
}

// What a sequence's call is.
struct StepSeq {
  int n, first, source, target;
  int64_t token0;  // where position 0 would lie among the call's tokens
  int lo, hi;      // blocks complete before the call, and after it
  int boundary;    // of those that it completes, the ones whose window reaches into the state
  __device__ __forceinline__ StepSeq(const StepParams& p, int s) {
    const int a = __ldg(p.cu + s);
    n = __ldg(p.cu + s + 1) - a;
    first = __ldg(p.first + s);
    source = __ldg(p.source + s);
    target = __ldg(p.target + s);
    token0 = static_cast<int64_t>(a) - first;
    lo = first / p.ratio;
    hi = (first + n) / p.ratio;
    boundary = boundary_of(p, first, lo, hi - lo);
  }
  static __device__ __forceinline__ int boundary_of(const StepParams& p, int first, int lo, int made) {
    const bool part = first != lo * p.ratio;
    return min(made, p.coff == 1 ? (part ? 1 : 0) : part ? 2 : lo > 0 ? 1 : 0);
  }
};

// Rows before each sequence (x), and those of them whose windows reach into no state (y), in shared memory, [S]
// holding all of them; false with the reason reported where the call's numbers are refused. Every thread of the
// block calls it.
__device__ bool build_step_prefix(const StepParams& p, int2* sB, int* warp_sums) {
  pdl_wait();
  int2 carry = make_int2(0, 0);
  int bad = 0;
  for (int base = 0; base < p.S || base == 0; base += blockDim.x) {
    const int s = base + threadIdx.x;
    int made = 0, inner = 0;
    if (s < p.S) {
      const int a = __ldg(p.cu + s), b = __ldg(p.cu + s + 1), f = __ldg(p.first + s);
      const int from = __ldg(p.source + s), to = __ldg(p.target + s), n = b - a, lo = f / p.ratio;
      const bool live = f != lo * p.ratio || (p.coff == 2 && lo > 0);  // the state holds something
      if (b < a || a < 0 || b > p.capacity) {
        bad |= 1;
      } else if (f < 0 || f > INT_MAX - n || from >= p.num_states || to >= p.num_states ||
                 (from < 0 && live && (n > 0 || to >= 0))) {
        bad |= 2;
      } else {
        made = (f + n) / p.ratio - lo;
        inner = made - StepSeq::boundary_of(p, f, lo, made);
      }
    }
    int all, all_inner = 0;
    const int before = block_exclusive_scan(made, warp_sums, all);
    // (a call of single tokens has no such row)
    const int inner_before = __syncthreads_or(inner) ? block_exclusive_scan(inner, warp_sums, all_inner) : 0;
    if (s < p.S) sB[s] = make_int2(carry.x + before, carry.y + inner_before);
    carry.x += all;
    carry.y += all_inner;
  }
  if (threadIdx.x == 0) sB[p.S] = carry;
  int code = 0;
  if (__syncthreads_or(bad)) code = __syncthreads_or(bad & 1) ? CSA_DEVERR_CU_SEQLENS : CSA_DEVERR_STATE;
  else if (carry.x > p.out_rows) code = CSA_DEVERR_OUT_ROWS;
  if (code != 0) {
    if (threadIdx.x == 0 && p.dev_error != nullptr) *reinterpret_cast<volatile int32_t*>(p.dev_error) = code;
    return false;
  }
  return true;
}

// Where row o's entry goes.
__device__ __forceinline__ void describe_row(const StepParams& p, const int2* sB, int o) {
  int s = 0, h = p.S;  // sB[s].x <= o < sB[h].x, the last such s
  while (h - s > 1) {
    const int mid = (s + h) / 2;
    if (sB[mid].x <= o) s = mid;
    else h = mid;
  }
  const int block = __ldg(p.first + s) / p.ratio + (o - sB[s].x);
  if (p.positions != nullptr) p.positions[o] = block * p.ratio + p.offset;
  if (p.slots != nullptr) {
    const int e = block - (p.base != nullptr ? __ldg(p.base + s) : 0);
    int64_t slot = -1;
    if (e >= 0) {
      const int at = e / p.page_size;
      const int page = at < p.max_pages ? __ldg(p.table + static_cast<int64_t>(s) * p.max_pages + at) : -1;
      if (page >= 0) slot = static_cast<int64_t>(page) * p.page_size + (e - at * p.page_size);
      else if (p.dev_error != nullptr) *p.dev_error = CSA_DEVERR_PAGE;
    }
    p.slots[o] = slot;
  }
}

// UW: positions of a window that a thread takes; windows of up to 4 positions go through a thread several at a
// time instead (K rows), so that as many bytes are under way. SPLIT: windows of more than 8 positions, which
// PG threads share. The next rows' pieces are loaded while one is worked out.
template <int VEC, int UW, bool SPLIT>
__global__ void __launch_bounds__(kStepThreads, 2) step_kernel(const __grid_constant__ StepParams p) {
  constexpr int K = kStepFlight / UW, PART = VEC == 4 ? 2 : 1;
  extern __shared__ __align__(16) int2 s_prefix[];  // [S + 1]
  __shared__ int warp_sums[32];
  __shared__ __align__(16) float s_part[SPLIT ? 2 : 1][SPLIT ? 3 * kStepThreads * VEC : 4];
  if (!build_step_prefix(p, s_prefix, warp_sums)) return;
  const int g = blockIdx.x, tid = threadIdx.x, per = p.CL * p.PG;
  const int rs = tid / per, pg = tid % per / p.CL, cl = tid % p.CL;
  const int chunk = blockIdx.y * p.CL + cl, c0 = chunk * VEC;
  const bool slot = rs < p.RS, mine = slot && chunk < p.chunks;  // this thread has a window, and columns
  const int total = s_prefix[p.S].x, inner = s_prefix[p.S].y;

  // This thread's positions: elements from the block's first one (own columns), the embedding's the same way
  const bool two = p.coff == 2;
  int off[UW];
  uint32_t there = 0, own = 0;  // bits: the window has this position, the block itself has
#pragma unroll
  for (int u = 0; u < UW; ++u) {
    const int w = pg + u * p.PG;
    const bool prev = two && w < p.ratio;
    off[u] = prev ? (w - p.ratio) * p.C - p.d : (two ? w - p.ratio : w) * p.C;
    if (mine && w < p.W) there |= 1u << u;
    if (!prev) own |= 1u << u;
  }
  const float* const ape_own = p.ape + (two ? p.d : 0) + c0;
  const float* const ape_prev = ape_own + static_cast<int64_t>(p.ratio) * p.C;

  struct Pieces {
    Piece<VEC> kv[UW], score[UW];
    uint32_t on;  // positions that are there
    int row;      // -1: none
  };
  // maximum, weight sum and weighted sum of this thread's positions, to the row or to the threads that share it
  auto finish = [&](const Pieces& v, int turn) {
    if (!SPLIT && v.row < 0) return;
    if (mine) {
      float top[VEC], z[VEC], a[VEC];
      // (two columns at a time, for the registers)
#pragma unroll
      for (int part = 0; part < VEC / PART; ++part) {
        float x[UW][PART];
#pragma unroll
        for (int i = 0; i < PART; ++i) top[part * PART + i] = -INFINITY;
#pragma unroll
        for (int u = 0; u < UW; ++u) {
          float e[PART];
#pragma unroll
          for (int i = 0; i < PART; ++i) e[i] = 0.f;
          if (there >> u & 1u) load_embedding<PART>(e, (own >> u & 1u ? ape_own : ape_prev) + off[u] + part * PART);
#pragma unroll
          for (int i = 0; i < PART; ++i) {
            x[u][i] = v.on >> u & 1u ? fmaf(v.score[u].get(part * PART + i), kLog2e, e[i] * kLog2e) : -INFINITY;
            top[part * PART + i] = fmaxf(top[part * PART + i], x[u][i]);
          }
        }
#pragma unroll
        for (int i = 0; i < PART; ++i) {
          const int c = part * PART + i;
          const float to = top[c] == -INFINITY ? 0.f : top[c];  // (scores of -inf alone weigh nothing)
          z[c] = a[c] = 0.f;
#pragma unroll
          for (int u = 0; u < UW; ++u) {
            const float f = fast_exp2(x[u][i] - to);
            z[c] += f;
            a[c] = fmaf(f, v.kv[u].get(c), a[c]);
          }
        }
      }
      if constexpr (SPLIT) {
        const int wide = p.CL * VEC, step = p.PG * wide;
        float* to = s_part[turn & 1] + rs * 3 * step + (pg * p.CL + cl) * VEC;
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          to[i] = top[i];
          to[step + i] = z[i];
          to[2 * step + i] = a[i];
        }
      } else {
        uint16_t* to = p.out + static_cast<int64_t>(v.row) * p.d + c0;
        if constexpr (VEC == 4) {
          *reinterpret_cast<uint2*>(to) = make_uint2(pack_bf16x2(a[0] * rcp_nr(z[0]), a[1] * rcp_nr(z[1])),
                                                     pack_bf16x2(a[2] * rcp_nr(z[2]), a[3] * rcp_nr(z[3])));
        } else {
          *to = Element<CSA_DTYPE_BF16>::from_float(a[0] * rcp_nr(z[0]));
        }
      }
    }
    if constexpr (SPLIT) {
      // the parts meet in shared memory, a column to a thread, in the positions' order (two turns' parts, so
      // that one barrier a row is enough)
      __syncthreads();
      if (slot && v.row >= 0) {
        const int wide = p.CL * VEC, step = p.PG * wide;
        const float* part = s_part[turn & 1] + rs * 3 * step;
        for (int c = tid % per; c < wide; c += per) {
          const int col = blockIdx.y * wide + c;
          if (col >= p.d) break;
          float m = -INFINITY, zz = 0.f, aa = 0.f;
#pragma unroll 8
          for (int q = 0; q < p.PG; ++q) m = fmaxf(m, part[q * wide + c]);
          const float to = m == -INFINITY ? 0.f : m;
#pragma unroll 8
          for (int q = 0; q < p.PG; ++q) {
            const float f = fast_exp2(part[q * wide + c] - to);
            zz = fmaf(part[step + q * wide + c], f, zz);
            aa = fmaf(part[2 * step + q * wide + c], f, aa);
          }
          p.out[static_cast<int64_t>(v.row) * p.d + col] = Element<CSA_DTYPE_BF16>::from_float(aa * rcp_nr(zz));
        }
      }
    }
  };

  // sequences: the blocks that reach into the state, then the state
  const int64_t state = static_cast<int64_t>(p.W) * p.C;
  int turn = 0;
  for (int s0 = g * p.RS; s0 < p.S; s0 += p.R * p.RS) {
    const int s = s0 + rs;
    const bool some = slot && s < p.S;
    const StepSeq q(p, some ? s : s0);
#pragma unroll 1
    for (int i = 0; i < p.coff; ++i) {
      const bool now = some && i < q.boundary;
      if (SPLIT ? !__syncthreads_or(now) : !now) continue;
      Pieces v;
      v.on = 0;
      v.row = now ? s_prefix[s].x + i : -1;
#pragma unroll
      for (int u = 0; u < UW; ++u) {
        v.kv[u].clear();
        v.score[u].clear();
        const int w = pg + u * p.PG;
        const int pos = (q.lo + i - (two ? 1 : 0)) * p.ratio + w;
        if (now && (there >> u & 1u) && pos >= 0) {
          v.on |= 1u << u;
          const bool old = pos < q.first;
          const int64_t at = (old ? q.source * state + static_cast<int64_t>(pos % p.W) * p.C : (q.token0 + pos) * p.C) +
                             (two && (own >> u & 1u) ? p.d : 0) + c0;
          v.kv[u].load((old ? p.kv_state : p.kv) + at);
          v.score[u].load((old ? p.score_state : p.score) + at);
        }
      }
      finish(v, turn++);
    }
    if (!some) continue;
    if (chunk == 0 && pg == 0 && p.entries != nullptr) p.entries[s] = max(0, q.hi - (p.base != nullptr ? __ldg(p.base + s) : 0));
    if (!mine || q.target < 0) continue;
    asm volatile("" ::: "memory");  // the state is read above, by loads that the compiler does not see as such
    for (int half = 0; half < p.coff; ++half) {
      const int keep = max(0, q.hi - (p.coff - 1 - half)) * p.ratio;  // the first position that a later window reads
      const int end = q.first + q.n;
      for (int pos = (q.source == q.target ? max(keep, q.first) : keep) + pg; pos < end; pos += p.PG) {
        const bool old = pos < q.first;
        const int64_t at = static_cast<int64_t>(pos % p.W) * p.C + half * p.d + c0;
        const int64_t from = old ? q.source * state + at : (q.token0 + pos) * p.C + half * p.d + c0;
        Piece<VEC> k, x;
        k.load((old ? p.kv_state : p.kv) + from);
        x.load((old ? p.score_state : p.score) + from);
        k.store(p.kv_state + q.target * state + at);
        x.store(p.score_state + q.target * state + at);
      }
    }
  }

  if (blockIdx.y == 0 && (p.positions != nullptr || p.slots != nullptr))
    for (int64_t o = static_cast<int64_t>(g) * kStepThreads + tid; o < p.out_rows; o += static_cast<int64_t>(p.R) * kStepThreads) {
      if (o < total) {
        describe_row(p, s_prefix, static_cast<int>(o));
      } else {  // behind the last entry
        if (p.positions != nullptr) p.positions[o] = -1;
        if (p.slots != nullptr) p.slots[o] = -1;
      }
    }

  // all other blocks: contiguous runs of rows
  const int i0 = static_cast<int>(static_cast<int64_t>(g) * inner / p.R);
  const int i1 = static_cast<int>(static_cast<int64_t>(g + 1) * inner / p.R);
  if (i0 >= i1) return;
  int seg = 0, seg_end = i0;  // the sequence of the last row asked for, where its rows end,
  int64_t seg_at = 0;         // and the element that row 0 would have for its own block's first one
  int seg_row = 0, seg_first = -1;  // its output rows less its rows here, and the row that is its block 0, if any
  auto fetch = [&](int i, Pieces& v) {
    v.on = 0;
    v.row = -1;
    if (!slot || i >= i1) return;
    if (i >= seg_end) {
      int lo = seg, hi = p.S;  // sB[lo].y <= i < sB[hi].y, the last such lo
      while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (s_prefix[mid].y <= i) lo = mid;
        else hi = mid;
      }
      seg = lo;
      seg_end = s_prefix[lo + 1].y;
      const StepSeq q(p, lo);
      const int2 at = s_prefix[lo];
      const int block = q.lo + q.boundary - at.y;  // of row 0
      seg_at = (q.token0 + static_cast<int64_t>(block) * p.ratio) * p.C + (two ? p.d : 0) + c0;
      seg_row = at.x + q.boundary - at.y;
      seg_first = -block;
    }
    v.row = i + seg_row;
    const int64_t at = seg_at + static_cast<int64_t>(i) * p.ratio * p.C;
    v.on = i == seg_first ? there & own : there;
#pragma unroll
    for (int u = 0; u < UW; ++u) {
      if (v.on >> u & 1u) {
        v.kv[u].load(p.kv + at + off[u]);
        v.score[u].load(p.score + at + off[u]);
      } else {
        v.kv[u].clear();
        v.score[u].clear();
      }
    }
  };
  Pieces v[2][K];
  const int step = p.RS * K;
#pragma unroll
  for (int k = 0; k < K; ++k) fetch(i0 + k * p.RS + rs, v[0][k]);
  for (int i = i0; i < i1;) {
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      if (i < i1) {
#pragma unroll
        for (int k = 0; k < K; ++k) fetch(i + step + k * p.RS + rs, v[b ^ 1][k]);
#pragma unroll
        for (int k = 0; k < K; ++k) finish(v[b][k], turn++);
        i += step;
      }
    }
  }
}

}  // namespace
}  // namespace csa

using namespace csa;

extern "C" csa_status_t csa_compressor_step(
    const void* kv, const void* score, const float* ape, const int32_t* cu_seqlens, int32_t S, int32_t ratio,
    int32_t coff, int32_t d, int64_t capacity, const int32_t* first, const int32_t* source,
    const int32_t* target, int64_t num_states, void* kv_state, void* score_state, void* out,
    int64_t out_rows, const int32_t* base, const int32_t* page_table, int32_t max_pages, int32_t page_size,
    int32_t position_offset, int32_t* positions, int64_t* slots, int32_t* entries, int32_t* dev_error,
    csa_stream_t stream) {
  if (S < 0 || ratio < 1 || d < 1 || capacity < 0 || out_rows < 0 || num_states < 0 || max_pages < 0 ||
      position_offset < 0 || position_offset >= ratio || (slots != nullptr && page_size < 1))
    return CSA_ERR_INVALID_VALUE;
  if (coff != 1 && coff != 2) return CSA_ERR_UNSUPPORTED;
  if (S > CSA_MAX_SEGMENTS || ratio > CSA_MAX_WINDOW / coff || d > CSA_MAX_ELEMS / (coff * CSA_MAX_WINDOW))
    return CSA_ERR_UNSUPPORTED;
  const int64_t C = static_cast<int64_t>(coff) * d, W = static_cast<int64_t>(coff) * ratio;
  if (capacity > CSA_MAX_ELEMS / C || out_rows > CSA_MAX_ELEMS / d || num_states > INT64_MAX / 64 / (W * C) ||
      num_states > INT_MAX)
    return CSA_ERR_UNSUPPORTED;
  if (cu_seqlens == nullptr || ape == nullptr) return CSA_ERR_INVALID_VALUE;
  if (S > 0 && (first == nullptr || source == nullptr || target == nullptr)) return CSA_ERR_INVALID_VALUE;
  if ((capacity > 0 && (kv == nullptr || score == nullptr)) || (out_rows > 0 && out == nullptr) ||
      (num_states > 0 && (kv_state == nullptr || score_state == nullptr)))
    return CSA_ERR_INVALID_VALUE;
  if (S > 0 && slots != nullptr && max_pages > 0 && page_table == nullptr) return CSA_ERR_INVALID_VALUE;
  if (!is_aligned(kv, 2) || !is_aligned(score, 2) || !is_aligned(ape, 4) || !is_aligned(cu_seqlens, 4) ||
      !is_aligned(first, 4) || !is_aligned(source, 4) || !is_aligned(target, 4) || !is_aligned(kv_state, 2) ||
      !is_aligned(score_state, 2) || !is_aligned(out, 2) || !is_aligned(base, 4) || !is_aligned(page_table, 4) ||
      !is_aligned(positions, 4) || !is_aligned(slots, 8) || !is_aligned(entries, 4) || !is_aligned(dev_error, 4))
    return CSA_ERR_INVALID_VALUE;
  if (S == 0 && (out_rows == 0 || (positions == nullptr && slots == nullptr))) return CSA_OK;

  StepParams p{};
  p.kv = static_cast<const uint16_t*>(kv);
  p.score = static_cast<const uint16_t*>(score);
  p.ape = ape;
  p.cu = cu_seqlens;
  p.first = first;
  p.source = source;
  p.target = target;
  p.kv_state = static_cast<uint16_t*>(kv_state);
  p.score_state = static_cast<uint16_t*>(score_state);
  p.out = static_cast<uint16_t*>(out);
  p.base = base;
  p.table = page_table;
  p.positions = positions;
  p.slots = slots;
  p.entries = entries;
  p.dev_error = dev_error;
  p.capacity = capacity;
  p.out_rows = out_rows;
  p.num_states = num_states;
  p.S = S;
  p.ratio = ratio;
  p.coff = coff;
  p.d = d;
  p.C = static_cast<int>(C);
  p.W = static_cast<int>(W);
  p.max_pages = max_pages;
  p.page_size = page_size;
  p.offset = position_offset;
  const bool vec = d % 4 == 0 && is_aligned(kv, 8) && is_aligned(score, 8) && is_aligned(ape, 16) &&
                   is_aligned(kv_state, 8) && is_aligned(score_state, 8) && is_aligned(out, 8);
  p.chunks = vec ? d / 4 : d;
  p.PG = 1;  // (at most 256: CSA_MAX_WINDOW is 2048)
  while (p.PG * kStepFlight < p.W) p.PG *= 2;
  const int most = kStepThreads / p.PG, slices = (p.chunks + most - 1) / most;
  p.CL = (p.chunks + slices - 1) / slices;
  p.RS = kStepThreads / (p.CL * p.PG);
  const int uw = p.W > 4 ? 8 : p.W > 2 ? 4 : p.W > 1 ? 2 : 1;
  auto pick = [&](auto v) -> const void* {
    constexpr int V = decltype(v)::value;
    return p.PG > 1  ? reinterpret_cast<const void*>(step_kernel<V, 8, true>)
           : uw == 8 ? reinterpret_cast<const void*>(step_kernel<V, 8, false>)
           : uw == 4 ? reinterpret_cast<const void*>(step_kernel<V, 4, false>)
           : uw == 2 ? reinterpret_cast<const void*>(step_kernel<V, 2, false>)
                     : reinterpret_cast<const void*>(step_kernel<V, 1, false>);
  };
  const void* k = vec ? pick(std::integral_constant<int, 4>{}) : pick(std::integral_constant<int, 1>{});
  const size_t smem = sizeof(int2) * (static_cast<size_t>(S) + 1);
  int dev = 0, sms = 0, bps = 0;
  if (note(cudaGetDevice(&dev)) != cudaSuccess || device_sms(dev, &sms) != cudaSuccess ||
      blocks_per_sm(dev, k, kStepThreads, smem, &bps) != cudaSuccess)
    return CSA_ERR_CUDA;
  if (bps < 1) return CSA_ERR_UNSUPPORTED;
  if (slices > 65535) return CSA_ERR_UNSUPPORTED;
  const int64_t by_rows = (out_rows + p.RS * (kStepFlight / uw) - 1) / (p.RS * (kStepFlight / uw));
  const int64_t by_seqs = (S + p.RS - 1) / p.RS;
  const int64_t want = by_rows > by_seqs ? by_rows : by_seqs, room = static_cast<int64_t>(sms) * bps / slices;
  p.R = static_cast<int>(want < room ? (want > 0 ? want : 1) : (room > 0 ? room : 1));
  void* args[] = {&p};
  return launch_pdl(k, dim3(p.R, slices), dim3(kStepThreads), smem, reinterpret_cast<cudaStream_t>(stream), args) ==
                 cudaSuccess
             ? CSA_OK
             : CSA_ERR_CUDA;
}
