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
constexpr int kStepFlight = 8;  // (kv, score) pieces of a thread under way

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
  int R;      // CTAs of a column slice
  int CL;     // pieces of a slice
  int PG;     // threads that share a window's positions
  int RS;     // windows that a CTA works on at once
  int chunks; // pieces of a row
};

// VEC consecutive bf16 values (8: 16 bytes, aligned).
template <int VEC>
struct Piece;
template <>
struct Piece<8> {
  uint4 w;
  // evict-first where nothing reads them again
  __device__ __forceinline__ void load_once(const uint16_t* p) {
    asm volatile("ld.global.cs.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w) : "l"(p));
  }
  __device__ __forceinline__ void store(uint16_t* p) const { *reinterpret_cast<uint4*>(p) = w; }
  __device__ __forceinline__ void clear() { w = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ float get(int i) const {
    const uint32_t x = i < 2 ? w.x : i < 4 ? w.y : i < 6 ? w.z : w.w;
    return i % 2 == 0 ? bf16_lo(x) : bf16_hi(x);
  }
};
template <>
struct Piece<1> {
  uint16_t w;
  __device__ __forceinline__ void load_once(const uint16_t* p) {
    asm volatile("ld.global.cs.u16 %0, [%1];" : "=h"(w) : "l"(p));
  }
  __device__ __forceinline__ void store(uint16_t* p) const { *p = w; }
  __device__ __forceinline__ void clear() { w = 0; }
  __device__ __forceinline__ float get(int) const { return __uint_as_float(static_cast<uint32_t>(w) << 16); }
};
template <int VEC>
__device__ __forceinline__ void load_embedding(float (&a)[VEC], const float* p) {
  if constexpr (VEC > 1) {
    load_ape<VEC>(a, p);
  } else {
    a[0] = __ldg(p);
  }
}

// What a sequence's call is.
struct StepSeq {
  int n, first, source, target;
  int64_t token0;  // where position 0 would lie among the call's tokens
  int lo, hi;      // blocks complete before the call, and after it
  int boundary;    // completed ones whose window reaches into the state
  __device__ __forceinline__ StepSeq(const StepParams& p, int s) {
    const int a = __ldg(p.cu + s);
    n = __ldg(p.cu + s + 1) - a;
    first = __ldg(p.first + s);
    source = __ldg(p.source + s);
    target = __ldg(p.target + s);
    token0 = static_cast<int64_t>(a) - first;
    lo = first / p.ratio;
    hi = (first + n) / p.ratio;
    const bool part = first % p.ratio != 0;
    boundary = min(hi - lo, p.coff == 1 ? (part ? 1 : 0) : part ? 2 : lo > 0 ? 1 : 0);
  }
};

// Rows before each sequence in shared memory, sB[S] = all, as build_block_prefix does for whole segments; -1
// with the reason reported where the call's numbers are refused. Every thread of the block calls it.
__device__ int build_step_prefix(const StepParams& p, int* sB, int* warp_sums) {
  pdl_wait();
  int carry = 0, bad = 0;
  if (threadIdx.x == 0 && (__ldg(p.cu) < 0 || __ldg(p.cu + p.S) > p.capacity)) bad = 1;
  for (int base = 0; base < p.S; base += blockDim.x) {
    const int s = base + threadIdx.x;
    int made = 0;
    if (s < p.S) {
      const int n = __ldg(p.cu + s + 1) - __ldg(p.cu + s), f = __ldg(p.first + s);
      const int from = __ldg(p.source + s), to = __ldg(p.target + s);
      const bool live = f % p.ratio != 0 || (p.coff == 2 && f >= p.ratio);  // the state holds something
      if (n < 0) {
        bad |= 1;
      } else if (f < 0 || f > INT_MAX - n || from >= p.num_states || to >= p.num_states ||
                 (from < 0 && live && (n > 0 || to >= 0))) {
        bad |= 2;
      } else {
        made = (f + n) / p.ratio - f / p.ratio;
      }
    }
    int total;
    const int before = block_exclusive_scan(made, warp_sums, total);
    if (s < p.S) sB[s] = carry + before;
    carry += total;
  }
  if (threadIdx.x == 0) sB[p.S] = carry;
  int code = 0;
  if (__syncthreads_or(bad & 1)) code = CSA_DEVERR_CU_SEQLENS;
  else if (__syncthreads_or(bad & 2)) code = CSA_DEVERR_STATE;
  else if (carry > p.out_rows) code = CSA_DEVERR_OUT_ROWS;
  if (code != 0) {
    if (threadIdx.x == 0 && p.dev_error != nullptr) *reinterpret_cast<volatile int32_t*>(p.dev_error) = code;
    return -1;
  }
  return carry;
}

// A block of a sequence whose window a thread works on.
struct StepRow {
  int64_t token0;  // as in StepSeq
  int64_t state;   // first element of the state that it goes on from
  int first, block, row;
  bool on;
};

// UW: positions of a window that a thread has under way at once; windows of up to 4 positions go
// through a thread several at a time instead, so that as many bytes are under way. SPLIT: windows of more
// than 8 positions, which PG threads share.
template <int VEC, int UW, bool SPLIT>
__global__ void __launch_bounds__(kStepThreads, 2) step_kernel(const __grid_constant__ StepParams p) {
  constexpr int K = kStepFlight / UW, PART = VEC == 8 ? 4 : 1;
  extern __shared__ __align__(16) int s_prefix[];  // [S + 1]
  __shared__ int warp_sums[32];
  __shared__ __align__(16) float s_part[SPLIT ? 3 * kStepThreads * VEC : 4];
  const int total = build_step_prefix(p, s_prefix, warp_sums);
  if (total < 0) return;
  const int g = blockIdx.x, tid = threadIdx.x, per = p.CL * p.PG;
  const int rs = tid / per, pg = tid % per / p.CL, cl = tid % p.CL;
  const int chunk = blockIdx.y * p.CL + cl;
  const bool mine = rs < p.RS && chunk < p.chunks;  // this thread has columns
  const int c0 = chunk * VEC;
  const bool scribe = rs < p.RS && pg == 0 && chunk == 0;  // it writes a row's position and slot

  if (blockIdx.y == 0)  // rows behind the last one
    for (int64_t o = total + static_cast<int64_t>(g) * kStepThreads + tid; o < p.out_rows;
         o += static_cast<int64_t>(p.R) * kStepThreads) {
      if (p.positions != nullptr) p.positions[o] = -1;
      if (p.slots != nullptr) p.slots[o] = -1;
    }

  auto describe = [&](int s, const StepRow& r) {
    if (!scribe || !r.on) return;
    if (p.positions != nullptr) p.positions[r.row] = r.block * p.ratio + p.offset;
    if (p.slots != nullptr) {
      const int e = r.block - (p.base != nullptr ? __ldg(p.base + s) : 0);
      int64_t slot = -1;
      if (e >= 0) {
        const int at = e / p.page_size;
        const int page = at < p.max_pages ? __ldg(p.table + static_cast<int64_t>(s) * p.max_pages + at) : -1;
        if (page >= 0) slot = static_cast<int64_t>(page) * p.page_size + e % p.page_size;
        else if (p.dev_error != nullptr) *p.dev_error = CSA_DEVERR_PAGE;
      }
      p.slots[r.row] = slot;
    }
  };

  // one window's (kv, score) pieces under way, for the positions w0, w0 + PG, ...: those at once of N rows
  auto pool = [&](auto count, const StepRow* rows) {
    constexpr int N = decltype(count)::value;
    float m[SPLIT ? VEC : 1], z[SPLIT ? VEC : 1], a[SPLIT ? VEC : 1];
    if constexpr (SPLIT) {
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        m[i] = -INFINITY;
        z[i] = a[i] = 0.f;
      }
    }
    for (int w0 = pg; w0 < p.W; w0 += UW * p.PG) {
      Piece<VEC> kv[N][UW], sc[N][UW];
      uint32_t on[N];  // positions that are there, a bit each
#pragma unroll
      for (int k = 0; k < N; ++k) {
        on[k] = 0;
#pragma unroll
        for (int u = 0; u < UW; ++u) {
          const int w = w0 + u * p.PG;
          const bool prev = p.coff == 2 && w < p.ratio;
          const int at = prev || p.coff == 1 ? w : w - p.ratio;
          const int pos = (rows[k].block - (prev ? 1 : 0)) * p.ratio + at;
          kv[k][u].clear();
          sc[k][u].clear();
          if (mine && rows[k].on && w < p.W && pos >= 0) {
            on[k] |= 1u << u;
            const bool old = pos < rows[k].first;
            const int64_t off = (old ? rows[k].state + static_cast<int64_t>(pos % p.W) * p.C : (rows[k].token0 + pos) * p.C) +
                                (prev || p.coff == 1 ? 0 : p.d) + c0;
            kv[k][u].load_once((old ? p.kv_state : p.kv) + off);
            sc[k][u].load_once((old ? p.score_state : p.score) + off);
          }
        }
      }
      if (!mine) continue;
      // PART columns of a row at a time
#pragma unroll
      for (int k = 0; k < N; ++k) {
        if (on[k] == 0 && (SPLIT || !rows[k].on)) continue;
        uint32_t y[VEC / 2 > 0 ? VEC / 2 : 1];
#pragma unroll
        for (int part = 0; part < VEC / PART; ++part) {
          float x[UW][PART];
          float top[PART], zz[PART], aa[PART];
#pragma unroll
          for (int i = 0; i < PART; ++i) top[i] = -INFINITY;
#pragma unroll
          for (int u = 0; u < UW; ++u) {
            const int w = w0 + u * p.PG;
            const bool own = p.coff == 2 && w >= p.ratio;
            float e[PART];
#pragma unroll
            for (int i = 0; i < PART; ++i) e[i] = 0.f;
            if (w < p.W) load_embedding<PART>(e, p.ape + static_cast<int64_t>(own ? w - p.ratio : w) * p.C + (own ? p.d : 0) + c0 + part * PART);
#pragma unroll
            for (int i = 0; i < PART; ++i) {
              x[u][i] = on[k] >> u & 1u ? fmaf(sc[k][u].get(part * PART + i), kLog2e, e[i] * kLog2e) : -INFINITY;
              top[i] = fmaxf(top[i], x[u][i]);
            }
          }
#pragma unroll
          for (int i = 0; i < PART; ++i) {
            // (while all scores are -inf their weights are 0)
            const float to = top[i] == -INFINITY ? 0.f : top[i];
            zz[i] = aa[i] = 0.f;
#pragma unroll
            for (int u = 0; u < UW; ++u) {
              const float f = fast_exp2(x[u][i] - to);
              zz[i] += f;
              aa[i] = fmaf(f, kv[k][u].get(part * PART + i), aa[i]);
            }
          }
          if constexpr (SPLIT) {
#pragma unroll
            for (int i = 0; i < PART; ++i) {
              const int c = part * PART + i;
              if (w0 == pg) {
                m[c] = top[i];
                z[c] = zz[i];
                a[c] = aa[i];
              } else {
                const float both = fmaxf(m[c], top[i]), to = both == -INFINITY ? 0.f : both;
                const float f = fast_exp2(m[c] - to), g2 = fast_exp2(top[i] - to);
                m[c] = both;
                z[c] = z[c] * f + zz[i] * g2;
                a[c] = a[c] * f + aa[i] * g2;
              }
            }
          } else if constexpr (VEC == 1) {
            p.out[static_cast<int64_t>(rows[k].row) * p.d + c0] = Element<CSA_DTYPE_BF16>::from_float(aa[0] / zz[0]);
          } else {
#pragma unroll
            for (int i = 0; i < PART; i += 2) y[(part * PART + i) / 2] = pack_bf16x2(aa[i] * rcp_nr(zz[i]), aa[i + 1] * rcp_nr(zz[i + 1]));
          }
        }
        if constexpr (!SPLIT && VEC == 8)
          *reinterpret_cast<uint4*>(p.out + static_cast<int64_t>(rows[k].row) * p.d + c0) = make_uint4(y[0], y[1], y[2], y[3]);
      }
    }
    if constexpr (SPLIT) {
      // (N is 1) the position groups' parts meet in shared memory, a column to a thread, in their order
      const int wide = p.CL * VEC;
      float* part = s_part + static_cast<size_t>(rs) * 3 * p.PG * wide;
      if (rs < p.RS) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          float* to = part + (pg * p.CL + cl) * VEC + i;
          to[0] = m[i];
          to[p.PG * wide] = z[i];
          to[2 * p.PG * wide] = a[i];
        }
      }
      __syncthreads();
      if (rs < p.RS && rows[0].on) {
        for (int c = tid % per; c < wide; c += per) {
          const int col = blockIdx.y * wide + c;
          if (col >= p.d) break;
          float top = -INFINITY, zz = 0.f, aa = 0.f;
          for (int q = 0; q < p.PG; ++q) top = fmaxf(top, part[q * wide + c]);
          const float to = top == -INFINITY ? 0.f : top;
          for (int q = 0; q < p.PG; ++q) {
            const float f = fast_exp2(part[q * wide + c] - to);
            zz = fmaf(part[(p.PG + q) * wide + c], f, zz);
            aa = fmaf(part[(2 * p.PG + q) * wide + c], f, aa);
          }
          p.out[static_cast<int64_t>(rows[0].row) * p.d + col] = Element<CSA_DTYPE_BF16>::from_float(aa / zz);
        }
      }
      __syncthreads();
    }
  };

  // sequences: the blocks that reach into the state, then the state
  const int64_t state = static_cast<int64_t>(p.W) * p.C;
  for (int s0 = g * p.RS; s0 < p.S; s0 += p.R * p.RS) {
    const int s = s0 + rs;
    const bool some = rs < p.RS && s < p.S;
    const StepSeq q(p, some ? s : s0);
    for (int i = 0; i < p.coff; ++i) {
      const StepRow r{q.token0, q.source * state, q.first, q.lo + i, s_prefix[some ? s : s0] + i, some && i < q.boundary};
      pool(std::integral_constant<int, 1>{}, &r);
      describe(s, r);
    }
    if (!some) continue;
    if (scribe && p.entries != nullptr) p.entries[s] = max(0, q.hi - (p.base != nullptr ? __ldg(p.base + s) : 0));
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
        k.load_once((old ? p.kv_state : p.kv) + from);
        x.load_once((old ? p.score_state : p.score) + from);
        k.store(p.kv_state + q.target * state + at);
        x.store(p.score_state + q.target * state + at);
      }
    }
  }

  // all other blocks: contiguous runs of rows
  const int o0 = static_cast<int>(static_cast<int64_t>(g) * total / p.R);
  const int o1 = static_cast<int>(static_cast<int64_t>(g + 1) * total / p.R);
  if (o0 >= o1) return;
  int seg = find_segment(s_prefix, p.S, o0);
  for (int o = o0; o < o1; o += p.RS * K) {
    StepRow rows[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int at = o + k * p.RS + rs;
      rows[k].on = false;
      rows[k].row = at;
      rows[k].block = 0;
      rows[k].first = 0;
      rows[k].state = rows[k].token0 = 0;
      if (rs < p.RS && at < o1) {
        seg = advance_segment(s_prefix, seg, at);
        const StepSeq q(p, seg);
        const int i = at - s_prefix[seg];
        rows[k].on = i >= q.boundary;
        rows[k].block = q.lo + i;
        rows[k].first = q.first;
        rows[k].token0 = q.token0;
        describe(seg, rows[k]);
      }
    }
    pool(std::integral_constant<int, K>{}, rows);
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
  const bool vec = d % 8 == 0 && is_aligned(kv, 16) && is_aligned(score, 16) && is_aligned(ape, 16) &&
                   is_aligned(kv_state, 16) && is_aligned(score_state, 16) && is_aligned(out, 16);
  p.chunks = vec ? d / 8 : d;
  // eight positions a thread, more than that only in windows that 32 threads cannot take so
  p.PG = 1;
  while (p.PG < 32 && p.PG * kStepFlight < p.W) p.PG *= 2;
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
  const void* k = vec ? pick(std::integral_constant<int, 8>{}) : pick(std::integral_constant<int, 1>{});
  const size_t smem = sizeof(int) * (static_cast<size_t>(S) + 1);
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
