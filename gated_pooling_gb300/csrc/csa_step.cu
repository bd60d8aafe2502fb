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
#include <type_traits>

#include "csa_compressor.h"
#include "csa_element.cuh"
#include "csa_internal.h"

namespace csa {
namespace {

constexpr int kStepThreads = 256;
constexpr int kStepFlight = 8;  // (kv, score) pieces that a thread loads at a time
constexpr int kStepJoin = 4;    // threads that join a column's parts, of at least as many
constexpr int kStepRound = 4;   // sequences whose numbers a thread looks up at a time, where there are many
// A sequence's positions end below this, so that one that is counted on by a round (kStepFlight times the threads that
// share a window, CSA_MAX_WINDOW), or by two, is an int still.
constexpr int kStepEnd = INT_MAX - 2 * CSA_MAX_WINDOW;

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
  int stages;  // turns under way
  // the first CTAs of a slice see to the sequences; those behind first_row_cta to the other blocks' rows
  int seq_ctas, first_row_cta;
  unsigned own_blocks;  // few tokens a sequence: the blocks of one that its own CTA works out
  unsigned checker;  // the CTA of a slice (the first one's works) that looks for states that sequences meet in
};

// VEC consecutive bf16 values (4: 8 bytes, aligned; 1: any).
template <int VEC>
struct Piece;
template <>
struct Piece<4> {
  uint2 w;
  __device__ __forceinline__ void load(const uint16_t* p) {
    asm volatile("ld.global.cs.v2.u32 {%0, %1}, [%2];" : "=r"(w.x), "=r"(w.y) : "l"(p) : "memory");
  }
  __device__ __forceinline__ void store(uint16_t* p) const { *reinterpret_cast<uint2*>(p) = w; }
  __device__ __forceinline__ void fill(uint16_t v) { w.x = w.y = v * 0x10001u; }
  __device__ __forceinline__ uint64_t pair(int i) const { return bf2_to_f2(i == 0 ? w.x : w.y); }
};
template <>
struct Piece<1> {
  uint16_t w;
  __device__ __forceinline__ void load(const uint16_t* p) {
    asm volatile("ld.global.cs.u16 %0, [%1];" : "=h"(w) : "l"(p) : "memory");
  }
  __device__ __forceinline__ void store(uint16_t* p) const { *p = w; }
  __device__ __forceinline__ void fill(uint16_t v) { w = v; }
  // (its second column is nobody's)
  __device__ __forceinline__ uint64_t pair(int) const { return f2_pack(__uint_as_float(static_cast<uint32_t>(w) << 16), 0.f); }
};
// What an absent position's pieces hold: a score of -inf, whose weight is 0, and a value of 0.
constexpr uint16_t kAbsentScore = 0xFF80, kAbsentValue = 0;

// A piece from memory into the thread's own place in shared memory, asynchronously where it has 8 bytes.
template <int VEC>
__device__ __forceinline__ void stage_piece(Piece<VEC>* to, const uint16_t* from) {
  if constexpr (VEC == 4) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(smem_addr(to)), "l"(from) : "memory");
  } else {
    to->load(from);
  }
}
__device__ __forceinline__ void stage_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Waits until all but the newest n stages are there.
__device__ __forceinline__ void stage_wait(int n) {
  if (n >= 2) asm volatile("cp.async.wait_group 2;" ::: "memory");
  else if (n == 1) asm volatile("cp.async.wait_group 1;" ::: "memory");
  else asm volatile("cp.async.wait_group 0;" ::: "memory");
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

// Exclusive sums of both over the block, and the block's totals. All threads call it; warp_sums: [32].
__device__ __forceinline__ int2 step_scan(int2 v, int2* warp_sums, int2& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int2 x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int a = __shfl_up_sync(0xFFFFFFFFu, x.x, o), b = __shfl_up_sync(0xFFFFFFFFu, x.y, o);
    if (lane >= o) {
      x.x += a;
      x.y += b;
    }
  }
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  int2 before = make_int2(x.x - v.x, x.y - v.y);
  total = make_int2(0, 0);
#pragma unroll
  for (int w = 0; w < kStepThreads / 32; ++w) {
    const int2 t = warp_sums[w];
    if (w < warp) {
      before.x += t.x;
      before.y += t.y;
    }
    total.x += t.x;
    total.y += t.y;
  }
  __syncthreads();
  return before;
}

// What is wrong with a sequence's numbers: 0, 1 (offsets) or 2 (lengths and states).
__device__ __forceinline__ int step_wrong(const StepParams& p, int a, int b, int f, int from, int to) {
  if (b < a || a < 0 || b > p.capacity) return 1;
  const int n = b - a;
  const bool live = f % p.ratio != 0 || (p.coff == 2 && f >= p.ratio);  // the state holds something
  return f < 0 || f > kStepEnd - n || from >= p.num_states || to >= p.num_states || (from < 0 && live && (n > 0 || to >= 0)) ? 2 : 0;
}

// The states that a sequence writes (x) and reads (y), -1: none. What it goes on from in place it only writes.
__device__ __forceinline__ int2 states_of(const StepParams& p, int n, int f, int from, int to) {
  const bool live = f % p.ratio != 0 || (p.coff == 2 && f >= p.ratio), moved = to != from && live;
  return make_int2(to >= 0 && (n > 0 || moved) ? to : -1, from >= 0 && moved && (n > 0 || to >= 0) ? from : -1);
}

// Reports a state that one sequence writes and another one writes or reads: CTAs that do not wait for one another would
// do so in any order. One CTA looks at all sequences, in a set of the written states (table: [slots] in shared
// memory, twice as many as sequences at least), beside the others' work: marks made by all CTAs while they count rows
// took 0.6 us of a single step's 4.9. All its threads; nothing is reported where the call's numbers are refused.
__device__ __noinline__ void check_states(const StepParams& p, int* table, int slots) {
  for (int i = threadIdx.x; i < slots; i += blockDim.x) table[i] = -1;
  __syncthreads();
  auto place = [&](int state) { return static_cast<int>(__umulhi(static_cast<unsigned>(state) * 0x9E3779B1u, static_cast<unsigned>(slots))); };
  // f(the states that it writes and reads) of every sequence of this thread whose numbers are right, kAt at a time: they come
  // side by side (one after another, 16384 sequences took 82 us)
  constexpr int kAt = 8;
  bool wrong = false, meet = false, reads = false;
  auto each = [&](auto f) {
    for (int s0 = threadIdx.x; s0 < p.S; s0 += kAt * blockDim.x) {
      int a[kAt], b[kAt], first[kAt], from[kAt], to[kAt];
#pragma unroll
      for (int i = 0; i < kAt; ++i) {
        const int s = min(s0 + i * static_cast<int>(blockDim.x), p.S - 1);
        a[i] = __ldg(p.cu + s);
        b[i] = __ldg(p.cu + s + 1);
        first[i] = __ldg(p.first + s);
        from[i] = __ldg(p.source + s);
        to[i] = __ldg(p.target + s);
      }
#pragma unroll
      for (int i = 0; i < kAt; ++i) {
        if (s0 + i * static_cast<int>(blockDim.x) >= p.S) break;
        if (step_wrong(p, a[i], b[i], first[i], from[i], to[i]) != 0) wrong = true;
        else f(states_of(p, b[i] - a[i], first[i], from[i], to[i]));
      }
    }
  };
  each([&](int2 m) {
    reads = reads || m.y >= 0;
    for (int at = m.x < 0 ? -1 : place(m.x); at >= 0; at = at + 1 < slots ? at + 1 : 0) {
      const int old = atomicCAS(table + at, -1, m.x);
      if (old == -1) break;
      if (old == m.x) {
        meet = true;
        break;
      }
    }
  });
  if (__syncthreads_or(wrong)) return;
  if (__syncthreads_or(reads))
    each([&](int2 m) {
      for (int at = m.y < 0 ? -1 : place(m.y); at >= 0 && table[at] != -1; at = at + 1 < slots ? at + 1 : 0)
        if (table[at] == m.y) {
          meet = true;
          break;
        }
    });
  if (meet && p.dev_error != nullptr) *reinterpret_cast<volatile int32_t*>(p.dev_error) = CSA_DEVERR_STATE;
}

// Asks L2 for the tokens of about the first `rows` rows of this CTA, by its place among those that see to rows: which
// they are is not known before the rows are counted, but the rows lie about as the tokens do.
__device__ __forceinline__ void ask_ahead(const StepParams& p, int tokens, int rows) {
  const int worker = static_cast<int>(blockIdx.x) - p.first_row_cta, workers = p.R - p.first_row_cta;
  if (worker < 0 || blockIdx.y != 0 || tokens <= 0 || tokens > p.capacity) return;
  const int64_t t0 = static_cast<int64_t>(tokens) * worker / workers, share = static_cast<int64_t>(tokens) * (worker + 1) / workers;
  const int64_t t1 = min(share, t0 + static_cast<int64_t>(rows) * p.ratio);
  const char *kv = reinterpret_cast<const char*>(p.kv), *score = reinterpret_cast<const char*>(p.score);
  for (int64_t at = t0 * p.C * 2 + threadIdx.x * 128; at < t1 * p.C * 2; at += kStepThreads * 128) {
    asm volatile("prefetch.global.L2 [%0];" ::"l"(kv + at));
    asm volatile("prefetch.global.L2 [%0];" ::"l"(score + at));
  }
}

// Rows before each sequence (x), and those of them whose windows reach into no state (y), in shared memory, [S]
// holding all of them; false with the reason reported where the call's numbers are refused. Every thread of the
// block calls it.
__device__ bool build_step_prefix(const StepParams& p, int2* sB, int2* warp_sums, int rows) {
  pdl_wait();
  int2 carry = make_int2(0, 0);
  int bad = 0;
  // a sequence a thread; of more than there are threads four neighbouring ones, so that there are fewer rounds
  const int per = p.S > kStepThreads ? kStepRound : 1;
  for (int base = 0; base < p.S || base == 0; base += kStepThreads * per) {
    const int s0 = base + static_cast<int>(threadIdx.x) * per;
    const int tokens = base == 0 ? __ldg(p.cu + p.S) : 0;
    int a[kStepRound + 1], f[kStepRound], from[kStepRound], to[kStepRound];
    int2 rows_of[kStepRound], mine = make_int2(0, 0);
    if (s0 < p.S) a[0] = __ldg(p.cu + s0);
#pragma unroll
    for (int j = 0; j < kStepRound; ++j)
      if (j < per && s0 + j < p.S) {
        a[j + 1] = __ldg(p.cu + s0 + j + 1);
        f[j] = __ldg(p.first + s0 + j);
        from[j] = __ldg(p.source + s0 + j);
        to[j] = __ldg(p.target + s0 + j);
      }
    if (base == 0) ask_ahead(p, tokens, rows);
#pragma unroll
    for (int j = 0; j < kStepRound; ++j) {
      rows_of[j] = mine;
      if (j < per && s0 + j < p.S) {
        const int why = step_wrong(p, a[j], a[j + 1], f[j], from[j], to[j]);
        bad |= why;
        if (why == 0) {
          const int lo = f[j] / p.ratio, made = (f[j] + (a[j + 1] - a[j])) / p.ratio - lo;
          mine.x += made;
          mine.y += made - StepSeq::boundary_of(p, f[j], lo, made);
        }
      }
    }
    int2 all;
    const int2 before = step_scan(mine, warp_sums, all);
#pragma unroll
    for (int j = 0; j < kStepRound; ++j)
      if (j < per && s0 + j < p.S) sB[s0 + j] = make_int2(carry.x + before.x + rows_of[j].x, carry.y + before.y + rows_of[j].y);
    carry.x += all.x;
    carry.y += all.y;
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

// Where the entry of a sequence's block goes, which is row o.
__device__ __forceinline__ void describe_row(const StepParams& p, int s, int block, int64_t o) {
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
__device__ __forceinline__ void no_row(const StepParams& p, int64_t o) {  // behind the last entry
  if (p.positions != nullptr) p.positions[o] = -1;
  if (p.slots != nullptr) p.slots[o] = -1;
}

// The maximum of a thread's positions, the sum of their weights against it, and their weighted sum, of each of its
// columns. A score less the maximum is what log2 e multiplies: multiplied before, one beyond 2.3e38 (a type's lowest
// value as a mask, wherever a window has no other) would be infinite.
template <int VEC>
struct Weighed {
  static constexpr int kPairs = VEC == 4 ? 2 : 1;
  uint64_t z[kPairs], a[kPairs];
  float top[2 * kPairs];
  template <int UW>
  __device__ __forceinline__ void of(const Piece<VEC> (&kv)[UW], const Piece<VEC> (&score)[UW], const uint64_t (&embedding)[UW][kPairs]) {
    const uint64_t log2e = f2_pack(kLog2e, kLog2e);
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
      uint64_t x[UW];
#pragma unroll
      for (int u = 0; u < UW; ++u) x[u] = f2_add(score[u].pair(i), embedding[u][i]);
      float lo = f2_lo(x[0]), hi = f2_hi(x[0]);
#pragma unroll
      for (int u = 1; u + 1 < UW; u += 2) {
        lo = fmax3(lo, f2_lo(x[u]), f2_lo(x[u + 1]));
        hi = fmax3(hi, f2_hi(x[u]), f2_hi(x[u + 1]));
      }
      if constexpr (UW % 2 == 0) {
        lo = fmaxf(lo, f2_lo(x[UW - 1]));
        hi = fmaxf(hi, f2_hi(x[UW - 1]));
      }
      top[2 * i] = lo;
      top[2 * i + 1] = hi;
      // (scores of -inf alone weigh nothing)
      const uint64_t to = f2_pack(lo == -INFINITY ? 0.f : -lo, hi == -INFINITY ? 0.f : -hi);
      z[i] = a[i] = 0;
#pragma unroll
      for (int u = 0; u < UW; ++u) {
        const uint64_t t = f2_mul(f2_add(x[u], to), log2e), f = f2_pack(fast_exp2(f2_lo(t)), fast_exp2(f2_hi(t)));
        z[i] = f2_add(z[i], f);
        a[i] = f2_fma(f, kv[u].pair(i), a[i]);
      }
    }
  }
  __device__ __forceinline__ uint32_t two_columns(int i) const {
    return f2_to_bf2(f2_mul(a[i], f2_pack(rcp_nr(f2_lo(z[i])), rcp_nr(f2_hi(z[i])))));
  }
  __device__ __forceinline__ void store(uint16_t* to) const {  // the entry, of whole windows
    if constexpr (VEC == 4) *reinterpret_cast<uint2*>(to) = make_uint2(two_columns(0), two_columns(1));
    else *to = static_cast<uint16_t>(two_columns(0));
  }
  __device__ __forceinline__ void leave(float* to, int step) const {  // as a part: three rows of a column each
    if constexpr (VEC == 4) {
      *reinterpret_cast<float4*>(to) = make_float4(top[0], top[1], top[2], top[3]);
      *reinterpret_cast<ulonglong2*>(to + step) = make_ulonglong2(z[0], z[1]);
      *reinterpret_cast<ulonglong2*>(to + 2 * step) = make_ulonglong2(a[0], a[1]);
    } else {
      to[0] = top[0];
      to[step] = f2_lo(z[0]);
      to[2 * step] = f2_lo(a[0]);
    }
  }
};

// Parts of a window's columns, of PG threads, [3][PG][wide], and the threads that join them: kStepJoin neighbouring ones
// to a column. The parts of each of those lie 8 columns on from the one's before, for the banks of the threads that
// read them together.
struct Join {
  static constexpr int kJ = kStepJoin, kTurn = 32 / kJ;
  int wide, many, step, from, turned;
  __device__ __forceinline__ Join(int PG, int wide_)
      : wide(wide_), many(PG / kJ), step(PG * wide), from(threadIdx.x % kJ * many * wide), turned(threadIdx.x % kJ * kTurn % wide) {}
  // where column c of part pg lies
  __device__ __forceinline__ int place(int pg, int c) const {
    c += pg / many * kTurn % wide;
    return pg * wide + (c >= wide ? c - wide : c);
  }
  // Column c of `parts`, for this thread's share of them, to `to` where that is given. All lanes of a warp call it
  // together (shuffles of a few lanes each by their own mask run one after another).
  __device__ __forceinline__ void column(const float* parts, int c, uint16_t* to) const {
    c += turned;
    const float* at = parts + from + (c >= wide ? c - wide : c);
    float m = -INFINITY, z = 0.f, a = 0.f;
#pragma unroll 4
    for (int q = 0; q < many; ++q) m = fmaxf(m, at[q * wide]);
#pragma unroll
    for (int o = 1; o < kJ; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    const float base = m == -INFINITY ? 0.f : m;
#pragma unroll 4
    for (int q = 0; q < many; ++q) {
      const float f = fast_exp2((at[q * wide] - base) * kLog2e);
      z = fmaf(at[step + q * wide], f, z);
      a = fmaf(at[2 * step + q * wide], f, a);
    }
#pragma unroll
    for (int o = 1; o < kJ; o <<= 1) {
      z += __shfl_xor_sync(0xFFFFFFFFu, z, o);
      a += __shfl_xor_sync(0xFFFFFFFFu, a, o);
    }
    if (to != nullptr && threadIdx.x % kJ == 0) *to = Element<CSA_DTYPE_BF16>::from_float(a * rcp_nr(z));
  }
};

// Bytes of shared memory: a stage holds the (kv, score) pieces of a thread's positions at once; SPLIT, two turns'
// parts; then the prefix.
__host__ __device__ constexpr int step_stage_bytes(int vec) { return 2 * kStepFlight * kStepThreads * vec * 2; }
__host__ __device__ constexpr int step_part_bytes(int vec, bool split) { return split ? 2 * 3 * kStepThreads * vec * 4 : 0; }

// UW: positions of a window that a thread takes; windows of up to 4 positions go through a thread several at a
// time instead (K rows), so that as many bytes are under way. SPLIT: windows of more than 8 positions, which
// PG threads share.
//
// A thread's pieces come into places of its own in shared memory (no barrier), p.stages turns ahead: 32 KB a turn
// and CTA. Two CTAs an SM, so that one has something to do while the other counts rows, waits or joins parts (one
// of 512 threads: 16.7, 35.7 and 14.1 us below). Three chunks of up to 8192 tokens of 512 in blocks of 4 take 15.6 us
// (64 % of the copy rate), four of up to 16384 in blocks of 128 33.6 us (60 %), five of up to 1805 tokens of 128 in
// blocks of 16 11.8; registers held one turn ahead, less than latency asks for: 22.7 and 43.8 for the first two.
template <int VEC, int UW, bool SPLIT>
__global__ void __launch_bounds__(kStepThreads, 2) step_kernel(const __grid_constant__ StepParams p) {
  constexpr int K = SPLIT ? 1 : kStepFlight / UW, PAIRS = VEC == 4 ? 2 : 1;
  constexpr uint32_t kAll = (1u << UW) - 1u;
  using P = Piece<VEC>;
  extern __shared__ __align__(16) unsigned char s_raw[];
  __shared__ int2 warp_sums[32];
  float* const s_part = reinterpret_cast<float*>(s_raw + p.stages * step_stage_bytes(VEC));  // [2][RS][3][PG][CL * VEC]
  int2* const s_prefix = reinterpret_cast<int2*>(s_raw + p.stages * step_stage_bytes(VEC) + step_part_bytes(VEC, SPLIT));  // [S + 1]
  if (blockIdx.x == p.checker) {
    pdl_wait();
    if (blockIdx.y == 0) check_states(p, reinterpret_cast<int*>(s_prefix), 2 * p.S);
    if (blockIdx.x == static_cast<unsigned>(p.R)) return;  // a CTA of its own
    __syncthreads();
  }
  if (!build_step_prefix(p, s_prefix, warp_sums, p.stages * p.RS * K)) return;
  const int g = blockIdx.x, tid = threadIdx.x, per = p.CL * p.PG;
  const int rs = tid / per, pg = tid % per / p.CL, cl = tid % p.CL;
  const int chunk = blockIdx.y * p.CL + cl, c0 = chunk * VEC;
  const bool slot = rs < p.RS, mine = slot && chunk < p.chunks;  // this thread has a window, and columns
  const int total = s_prefix[p.S].x, inner = s_prefix[p.S].y;
  // kv and score pieces of stage b: [k][u], a thread's 8 or 2 bytes beside the next one's
  auto place = [&](int b, int k, int u, int which) {
    return reinterpret_cast<P*>(s_raw + b * step_stage_bytes(VEC)) + ((k * UW + u) * 2 + which) * kStepThreads + tid;
  };

  // This thread's positions: elements from the block's first one (own columns)
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
  // the embedding at these positions, once for all rows; 0 behind the window
  uint64_t embedding[UW][PAIRS];
  bool embedded = false;
  auto embed = [&]() {
    if (embedded) return;
    embedded = true;
    const float* const ape_own = p.ape + (two ? p.d : 0) + c0;
    const float* const ape_prev = ape_own + static_cast<int64_t>(p.ratio) * p.C;
#pragma unroll
    for (int u = 0; u < UW; ++u) {
      float e[4] = {};
      const float* from = (own >> u & 1u ? ape_own : ape_prev) + off[u];
      if (there >> u & 1u) {
        if constexpr (VEC == 4) load_ape<4>(e, from);
        else e[0] = __ldg(from);
      }
#pragma unroll
      for (int i = 0; i < PAIRS; ++i) embedding[u][i] = f2_pack(e[2 * i], e[2 * i + 1]);
    }
  };

  const int wide = p.CL * VEC;
  const Join join(SPLIT ? p.PG : kStepJoin, wide);
  const int part_at = SPLIT ? join.place(pg, cl * VEC) : 0;
  // maximum, weight sum and weighted sum of this thread's positions in a stage, to the row (-1: none) or to the
  // threads that share it
  auto finish = [&](int b, int k, int row, int turn) {
    if (!SPLIT && row < 0) return;
    if (mine) {
      P kv[UW], score[UW];
#pragma unroll
      for (int u = 0; u < UW; ++u) {
        kv[u] = *place(b, k, u, 0);
        score[u] = *place(b, k, u, 1);
      }
      Weighed<VEC> r;
      r.template of<UW>(kv, score, embedding);
      if constexpr (SPLIT) {
        r.leave(s_part + (turn & 1) * 3 * kStepThreads * VEC + rs * 3 * join.step + part_at, join.step);
      } else {
        r.store(p.out + static_cast<int64_t>(row) * p.d + c0);
      }
    }
    if constexpr (SPLIT) {
      // the parts meet in shared memory in a fixed order, a column to J neighbouring threads (two turns'
      // parts, so that one barrier a row is enough)
      __syncthreads();
      const float* part = s_part + (turn & 1) * 3 * kStepThreads * VEC + min(rs, p.RS - 1) * 3 * join.step;
      for (int c0 = 0; c0 < wide; c0 += per / Join::kJ) {  // (as often for every lane)
        const int c = c0 + tid % per / Join::kJ, col = blockIdx.y * wide + c;
        join.column(part, min(c, wide - 1),
                    slot && row >= 0 && c < wide && col < p.d ? p.out + static_cast<int64_t>(row) * p.d + col : nullptr);
      }
    }
  };

  // Sequences: the blocks that reach into the state (two at most), then the state. All that is loaded for a sequence
  // is under way together, by way of this thread's places for three turns, where there are three.
  const int64_t state = static_cast<int64_t>(p.W) * p.C;
  int turn = 0;
  const bool room = p.stages == 3;
  for (int s0 = g * p.RS; s0 < p.S && g < p.seq_ctas; s0 += p.seq_ctas * p.RS) {
    const int s = s0 + rs;
    const bool some = slot && s < p.S;
    const StepSeq q(p, some ? s : s0);
    const bool now0 = some && q.boundary > 0, now1 = some && q.boundary > 1;
    const bool any0 = __syncthreads_or(now0), any1 = any0 && __syncthreads_or(now1);
    const int64_t old_at = q.source * state + c0, new_at = q.token0 * p.C + c0, keep_at = q.target * state + c0;
    // f(i, position, its row in a state) for kStepFlight (or n) positions from `from` on, p.PG apart
    auto each = [&](auto n, int from, auto f) {
      int r = max(from, 0) % p.W;  // (a position below 0 is not asked for)
      if (from < 0) r = from + p.W;
#pragma unroll
      for (int i = 0; i < decltype(n)::value; ++i) {
        f(i, from + i * p.PG, r);
        r += p.PG;
        if (r >= p.W) r -= p.W;
      }
    };
    auto load = [&](int b, int i, int pos, int r, int half) {
      const bool old = pos < q.first;
      const int64_t at = (old ? old_at + static_cast<int64_t>(r) * p.C : new_at + static_cast<int64_t>(pos) * p.C) + half;
      stage_piece(place(b, 0, i, 0), (old ? p.kv_state : p.kv) + at);
      stage_piece(place(b, 0, i, 1), (old ? p.score_state : p.score) + at);
    };
    auto window = [&](int b, int block, bool now) {
      each(std::integral_constant<int, UW>{}, (block - (two ? 1 : 0)) * p.ratio + pg, [&](int u, int pos, int r) {
        if (now && (there >> u & 1u) && pos >= 0) {
          load(b, u, pos, r, two && (own >> u & 1u) ? p.d : 0);
        } else {
          place(b, 0, u, 0)->fill(kAbsentValue);
          place(b, 0, u, 1)->fill(kAbsentScore);
        }
      });
    };
    // what goes into the state of a half's columns: the thread's positions from `from` on, kStepFlight at a time
    const int end = some && mine && q.target >= 0 ? q.first + q.n : 0;
    auto keep_from = [&](int half) {
      const int keep = max(0, q.hi - (p.coff - 1 - half)) * p.ratio;  // the first position that a later window reads
      return (q.source == q.target ? max(keep, q.first) : keep) + pg;
    };
    auto keep_load = [&](int b, int half, int from) {
      if (from >= end) return;
      each(std::integral_constant<int, kStepFlight>{}, from, [&](int i, int pos, int r) {
        if (pos < end) load(b, i, pos, r, half * p.d);
      });
    };
    auto keep_store = [&](int b, int half, int from) {
      if (from >= end) return;
      each(std::integral_constant<int, kStepFlight>{}, from, [&](int i, int pos, int r) {
        if (pos >= end) return;
        const int64_t to = keep_at + static_cast<int64_t>(r) * p.C + half * p.d;
        place(b, 0, i, 0)->store(p.kv_state + to);
        place(b, 0, i, 1)->store(p.score_state + to);
      });
    };
    const int from0 = keep_from(0), from1 = two ? keep_from(1) : 0;
    if (any0) window(0, q.lo, now0);
    stage_commit();
    if (room) {
      if (any1) window(1, q.lo + 1, now1);
      stage_commit();
      keep_load(2, 0, from0);
      stage_commit();
    }
    if (any0) {
      embed();
      stage_wait(room ? 2 : 0);
      finish(0, 0, now0 ? s_prefix[s].x : -1, turn++);
    }
    if (any1 && !room) {
      window(0, q.lo + 1, now1);
      stage_commit();
    }
    if (room && two) {
      keep_load(0, 1, from1);
      stage_commit();
    }
    if (any1) {
      stage_wait(room ? 2 : 0);
      finish(room ? 1 : 0, 0, now1 ? s_prefix[s].x + 1 : -1, turn++);
    }
    if (some && chunk == 0 && pg == 0 && p.entries != nullptr)
      p.entries[s] = max(0, q.hi - (p.base != nullptr ? __ldg(p.base + s) : 0));
    stage_wait(0);
    if (room) {
      keep_store(2, 0, from0);
      if (two) keep_store(0, 1, from1);
    }
    for (int half = 0; half < p.coff; ++half)
      for (int from = (half == 0 ? from0 : from1) + (room ? kStepFlight * p.PG : 0); from < end; from += kStepFlight * p.PG) {
        keep_load(0, half, from);
        stage_commit();
        stage_wait(0);
        keep_store(0, half, from);
      }
  }

  const int worker = g - p.first_row_cta, workers = p.R - p.first_row_cta;
  auto describe = [&]() {
    if (blockIdx.y == 0 && g >= p.first_row_cta && (p.positions != nullptr || p.slots != nullptr))
      for (int64_t o = static_cast<int64_t>(tid) * workers + worker; o < p.out_rows; o += static_cast<int64_t>(workers) * kStepThreads) {
        if (o >= total) {
          no_row(p, o);
          continue;
        }
        int s = 0, h = p.S;  // rows before s <= o < rows before h, the last such s
        while (h - s > 1) {
          const int mid = (s + h) / 2;
          if (s_prefix[mid].x <= o) s = mid;
          else h = mid;
        }
        describe_row(p, s, __ldg(p.first + s) / p.ratio + static_cast<int>(o - s_prefix[s].x), o);
      }
  };

  // all other blocks: contiguous runs of rows
  const int i0 = worker < 0 ? 0 : static_cast<int>(static_cast<int64_t>(worker) * inner / workers);
  const int i1 = worker < 0 ? 0 : static_cast<int>(static_cast<int64_t>(worker + 1) * inner / workers);
  if (i0 >= i1) {
    describe();
    return;
  }
  // a walk over them: the sequence of the row asked for last, where its rows end,
  struct Walk {
    int seg = 0, end;
    int64_t at = 0;          // the element that row 0 would have for its own block's first one,
    int row = 0, first = -1;  // its output rows less its rows here, and the row that is its block 0, if any
  };
  auto find = [&](Walk& w, int i) {
    if (i < w.end) return;
    int lo = w.seg, hi = p.S;  // sB[lo].y <= i < sB[hi].y, the last such lo
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (s_prefix[mid].y <= i) lo = mid;
      else hi = mid;
    }
    w.seg = lo;
    w.end = s_prefix[lo + 1].y;
    const StepSeq q(p, lo);
    const int2 before = s_prefix[lo];
    const int block = q.lo + q.boundary - before.y;  // of row 0
    w.at = (q.token0 + static_cast<int64_t>(block) * p.ratio) * p.C + (two ? p.d : 0) + c0;
    w.row = before.x + q.boundary - before.y;
    w.first = -block;
  };
  Walk ahead, here;
  ahead.end = here.end = i0;
  auto fetch = [&](unsigned i, int b, int k) {  // (may have passed 2^31 - 1)
    if (!mine || i >= static_cast<unsigned>(i1)) return;
    find(ahead, static_cast<int>(i));
    const int64_t at = ahead.at + static_cast<int64_t>(i) * p.ratio * p.C;
    const uint16_t *kv = p.kv + at, *score = p.score + at;
    const uint32_t on = static_cast<int>(i) == ahead.first ? there & own : there;
    if (on == kAll) {
#pragma unroll
      for (int u = 0; u < UW; ++u) {
        stage_piece(place(b, k, u, 0), kv + off[u]);
        stage_piece(place(b, k, u, 1), score + off[u]);
      }
      return;
    }
#pragma unroll
    for (int u = 0; u < UW; ++u) {
      if (on >> u & 1u) {
        stage_piece(place(b, k, u, 0), kv + off[u]);
        stage_piece(place(b, k, u, 1), score + off[u]);
      } else {
        place(b, k, u, 0)->fill(kAbsentValue);
        place(b, k, u, 1)->fill(kAbsentScore);
      }
    }
  };
  const int step = p.RS * K;
  for (int b = 0; b < p.stages; ++b) {
#pragma unroll
    for (int k = 0; k < K; ++k) fetch(i0 + b * step + k * p.RS + rs, b, k);
    stage_commit();
  }
  embed();
  describe();  // (while the first rows are on their way)
  for (unsigned i = i0, b = 0; i < static_cast<unsigned>(i1); i += step) {
    stage_wait(p.stages - 1);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const unsigned mine_i = i + k * p.RS + rs;
      int row = -1;
      if (slot && mine_i < static_cast<unsigned>(i1)) {
        find(here, static_cast<int>(mine_i));
        row = static_cast<int>(mine_i) + here.row;
      }
      finish(b, k, row, turn++);
    }
#pragma unroll
    for (int k = 0; k < K; ++k) fetch(i + p.stages * step + k * p.RS + rs, b, k);
    stage_commit();
    if (++b == static_cast<unsigned>(p.stages)) b = 0;
  }
}

// Calls of few tokens a sequence: a CTA per p.RS sequences and column slice, whose blocks it works out one after
// another. What counts is the way from the lengths to the entry, so there is little code; the first window and the
// embedding come while the rows before it are counted, and so does what goes into the states, which the lines of CL
// threads share out among them. Where one sequence has more tokens than the others (a chunk of a prompt in a batch of
// single ones), its blocks behind those of kFewTokens tokens (and behind the two that may read its state) are shared out
// among all CTAs: a CTA works out one after another in about 1 us each (449 tokens beside 63 single ones, blocks of 4,
// d 512: 11.0 us, 17.9 with eight blocks by its own CTA).
constexpr int kFewThreads = 256, kFewSeqs = 512, kFewTokens = 8;
template <int VEC, int UW, bool SPLIT>
__global__ void __launch_bounds__(kFewThreads, SPLIT ? 2 : 1) step_few_kernel(const __grid_constant__ StepParams p) {
  using P = Piece<VEC>;
  __shared__ __align__(16) float s_part[SPLIT ? 3 * kFewThreads * VEC : 4];
  __shared__ uint2 s_sums[kFewThreads / 32];
  __shared__ int2 s_rows[kFewSeqs];  // where blocks are shared out: rows before each sequence, and of those shared out
  const int tid = threadIdx.x, per = p.CL * p.PG, s0 = blockIdx.x * p.RS, s1 = min(p.S, s0 + p.RS);
  const int pg = tid / p.CL, cl = tid - pg * p.CL;
  const int chunk = blockIdx.y * p.CL + cl, c0 = chunk * VEC;
  const bool two = p.coff == 2, mine = tid < per && chunk < p.chunks;
  pdl_wait();
  if (blockIdx.x == p.checker) {
    if (blockIdx.y == 0) check_states(p, reinterpret_cast<int*>(s_rows), 2 * kFewSeqs);
    return;
  }
  // the whole call's lengths: what is wrong with them, the rows before these sequences and (from bit 13 on) of all, and
  // the shared-out ones. (All entries are at most `capacity`, of which calls with up to kFewTokens a sequence come here, whichever
  // sequences have them; offsets that are refused may add up to anything, without a sign so that they may.)
  static_assert(kFewTokens * kFewSeqs < 1 << 13);
  int bad = 0;
  unsigned rows = 0, shared = 0;
  for (int i = tid; i < p.S; i += blockDim.x) {
    const int a = __ldg(p.cu + i), b = __ldg(p.cu + i + 1), f = __ldg(p.first + i);
    const int from = __ldg(p.source + i), to = __ldg(p.target + i), why = step_wrong(p, a, b, f, from, to);
    bad |= why;
    if (why == 0) {
      const unsigned made = (f + (b - a)) / p.ratio - f / p.ratio;
      rows += (made << 13) + (i < s0 ? made : 0u);
      shared += made > p.own_blocks ? made - p.own_blocks : 0u;
    }
  }
  // (numbers of one sequence, of which nothing is read until they are known to be right)
  auto fine = [&](const StepSeq& q, int s) {
    return step_wrong(p, __ldg(p.cu + s), __ldg(p.cu + s + 1), q.first, q.source, q.target) == 0;
  };
  const int64_t state = static_cast<int64_t>(p.W) * p.C;
  P kv[UW], score[UW];
  uint64_t embedding[UW][Weighed<VEC>::kPairs];
  auto fetch = [&](const StepSeq& q, int block) {
    const int from = (block - (two ? 1 : 0)) * p.ratio + pg;
    int ring = from < 0 ? from + p.W : from % p.W;  // a position's row in a state
#pragma unroll
    for (int u = 0; u < UW; ++u) {
      const int w = pg + u * p.PG, r = ring;
      const bool prev = two && w < p.ratio;
      const int pos = from + u * p.PG;
      ring += p.PG;
      if (ring >= p.W) ring -= p.W;
      kv[u].fill(kAbsentValue);
      score[u].fill(kAbsentScore);
      if (mine && w < p.W && pos >= 0) {
        const bool old = pos < q.first;
        const int64_t at = (old ? q.source * state + static_cast<int64_t>(r) * p.C : (q.token0 + pos) * p.C) +
                           (two && !prev ? p.d : 0) + c0;
        kv[u].load((old ? p.kv_state : p.kv) + at);
        score[u].load((old ? p.score_state : p.score) + at);
      }
    }
  };
  int next = s0;  // the first of the sequences that completes a block
  while (next < s1) {
    const StepSeq q(p, next);
    if (q.hi > q.lo && fine(q, next)) {
      fetch(q, q.lo);
      break;
    }
    ++next;
  }
  auto embed = [&]() {
#pragma unroll
    for (int u = 0; u < UW; ++u) {
      const int w = pg + u * p.PG;
      const bool prev = two && w < p.ratio;
      float e[4] = {};
      if (mine && w < p.W) {
        const float* from = p.ape + static_cast<int64_t>(prev || !two ? w : w - p.ratio) * p.C + (two && !prev ? p.d : 0) + c0;
        if constexpr (VEC == 4) load_ape<4>(e, from);
        else e[0] = __ldg(from);
      }
#pragma unroll
      for (int i = 0; i < Weighed<VEC>::kPairs; ++i) embedding[u][i] = f2_pack(e[2 * i], e[2 * i + 1]);
    }
  };
  if (next < s1) embed();
  // what goes into the states: lines / RS of them to a sequence, each the positions of its turn
  const int lines = p.PG / p.RS, ks = s0 + pg / lines;
  const StepSeq kq(p, min(ks, p.S - 1));
  const bool keeps = mine && ks < s1 && kq.target >= 0 && fine(kq, ks);
  const int end = kq.first + kq.n;
  auto keep_from = [&](int half) {
    const int keep = max(0, kq.hi - (p.coff - 1 - half)) * p.ratio;
    return (kq.source == kq.target ? max(keep, kq.first) : keep) + pg % lines;
  };
  auto keep_place = [&](int half, int pos) { return static_cast<int64_t>(pos % p.W) * p.C + half * p.d + c0; };
  auto keep_load = [&](int half, int pos, P& k, P& x) {
    const bool old = pos < kq.first;
    const int64_t from = old ? kq.source * state + keep_place(half, pos) : (kq.token0 + pos) * p.C + half * p.d + c0;
    k.load((old ? p.kv_state : p.kv) + from);
    x.load((old ? p.score_state : p.score) + from);
  };
  auto keep_store = [&](int half, int pos, const P& k, const P& x) {
    const int64_t to = kq.target * state + keep_place(half, pos);
    k.store(p.kv_state + to);
    x.store(p.score_state + to);
  };
  const int from0 = keeps ? keep_from(0) : end, from1 = keeps && two ? keep_from(1) : end;
  P k0, x0, k1, x1;
  if (from0 < end) keep_load(0, from0, k0, x0);
  if (from1 < end) keep_load(1, from1, k1, x1);

  rows = __reduce_add_sync(0xFFFFFFFFu, rows);
  shared = __reduce_add_sync(0xFFFFFFFFu, shared);
  if ((tid & 31) == 0) s_sums[tid >> 5] = make_uint2(rows, shared);
  const bool wrong = __syncthreads_or(bad) != 0;
  rows = shared = 0;
  for (int w = 0; w < static_cast<int>(blockDim.x) / 32; ++w) {
    rows += s_sums[w].x;
    shared += s_sums[w].y;
  }
  const int before = rows & 0x1FFF, all = rows >> 13;
  if (wrong || all > p.out_rows) {
    const int which = __syncthreads_or(bad & 1) ? CSA_DEVERR_CU_SEQLENS : wrong ? CSA_DEVERR_STATE : CSA_DEVERR_OUT_ROWS;
    if (tid == 0 && p.dev_error != nullptr) *reinterpret_cast<volatile int32_t*>(p.dev_error) = which;
    return;
  }
  const int wide = p.CL * VEC;
  const Join join(SPLIT ? p.PG : kStepJoin, wide);
  bool here = true;  // the window is there already
  auto entry = [&](const StepSeq& q, int block, int row) {
    if (!here) fetch(q, block);
    here = false;
    uint16_t* out = p.out + static_cast<int64_t>(row) * p.d;
    if (mine) {
      Weighed<VEC> r;
      r.template of<UW>(kv, score, embedding);
      if constexpr (SPLIT) {
        r.leave(s_part + join.place(pg, cl * VEC), join.step);
      } else {
        r.store(out + c0);
      }
    }
    if constexpr (SPLIT) {
      __syncthreads();
      for (int c0 = 0; c0 < wide; c0 += per / Join::kJ) {  // (as often for every lane)
        const int c = c0 + tid / Join::kJ, col = blockIdx.y * wide + c;
        join.column(s_part, min(c, wide - 1), tid < per && c < wide && col < p.d ? out + col : nullptr);
      }
      __syncthreads();
    }
  };
  for (int s = next, row = before; s < s1; ++s) {
    const StepSeq q(p, s);
    for (int block = q.lo; block < min(q.hi, q.lo + static_cast<int>(p.own_blocks)); ++block) entry(q, block, row + block - q.lo);
    row += q.hi - q.lo;
  }
  // (the states were read by this thread, or before the last barrier)
  if (from0 < end) keep_store(0, from0, k0, x0);
  if (from1 < end) keep_store(1, from1, k1, x1);
  for (int half = 0; half < p.coff && keeps; ++half)
    for (int pos0 = (half == 0 ? from0 : from1) + lines; pos0 < end; pos0 += 4 * lines) {
      P k[4], x[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (pos0 + i * lines < end) keep_load(half, pos0 + i * lines, k[i], x[i]);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (pos0 + i * lines < end) keep_store(half, pos0 + i * lines, k[i], x[i]);
    }
  if (shared > 0) {
    if (next >= s1) embed();  // (no sequence of this CTA's own has wanted it)
    here = false;
    if (tid < 32) {
      int2 sum = make_int2(0, 0);
      for (int i0 = 0; i0 < p.S; i0 += 32) {
        const int i = i0 + tid;
        int made = 0;
        if (i < p.S) {
          const int f = __ldg(p.first + i);
          made = (f + __ldg(p.cu + i + 1) - __ldg(p.cu + i)) / p.ratio - f / p.ratio;
        }
        int2 x = make_int2(made, max(0, made - static_cast<int>(p.own_blocks)));
        const int2 own = x;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int a = __shfl_up_sync(0xFFFFFFFFu, x.x, o), b = __shfl_up_sync(0xFFFFFFFFu, x.y, o);
          if (tid >= o) x.x += a, x.y += b;
        }
        if (i < p.S) s_rows[i] = make_int2(sum.x + x.x - own.x, sum.y + x.y - own.y);
        sum.x += __shfl_sync(0xFFFFFFFFu, x.x, 31);
        sum.y += __shfl_sync(0xFFFFFFFFu, x.y, 31);
      }
    }
    __syncthreads();
    for (int i = blockIdx.x; i < static_cast<int>(shared); i += p.R) {
      int s = 0, h = p.S;  // shared-out rows before s <= i < those before h, the last such s
      while (h - s > 1) {
        const int mid = (s + h) / 2;
        if (s_rows[mid].y <= i) s = mid;
        else h = mid;
      }
      const StepSeq q(p, s);
      const int nth = static_cast<int>(p.own_blocks) + i - s_rows[s].y;  // of the sequence's blocks
      entry(q, q.lo + nth, s_rows[s].x + nth);
    }
  }
  // where the rows go, by the last threads; those behind the last entry
  if (blockIdx.y != 0) return;
  const int back = static_cast<int>(blockDim.x) - 1 - tid;
  for (int s = s0, row = before; s < s1; ++s) {
    const int lo = __ldg(p.first + s) / p.ratio, hi = (__ldg(p.first + s) + __ldg(p.cu + s + 1) - __ldg(p.cu + s)) / p.ratio;
    for (int i = back; i < hi - lo; i += blockDim.x) describe_row(p, s, lo + i, row + i);
    if (back == 0 && p.entries != nullptr) p.entries[s] = max(0, hi - (p.base != nullptr ? __ldg(p.base + s) : 0));
    row += hi - lo;
  }
  for (int64_t o = all + static_cast<int64_t>(blockIdx.x) * blockDim.x + tid; o < p.out_rows; o += static_cast<int64_t>(p.R) * blockDim.x)
    no_row(p, o);
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
  const bool split = W > kStepFlight;
  const bool vec = d % 4 == 0 && is_aligned(kv, 8) && is_aligned(score, 8) && is_aligned(ape, 16) &&
                   is_aligned(kv_state, 8) && is_aligned(score_state, 8) && is_aligned(out, 8);
  p.chunks = vec ? d / 4 : d;
  // up to 8 positions a thread; longer windows between 4 threads and more (256 at most: CSA_MAX_WINDOW is 2048)
  p.PG = split ? kStepJoin : 1;
  while (p.PG * kStepFlight < p.W) p.PG *= 2;
  static_assert(kFewThreads == kStepThreads, "columns and lines of either kernel");
  const int most = kStepThreads / p.PG, slices = (p.chunks + most - 1) / most;
  p.CL = (p.chunks + slices - 1) / slices;
  if (slices > 65535) return CSA_ERR_UNSUPPORTED;
  void* args[] = {&p};
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  int dev = 0, sms = 0, bps = 0;
  if (note(cudaGetDevice(&dev)) != cudaSuccess || device_sms(dev, &sms) != cudaSuccess) return CSA_ERR_CUDA;
  // Few tokens a sequence: the kernel without a pipeline, a CTA a sequence, as long as all CTAs run at once (384 sequences by
  // one token, blocks of 4, coff 2, d 512 do not: 9.4 us, 8.7 by the other). By it and by the other one, in us, with 1
  // and 8 tokens in each of 64 sequences, and with single ones but for one of 65 and of 449 (the host knows their sum alone):
  //   blocks of 4, coff 2, d 512     5.1 and 6.9, 8.2 and 10.5,   8.0 and 8.7, 11.0 and 9.5
  //   blocks of 16, d 128            6.0 and 6.7, 6.4 and 7.2,    9.2 and 8.0, 9.2 and 9.3
  //   blocks of 128, coff 2, d 128   5.1 and 6.4, 6.9 and 8.7,    6.2 and 7.2, 10.8 and 10.5
  // of 256 sequences (and 257 and 1793 tokens)
  //                                  5.9 and 7.2, 10.3 and 11.8,  10.3 and 9.2, 14.4 and 10.6
  //                                  6.7 and 6.7, 7.2 and 7.4,    11.5 and 9.5, 11.5 and 10.0
  //                                  6.4 and 12.6, 10.4 and 15.7, 14.9 and 16.6, 18.0 and 16.4
  // More sequences only where windows are of up to 4 or more than 32 positions: 384 by 1 and 8 tokens, blocks of 1 and 64, d
  // 128: 6.7 and 8.7, 10.3 and 16.7; 7.7 and 9.2, 10.5 and 12.3. Blocks of 16, coff 1 and 2: 9.0 and 8.5, 11.0 and 9.3; 9.5
  // and 10.1, 13.1 and 11.8; of 4, coff 2: 7.4 and 7.9, 10.8 and 12.3, but of 512 8.7 and 8.2.
  if (S > 0 && S <= (W > 4 && W <= 32 ? kFewSeqs / 2 : kFewSeqs) && capacity <= kFewTokens * static_cast<int64_t>(S)) {
    auto pick = [&](auto v) -> const void* {
      constexpr int V = decltype(v)::value;
      return split      ? reinterpret_cast<const void*>(step_few_kernel<V, 8, true>)
             : p.W <= 4 ? reinterpret_cast<const void*>(step_few_kernel<V, 4, false>)
                        : reinterpret_cast<const void*>(step_few_kernel<V, 8, false>);
    };
    const void* k = vec ? pick(std::integral_constant<int, 4>{}) : pick(std::integral_constant<int, 1>{});
    // as many sequences a CTA as leave about two CTAs an SM, no more than have lines of threads of their own
    p.RS = 1;
    while (2 * p.RS <= p.PG && static_cast<int64_t>(S) * slices > 2 * static_cast<int64_t>(sms) * p.RS) p.RS *= 2;
    p.R = (S + p.RS - 1) / p.RS;
    const int block = p.CL * p.PG <= 64 ? 64 : (p.CL * p.PG + 31) / 32 * 32;
    if (blocks_per_sm(dev, k, block, 0, &bps) != cudaSuccess) return CSA_ERR_CUDA;
    if (static_cast<int64_t>(p.R + 1) * slices <= static_cast<int64_t>(sms) * bps) {
      p.own_blocks = (kFewTokens + ratio - 1) / ratio > 2 ? (kFewTokens + ratio - 1) / ratio : 2;
      p.checker = S > 1 ? p.R : UINT_MAX;
      return launch_pdl(k, dim3(p.R + (S > 1), slices), dim3(block), 0, cs, args) == cudaSuccess ? CSA_OK : CSA_ERR_CUDA;
    }
  }
  p.RS = kStepThreads / (p.CL * p.PG);
  const int uw = p.W > (split ? 16 : 4) ? 8 : p.W > 2 ? 4 : p.W > 1 ? 2 : 1;
  auto pick = [&](auto v) -> const void* {
    constexpr int V = decltype(v)::value;
    return split     ? (uw == 8 ? reinterpret_cast<const void*>(step_kernel<V, 8, true>) : reinterpret_cast<const void*>(step_kernel<V, 4, true>))
           : uw == 8 ? reinterpret_cast<const void*>(step_kernel<V, 8, false>)
           : uw == 4 ? reinterpret_cast<const void*>(step_kernel<V, 4, false>)
           : uw == 2 ? reinterpret_cast<const void*>(step_kernel<V, 2, false>)
                     : reinterpret_cast<const void*>(step_kernel<V, 1, false>);
  };
  const void* k = vec ? pick(std::integral_constant<int, 4>{}) : pick(std::integral_constant<int, 1>{});
  // Three turns under way, or as many as leave room for two CTAs an SM beside the sequences' numbers; a CTA an SM where
  // not one does (at most 155 KB of numbers and parts: one turn fits always).
  const int width = vec ? 4 : 1;
  const size_t fixed = sizeof(int2) * (static_cast<size_t>(S) + 1) + step_part_bytes(width, split), turn = step_stage_bytes(width);
  const size_t room_for = fixed + turn <= 112 * 1024 ? 112 * 1024 : 224 * 1024;
  p.stages = 3;
  while (p.stages > 1 && fixed + p.stages * turn > room_for) --p.stages;
  const size_t smem = fixed + p.stages * turn;
  if (blocks_per_sm(dev, k, kStepThreads, smem, &bps) != cudaSuccess) return CSA_ERR_CUDA;
  if (bps < 1) return CSA_ERR_UNSUPPORTED;
  const int64_t rows_at_once = p.RS * (split ? 1 : kStepFlight / uw), by_rows = (out_rows + rows_at_once - 1) / rows_at_once;
  const int64_t by_seqs = (S + p.RS - 1) / p.RS;
  const int64_t want = by_rows > by_seqs ? by_rows : by_seqs, room = static_cast<int64_t>(sms) * bps / slices;
  p.R = static_cast<int>(want < room ? (want > 0 ? want : 1) : (room > 0 ? room : 1));
  // Few sequences (a chunk's) have CTAs of their own, so that nobody comes late to the rows; many (single
  // tokens') are spread over all.
  p.seq_ctas = static_cast<int>(by_seqs < p.R ? (by_seqs > 0 ? by_seqs : 1) : p.R);
  p.first_row_cta = 4 * p.seq_ctas <= p.R ? p.seq_ctas : 0;
  // Sequences' own CTAs are done before those of rows, so the first one looks for states that sequences meet in; otherwise
  // an additional CTA does, which has the place of one of 32 and more (or else the first one before its own work; 12000
  // single tokens in blocks of 128, coff 2, d 128, with 38 CTAs a slice: 727 us, 759 in the first one's place).
  const bool added = S > 1 && p.first_row_cta == 0 && (p.R < room || p.R >= 32);
  if (added && p.R == room) {
    --p.R;
    p.seq_ctas = p.seq_ctas < p.R ? p.seq_ctas : p.R;
  }
  p.checker = S < 2 ? UINT_MAX : added ? p.R : 0;
  return launch_pdl(k, dim3(p.R + added, slices), dim3(kStepThreads), smem, cs, args) == cudaSuccess ? CSA_OK : CSA_ERR_CUDA;
}
