// csa_attn.cu -- attention of new tokens over the paged cache of entries that are key and value
// at once (the interface and the formulas are in csa_compressor.h).
#include <climits>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "csa_compressor.h"
#include "csa_attn_tile.cuh"
#include "csa_internal.h"

namespace csa {
namespace {

// Sequence of a token, and -1 when it belongs to none (cu holds S + 1 non-decreasing offsets):
// the largest s with cu[s] <= t whose end lies behind t.
__device__ __forceinline__ int sequence_of(const int32_t* cu, int S, int64_t t) {
  if (t < cu[0] || t >= cu[S]) return -1;
  int lo = 0, hi = S;  // cu[lo] <= t < cu[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (cu[mid] <= t) lo = mid;
    else hi = mid;
  }
  return lo;
}

// Exclusive sum over the block, and the block's total (64 bits).
// (few threads: every warp walks through all of the plan's code, 1024 threads took 13 thousand
// cycles for 48 sequences)
constexpr int kPlanThreads = 256, kPlanUnits = 1024;
__device__ __forceinline__ int64_t plan_scan(int64_t v, int64_t* warps, int64_t& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xFFFFFFFFu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();
  if (lane == 31) warps[warp] = x;
  __syncthreads();
  if (warp == 0) {
    int64_t s = lane < kPlanThreads / 32 ? warps[lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xFFFFFFFFu, s, o);
      if (lane >= o) s += y;
    }
    warps[lane] = s;
  }
  __syncthreads();
  total = warps[31];
  return x - v + (warp > 0 ? warps[warp - 1] : 0);
}

// Where each worker's share of the units' work begins, and the units that several workers share. All threads
// of the plan's block; `work`: where each unit's work begins, `all` of them together.
// span_tile and held: behind prefixes the spans' first tiles and the units, where shared memory holds them. W: int
// where all of the work fits it.
template <typename W>
__device__ __forceinline__ void plan_shares(const AttnParams& p, W units, W all, const W* work, int* s_joins,
                                            const int* span_tile, const AttnUnit* held) {
  // the unit and tile that a place in the work stands for, and how many tiles lie before it
  struct Place {
    W unit, tile, before;
  };
  auto place = [&](W x) {
    if (x >= all) return Place{units, 0, all - units * p.unit_cost};
    W l = 0, h = units;  // work[l] <= x < work[h]
    while (h - l > 1) {
      const W mid = (l + h) / 2;
      if (work[mid] <= x) l = mid;
      else h = mid;
    }
    const W tile = x - work[l];
    if (tile >= work[l + 1] - work[l] - p.unit_cost) return Place{l + 1, 0, work[l + 1] - (l + 1) * p.unit_cost};  // behind the unit's last tile
    return Place{l, tile, x - l * p.unit_cost};
  };
  const AttnShares share(all, p.workers);
  for (int i = threadIdx.x; i < p.workers; i += kPlanThreads) {
    const Place a = place(static_cast<W>(share(i))), b = place(static_cast<W>(share(i + 1)));
    AttnStart start{};
    start.left = b.before - a.before;
    if (start.left > 0) {
      start.u = held != nullptr ? held[a.unit] : p.units[a.unit];
      start.unit = static_cast<int32_t>(a.unit);
      start.tile = static_cast<int32_t>(a.tile);
      if (p.groups > 0) {  // behind prefixes: the span that tile lies in
        int l = start.u.span, h = l + start.u.spans;
        while (h - l > 1) {
          const int mid = (l + h) / 2;
          if ((span_tile != nullptr ? span_tile[mid] : p.spans[mid].tile) <= start.tile) l = mid;
          else h = mid;
        }
        start.u.span = l;
      }
      // a unit that begins in this share and goes on in later ones
      if (b.tile > 0 && (b.unit > a.unit || a.tile == 0)) {
        const W end = work[b.unit + 1] - p.unit_cost;
        AttnJoin join{};
        join.u = held != nullptr ? held[b.unit] : p.units[b.unit];
        join.worker = i;
        int last = max(i + 1, share.near(end - 1));  // the worker whose share the unit's last tile lies in
        while (share(last + 1) < end) ++last;
        while (last > i + 1 && share(last) >= end) --last;
        join.pieces = last - i + 1;
        // (in any order: each is joined by itself; those of many pieces from the list's other end)
        const bool few = join.pieces <= kFewPieces;
        const int at = atomicAdd(&s_joins[few ? 0 : 1], 1);
        p.joins[few ? at : p.workers - 1 - at] = join;
      }
    }
    p.starts[i] = start;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    p.head->few = s_joins[0];
    p.head->many = s_joins[1];
  }
}

// Exclusive sums of two ints over the block, and the block's totals; all threads call it, sums: [kPlanThreads / 32].
__device__ __forceinline__ int2 plan_scan(int2 v, int2* sums, int2& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int2 x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int a = __shfl_up_sync(0xFFFFFFFFu, x.x, o), b = __shfl_up_sync(0xFFFFFFFFu, x.y, o);
    if (lane >= o) x.x += a, x.y += b;
  }
  if (lane == 31) sums[warp] = x;
  __syncthreads();
  int2 before = make_int2(x.x - v.x, x.y - v.y);
  total = make_int2(0, 0);
#pragma unroll
  for (int w = 0; w < kPlanThreads / 32; ++w) {
    const int2 t = sums[w];
    if (w < warp) before.x += t.x, before.y += t.y;
    total.x += t.x, total.y += t.y;
  }
  __syncthreads();
  return before;
}

// One block: checks the call's lengths, publishes the verdict for the kernels behind it, and
// (units wanted) lists the units, where each worker's share begins, and the units that several
// workers share.
__global__ void __launch_bounds__(kPlanThreads) attn_plan_kernel(AttnParams p) {
  extern __shared__ int s_first[];  // [S + 1] first row block of each sequence
  __shared__ int64_t s_warps[32];
  __shared__ int64_t s_work[kPlanUnits + 1];  // where the units' work begins, if there are no more
  __shared__ int s_joins[2];  // of few pieces, of many
  if (threadIdx.x < 2) s_joins[threadIdx.x] = 0;
  pdl_wait();
  const int per = (p.S + kPlanThreads - 1) / kPlanThreads;
  const int lo = min(p.S, static_cast<int>(threadIdx.x) * per), hi = min(p.S, lo + per);
  int bad = 0;
  int64_t mine = 0, blocks = 0;
  for (int s = lo; s < hi; ++s) {
    const int32_t a = __ldg(p.cu + s), b = __ldg(p.cu + s + 1), n = __ldg(p.entries + s);
    if (b < a || a < 0 || b > p.tokens) bad |= 1;
    else mine += ((b - a) * p.group + kAttnRows - 1) / kAttnRows;
    if (n < 0 || n > p.max_entries) bad |= 2;
  }
  int code = 0;
  if (__syncthreads_or(bad)) code = __syncthreads_or(bad & 1) ? CSA_DEVERR_CU_SEQLENS : CSA_DEVERR_ENTRIES;
  if (threadIdx.x == 0) {
    p.head->status = code;
    if (code != 0 && p.dev_error != nullptr) *p.dev_error = code;
  }
  if (code != 0 || p.units == nullptr) return;
  int64_t at = plan_scan(mine, s_warps, blocks);
  for (int s = lo; s < hi; ++s) {
    s_first[s] = static_cast<int>(at);
    at += (sequence_rows(p, s) + kAttnRows - 1) / kAttnRows;
  }
  if (threadIdx.x == 0) s_first[p.S] = static_cast<int>(blocks);
  __syncthreads();
  const int64_t units = blocks * p.kv_heads;
  const bool few = units <= kPlanUnits;
  int64_t all = 0;
  for (int64_t u0 = 0; u0 < units; u0 += kPlanThreads) {
    const int64_t i = u0 + threadIdx.x;
    AttnUnit u{};
    if (i < units) {
      const int b = static_cast<int>(units < INT_MAX ? static_cast<int>(i) / p.kv_heads : i / p.kv_heads);
      int l = 0, h = p.S;  // s_first[l] <= b < s_first[h]
      while (h - l > 1) {
        const int mid = (l + h) / 2;
        if (s_first[mid] <= b) l = mid;
        else h = mid;
      }
      u = make_unit(p, l, static_cast<int>(i - static_cast<int64_t>(b) * p.kv_heads), b - s_first[l]);
    }
    int64_t sum = 0;
    const int64_t first = all + plan_scan(i < units ? u.tiles + p.unit_cost : 0, s_warps, sum);
    if (i < units) {
      p.units[i] = u;
      p.unit_first[i] = first;
      if (few) s_work[i] = first;
    }
    all += sum;
  }
  if (threadIdx.x == 0) {
    p.unit_first[units] = all;
    if (few) s_work[units] = all;
  }
  __syncthreads();
  plan_shares<int64_t>(p, units, all, few ? s_work : p.unit_first, s_joins, nullptr, nullptr);
}

// The same behind shared prefixes: units of a group's rows, whatever sequences they are of, and their spans.
// `lanes` neighbouring threads work on a block of 64 rows, a sequence each (as many as single tokens have in
// one), and write its units of all cache heads. What is looked up again and again is held in shared
// memory: sequences' numbers where they fit beside the groups' (plan_cached), spans' first tiles up to kPlanSpans.
// (A thread a unit, which walked through its sequences three times, took 9 us for 64 sequences of 64 heads
// and 23 for 120 of 8.)
// SMALL: at most kSmallSeqs sequences and 32 groups, whose blocks go through in one round, and up to kSmallUnits
// units with all their work in 32 bits. There the plan's time is a chain of loads and code that runs once, so the
// loads come side by side, and nothing is 64 bits wide or read back from memory.
constexpr int kPlanSpans = 2048, kSmallSeqs = kPlanThreads, kSmallUnits = 256;
// (4096 sequences, fewer beside more than 12500 groups, whose numbers are held in any case)
__host__ __device__ constexpr bool plan_cached(int S, int G) { return S <= 4096 && S + G <= 16600; }
template <bool SMALL>
__global__ void __launch_bounds__(kPlanThreads) attn_prefix_plan_kernel(AttnParams p, int lanes) {
  using W = std::conditional_t<SMALL, int, int64_t>;
  extern __shared__ int s_mem[];
  __shared__ int64_t s_warps[32];
  __shared__ W s_work[(SMALL ? kSmallUnits : kPlanUnits) + 1];
  __shared__ W s_begin[kPlanThreads];  // of a round's blocks: where their units' work begins,
  __shared__ int s_span[kPlanThreads];       // their first spans,
  __shared__ int s_tiles[kPlanThreads], s_spans[kPlanThreads];  // and how many tiles and spans a unit has
  __shared__ int s_span_tile[kPlanSpans];
  __shared__ __align__(16) AttnUnit s_units[SMALL ? kSmallUnits : 1];
  __shared__ int s_joins[2];
  const int G = p.groups;
  int* s_first = s_mem;          // [groups + 1] first row block of each group
  int* s_seqs = s_first + G + 1;  // [groups + 1]
  int* s_prefix = s_seqs + G + 1;  // [groups]
  int* s_cu = s_prefix + G;
  int* s_own = s_cu + p.S + 1;
  int* s_pos = s_own + p.S;
  const bool cached = SMALL || plan_cached(p.S, G);
  if (threadIdx.x < 2) s_joins[threadIdx.x] = 0;
  pdl_wait();
  // (one block, which leaves room for the next kernel's: they set themselves up meanwhile, and wait for this one's
  // end before they read anything; 36.0 -> 34.8 us for 120 sequences of grouped heads)
  asm volatile("griddepcontrol.launch_dependents;");
  int bad = 0;
  auto group = [&](int g, int a, int b, int n) {
    if (a < 0 || b < a || b > p.S || (g == 0 && a != 0) || (g == G - 1 && b != p.S) || n < 0 || n > p.max_prefix) bad |= 4;
    s_seqs[g] = a;
    s_prefix[g] = n;
    if (g == G - 1) s_seqs[G] = b;
  };
  auto sequence_numbers = [&](int s, int a, int b, int n, int pos) {
    if (b < a || a < 0 || b > p.tokens) bad |= 1;
    if (n < 0 || n > p.max_entries) bad |= 2;
    if (cached) {
      s_cu[s] = a;
      if (s == p.S - 1) s_cu[s + 1] = b;
      s_own[s] = n;
      s_pos[s] = pos;
    }
  };
  if constexpr (SMALL) {
    const int t = threadIdx.x, s = min(t, p.S - 1), g = min(t, G - 1);
    const int a = __ldg(p.cu + s), b = __ldg(p.cu + s + 1), n = __ldg(p.entries + s), pos = p.first != nullptr ? __ldg(p.first + s) : 0;
    const int ga = __ldg(p.prefix_seqs + g), gb = __ldg(p.prefix_seqs + g + 1), gn = __ldg(p.prefix_entries + g);
    if (t < p.S) sequence_numbers(t, a, b, n, pos);
    if (t < G) group(t, ga, gb, gn);
  } else {
    for (int g = threadIdx.x; g < G; g += kPlanThreads)
      group(g, __ldg(p.prefix_seqs + g), __ldg(p.prefix_seqs + g + 1), __ldg(p.prefix_entries + g));
    for (int s = threadIdx.x; s < p.S; s += kPlanThreads)
      sequence_numbers(s, __ldg(p.cu + s), __ldg(p.cu + s + 1), __ldg(p.entries + s), p.first != nullptr ? __ldg(p.first + s) : 0);
  }
  const int32_t* const cu = cached ? s_cu : p.cu;
  const int32_t* const own = cached ? s_own : p.entries;
  const int32_t* const first = cached ? s_pos : p.first;
  int code = 0;
  if (__syncthreads_or(bad)) {
    code = __syncthreads_or(bad & 1) ? CSA_DEVERR_CU_SEQLENS : CSA_DEVERR_PREFIX;
    if (__syncthreads_or(bad & 2) && code == CSA_DEVERR_PREFIX) code = CSA_DEVERR_ENTRIES;
  }
  if (threadIdx.x == 0) {
    p.head->status = code;
    if (code != 0 && p.dev_error != nullptr) *p.dev_error = code;
  }
  if (code != 0 || p.units == nullptr) return;
  auto group_rows = [&](int g) { return (cu[s_seqs[g + 1]] - cu[s_seqs[g]]) * p.group; };
  W blocks = 0;
  if constexpr (SMALL) {
    if (threadIdx.x < 32) {
      const int g = threadIdx.x, mine = g < G ? (group_rows(g) + kAttnRows - 1) / kAttnRows : 0;
      int x = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xFFFFFFFFu, x, o);
        if (g >= o) x += y;
      }
      if (g < G) s_first[g] = x - mine;
      if (g == G - 1) s_first[G] = x;
    }
    __syncthreads();
    blocks = s_first[G];
  } else {
    const int per = (G + kPlanThreads - 1) / kPlanThreads;
    const int lo = min(G, static_cast<int>(threadIdx.x) * per), hi = min(G, lo + per);
    int64_t mine = 0;
    for (int g = lo; g < hi; ++g) mine += (group_rows(g) + kAttnRows - 1) / kAttnRows;
    int64_t at = plan_scan(mine, s_warps, blocks);
    for (int g = lo; g < hi; ++g) {
      s_first[g] = static_cast<int>(at);
      at += (group_rows(g) + kAttnRows - 1) / kAttnRows;
    }
    if (threadIdx.x == 0) s_first[G] = static_cast<int>(blocks);
    __syncthreads();
  }
  const W units = blocks * p.kv_heads;
  const bool few = SMALL || units <= kPlanUnits;
  W all = 0;
  int all_spans = 0;
  const int shift = __ffs(lanes) - 1, round = kPlanThreads >> shift, mine = threadIdx.x >> shift, lane = threadIdx.x & (lanes - 1);
  for (W b0 = 0; b0 < blocks; b0 += round) {
    const W b = b0 + mine;
    int g = 0, seq0 = 0, seq1 = -1, row0 = 0, before = 0, t0 = 0, t1 = 0, token = 0, rows = 0;
    if (b < blocks) {
      int h = G;  // s_first[g] <= b < s_first[h]
      while (h - g > 1) {
        const int mid = (g + h) / 2;
        if (s_first[mid] <= b) g = mid;
        else h = mid;
      }
      const int from = s_seqs[g], to = s_seqs[g + 1];
      token = cu[from];
      rows = group_rows(g);
      row0 = static_cast<int>(b - s_first[g]) * kAttnRows;
      t0 = token + row0 / p.group;
      t1 = token + (min(row0 + kAttnRows, rows) - 1) / p.group;
      auto sequence = [&](int t) {  // the last one of the group that begins by t: it holds t
        int l = from, r = to;
        while (r - l > 1) {
          const int mid = (l + r) / 2;
          if (cu[mid] <= t) l = mid;
          else r = mid;
        }
        return l;
      };
      seq0 = sequence(t0);
      seq1 = sequence(t1);
      before = s_prefix[g];
    }
    // what the block's tokens of sequence s see: all of them, and some
    auto sees = [&](int s, int& some, int& every) {
      const int a = cu[s], e = cu[s + 1];
      if (s > seq1 || a == e) return false;
      const int64_t pos = first != nullptr ? first[s] : 0;
      every = visible(pos + (max(a, t0) - a), p.ratio, before + own[s]);
      some = p.ratio == 0 ? every : visible(pos + (min(e - 1, t1) - a), p.ratio, before + own[s]);
      return true;
    };
    int own_tiles = 0, own_spans = 0, seen = 0, seen_all = INT_MAX;
    for (int s = seq0 + lane; s <= seq1; s += lanes) {
      int some, every;
      if (!sees(s, some, every)) continue;
      seen = max(seen, min(some, before));
      seen_all = min(seen_all, min(every, before));
      own_tiles += tiles_of(some - before);
      own_spans += some > before ? 1 : 0;
    }
    __syncwarp();
    for (int o = lanes / 2; o > 0; o >>= 1) {
      seen = max(seen, __shfl_xor_sync(0xFFFFFFFFu, seen, o));
      seen_all = min(seen_all, __shfl_xor_sync(0xFFFFFFFFu, seen_all, o));
      own_tiles += __shfl_xor_sync(0xFFFFFFFFu, own_tiles, o);
      own_spans += __shfl_xor_sync(0xFFFFFFFFu, own_spans, o);
    }
    // (a unit that sees nothing has a tile of nothing)
    const bool prefix = seen > 0 || own_tiles == 0;
    const int prefix_tiles = prefix ? max(1, tiles_of(seen)) : 0;
    if (lane == 0) {
      s_tiles[mine] = b < blocks ? own_tiles + prefix_tiles : 0;
      s_spans[mine] = b < blocks ? own_spans + (prefix ? 1 : 0) : 0;
    }
    __syncthreads();
    const bool holds = static_cast<int>(threadIdx.x) < round && b0 + threadIdx.x < blocks;
    if constexpr (SMALL) {
      int2 sum;
      const int2 at = plan_scan(holds ? make_int2((s_tiles[threadIdx.x] + p.unit_cost) * p.kv_heads, s_spans[threadIdx.x] * p.kv_heads)
                                      : make_int2(0, 0), reinterpret_cast<int2*>(s_warps), sum);
      all = sum.x;
      all_spans = sum.y;
      if (holds) {
        s_begin[threadIdx.x] = at.x;
        s_span[threadIdx.x] = at.y;
      }
    } else {
      int64_t sum = 0;
      const int64_t begin = all + plan_scan(holds ? static_cast<int64_t>(s_tiles[threadIdx.x] + p.unit_cost) * p.kv_heads : 0, s_warps, sum);
      all += sum;
      const int64_t span = all_spans + plan_scan(holds ? s_spans[threadIdx.x] * p.kv_heads : 0, s_warps, sum);
      all_spans += static_cast<int>(sum);
      if (holds) {
        s_begin[threadIdx.x] = begin;
        s_span[threadIdx.x] = static_cast<int>(span);
      }
    }
    __syncthreads();
    const int unit_tiles = s_tiles[mine], unit_spans = s_spans[mine], span0 = s_span[mine];
    auto put = [&](int at, AttnSpan v, int kvh, int packed) {  // the unit's span `at`
      v.tiles = max(1, tiles_of(v.seen));
      v.packed = packed;
      const int to = span0 + kvh * unit_spans + at;
      p.spans[to] = v;
      if (to < kPlanSpans) s_span_tile[to] = v.tile;
    };
    if (b < blocks && lane == 0) {
      AttnUnit u{};
      u.s = g;
      u.block = row0 / kAttnRows;
      u.tiles = unit_tiles;
      u.token = token;
      u.rows = rows;
      u.spans = unit_spans;
      AttnSpan v{};
      v.table = p.prefix_table + static_cast<int64_t>(g) * p.max_prefix_pages;
      v.seen = seen;
      v.seen_all = seen_all;
      v.row1 = kAttnRows;
      v.token = seq0;
      v.first = seq1;
      v.n = before;
      for (int kvh = 0; kvh < p.kv_heads; ++kvh) {
        const W i = b * p.kv_heads + kvh, at = s_begin[mine] + kvh * static_cast<W>(unit_tiles + p.unit_cost);
        u.kvh = kvh;
        u.span = span0 + kvh * unit_spans;
        p.units[i] = u;
        if constexpr (SMALL) s_units[i] = u;
        p.unit_first[i] = at;
        if (few) s_work[i] = at;
        if (prefix) put(0, v, kvh, (g * p.kv_heads + kvh) * p.prefix_rows);
      }
    }
    int tile = prefix_tiles, at = prefix ? 1 : 0;  // of the next of the lanes' sequences
    for (int s = seq0 + lane; __any_sync(0xFFFFFFFFu, s <= seq1); s += lanes) {
      int some = 0, every = 0;
      const bool has = s <= seq1 && sees(s, some, every) && some > before;
      const int mine_tiles = has ? tiles_of(some - before) : 0;
      int to_tile = mine_tiles, to_span = has ? 1 : 0;  // inclusive sums over the lanes
      for (int o = 1; o < lanes; o <<= 1) {
        const int x = __shfl_up_sync(0xFFFFFFFFu, to_tile, o, lanes), y = __shfl_up_sync(0xFFFFFFFFu, to_span, o, lanes);
        if (lane >= o) {
          to_tile += x;
          to_span += y;
        }
      }
      if (has) {
        AttnSpan v{};
        v.table = p.table + static_cast<int64_t>(s) * p.max_pages;
        v.tile = tile + to_tile - mine_tiles;
        v.seen = some - before;
        v.row0 = max(0, (cu[s] - token) * p.group - row0);
        v.row1 = s == seq1 ? kAttnRows : min(kAttnRows, (cu[s + 1] - token) * p.group - row0);
        v.seen_all = v.row0 == 0 && v.row1 == kAttnRows ? max(0, every - before) : 0;
        v.token = cu[s];
        v.first = first != nullptr ? first[s] : 0;
        v.n = before + own[s];
        v.before = before;
        v.own = 1;
        for (int kvh = 0; kvh < p.kv_heads; ++kvh)
          put(at + to_span - 1, v, kvh, G * p.kv_heads * p.prefix_rows + (s * p.kv_heads + kvh) * p.packed_rows);
      }
      tile += __shfl_sync(0xFFFFFFFFu, to_tile, lanes - 1, lanes);
      at += __shfl_sync(0xFFFFFFFFu, to_span, lanes - 1, lanes);
    }
    __syncthreads();
  }
  if (threadIdx.x == 0) {
    p.unit_first[units] = all;
    if (few) s_work[units] = all;
  }
  __syncthreads();
  const int* const span_tile = all_spans <= kPlanSpans ? s_span_tile : nullptr;
  if constexpr (SMALL) plan_shares<int>(p, units, all, s_work, s_joins, span_tile, s_units);
  else plan_shares<int64_t>(p, units, all, few ? s_work : p.unit_first, s_joins, span_tile, nullptr);
}

// Scalar kernel, any d and alignment: a warp per new token and query head, a lane the columns
// lane, lane + 32, ...; one pass over the entries with the running maximum and sum.
constexpr int kScalarThreads = 128;
template <int FORMAT, int NL, bool PREFIX>
__global__ void __launch_bounds__(kScalarThreads) attn_scalar_kernel(AttnParams p) {
  using B = Element<CSA_DTYPE_BF16>;
  const int lane = threadIdx.x & 31;
  pdl_wait();
  if (p.head->status != 0) return;
  const int64_t u = (static_cast<int64_t>(blockIdx.x) * kScalarThreads + threadIdx.x) / 32;
  if (u >= p.tokens * p.q_heads) return;
  const int64_t t = u / p.q_heads;
  const int h = static_cast<int>(u - t * p.q_heads);
  const int s = sequence_of(p.cu, p.S, t);
  if (s < 0) return;
  const int64_t pos = static_cast<int64_t>(p.first != nullptr ? p.first[s] : 0) + (t - p.cu[s]);
  // behind a prefix its entries come first
  int before = 0;
  const int32_t* table = p.table + static_cast<int64_t>(s) * p.max_pages;
  const int32_t* prefix = nullptr;
  if constexpr (PREFIX) {
    int lo = 0, hi = p.groups;  // the last group that begins by s: it holds s
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (p.prefix_seqs[mid] <= s) lo = mid;
      else hi = mid;
    }
    before = p.prefix_entries[lo];
    prefix = p.prefix_table + static_cast<int64_t>(lo) * p.max_prefix_pages;
  }
  const int n = visible(pos, p.ratio, before + p.entries[s]);
  const uint16_t* q = p.q + t * p.q_row + h * p.q_head;
  float qv[NL], acc[NL];
#pragma unroll
  for (int j = 0; j < NL; ++j) {
    const int c = lane + 32 * j;
    qv[j] = c < p.d ? B::to_float(q[c]) * p.scale : 0.f;
    acc[j] = 0.f;
  }
  float m = -INFINITY, z = 0.f;
  const int kvh = h / p.group;
  for (int e = 0; e < n; ++e) {
    const bool own = !PREFIX || e >= before;
    const int at = own ? e - before : e;
    const int page = own ? table[at / p.page_size] : prefix[at / p.page_size];
    if (page < 0 || page >= p.num_pages) {
      if (p.dev_error != nullptr) *p.dev_error = CSA_DEVERR_PAGE;
      continue;
    }
    const int64_t entry = (static_cast<int64_t>(page) * p.page_size + at % p.page_size) * p.kv_heads + kvh;
    float k[NL], x = 0.f;
#pragma unroll
    for (int j = 0; j < NL; ++j) {
      const int c = lane + 32 * j;
      k[j] = 0.f;
      if (c < p.d) {
        if constexpr (FORMAT == CSA_CACHE_BF16)
          k[j] = B::to_float(reinterpret_cast<const uint16_t*>(p.data)[entry * p.d + c]);
        else {
          const float sc = scale_value(p.scales[entry * (p.d / 32) + j]);
          if constexpr (FORMAT == CSA_CACHE_E4M3) {
            k[j] = e4m3x2_to_float2(p.data[entry * p.d + c]).x * sc;
          } else {
            const float2 two = e2m1x2_to_float2(p.data[entry * (p.d / 2) + c / 2]);
            k[j] = (lane % 2 == 0 ? two.x : two.y) * sc;
          }
        }
      }
      x = fmaf(qv[j], k[j], x);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, o);
    const float top = fmaxf(m, x);
    // a score of -inf adds nothing; while every score was -inf the maximum stays -inf
    const float old = m == top ? 1.f : expf(m - top), w = x == -INFINITY ? 0.f : expf(x - top);
    z = z * old + w;
#pragma unroll
    for (int j = 0; j < NL; ++j) acc[j] = acc[j] * old + w * k[j];
    m = top;
  }
  const float sink = p.sink != nullptr ? p.sink[h] : -INFINITY;
  const float top = fmaxf(m, sink);
  // a row that has seen an infinity or NaN has one in its sums (0 * inf where its weight was 0)
  bool odd = false;
#pragma unroll
  for (int j = 0; j < NL; ++j) odd = odd || acc[j] != acc[j];
  odd = __any_sync(0xFFFFFFFFu, odd);
  if (odd) {
#pragma unroll
    for (int j = 0; j < NL; ++j) acc[j] = __uint_as_float(0x7FFFFFFFu);
    z = acc[0];
  } else if (top != -INFINITY) {
    const float old = m == -INFINITY ? 0.f : expf(m - top);
    z = z * old + (sink == -INFINITY ? 0.f : sink == top ? 1.f : expf(sink - top));
    const float f = old / z;
#pragma unroll
    for (int j = 0; j < NL; ++j) acc[j] *= f;
  }
  uint16_t* out = p.out + t * p.out_row + h * p.out_head;
#pragma unroll
  for (int j = 0; j < NL; ++j) {
    const int c = lane + 32 * j;
    if (c < p.d) out[c] = B::from_float(acc[j]);
  }
  if (p.lse != nullptr && lane == 0) p.lse[u] = top == -INFINITY && !odd ? sink : top + logf(z);
}

template <typename F>
auto by_format(int format, F f) {
  return format == CSA_CACHE_BF16   ? f(std::integral_constant<int, CSA_CACHE_BF16>{})
         : format == CSA_CACHE_E4M3 ? f(std::integral_constant<int, CSA_CACHE_E4M3>{})
                                    : f(std::integral_constant<int, CSA_CACHE_E2M1>{});
}
template <bool PREFIX>
const void* scalar_kernel_for(int format, int d) {
  auto pick = [&](auto f) -> const void* {
    constexpr int F = decltype(f)::value;
    return d <= 128   ? reinterpret_cast<const void*>(attn_scalar_kernel<F, 4, PREFIX>)
           : d <= 512 ? reinterpret_cast<const void*>(attn_scalar_kernel<F, 16, PREFIX>)
                      : reinterpret_cast<const void*>(attn_scalar_kernel<F, 32, PREFIX>);
  };
  return by_format(format, pick);
}

csa_status_t check_attn_sizes(int32_t S, int64_t tokens, int32_t q_heads, int32_t kv_heads,
                              int32_t d, int64_t max_entries) {
  if (S < 0 || tokens < 0 || q_heads < 1 || kv_heads < 1 || d < 1 || max_entries < 0 ||
      q_heads % kv_heads != 0)
    return CSA_ERR_INVALID_VALUE;
  // (row numbers go up to a last unit's end in 32 bits)
  if (d > CSA_MAX_HEAD_DIM || S > CSA_MAX_SEGMENTS || tokens > (INT_MAX - 256) / q_heads ||
      max_entries > INT_MAX)
    return CSA_ERR_UNSUPPORTED;
  return CSA_OK;
}

constexpr size_t kStatusBytes = sizeof(AttnHead);
constexpr int kTileMaxDim = 512;

int tile_chunks(int d) { return d <= 128 ? 2 : d <= 256 ? 4 : 8; }

// Rows of all packed entries.
int64_t packed_rows(const AttnParams& p) {
  return (static_cast<int64_t>(p.groups) * p.prefix_rows + static_cast<int64_t>(p.S) * p.packed_rows) * p.kv_heads;
}

// The workspace: the plan, the pieces, and (chunks) the packed entries. base may be null (sizes only).
size_t lay_out(AttnParams& p, int sms, bool chunks, unsigned char* base) {
  size_t at = 0;
  auto take = [&](size_t bytes) {
    unsigned char* r = base == nullptr ? nullptr : base + at;
    at += (bytes + 255) & ~static_cast<size_t>(255);
    return r;
  };
  p.head = reinterpret_cast<AttnHead*>(take(kStatusBytes));
  p.starts = reinterpret_cast<AttnStart*>(take(sizeof(AttnStart) * sms));
  p.joins = reinterpret_cast<AttnJoin*>(take(sizeof(AttnJoin) * sms));
  p.units = reinterpret_cast<AttnUnit*>(take(sizeof(AttnUnit) * p.max_units));
  p.unit_first = reinterpret_cast<int64_t*>(take(sizeof(int64_t) * (p.max_units + 1)));
  if (p.groups > 0) p.spans = reinterpret_cast<AttnSpan*>(take(sizeof(AttnSpan) * p.max_spans));
  const size_t pieces = 2 * static_cast<size_t>(sms), dpad = tile_chunks(p.d) * 64;
  p.part_ml = reinterpret_cast<float*>(take(pieces * 2 * kAttnRows * sizeof(float)));
  p.part_o = reinterpret_cast<float*>(take(pieces * kAttnRows * dpad * sizeof(float)));
  if (chunks) p.packed = reinterpret_cast<uint16_t*>(take(static_cast<size_t>(packed_rows(p)) * dpad * 2));
  return at;
}

// Sizes that the workspace depends on; d beyond the tile kernel's needs the status alone.
cudaError_t plan_sizes(AttnParams& p, int* sms, int32_t S, int64_t tokens, int32_t q_heads, int32_t kv_heads,
                       int32_t d, int64_t max_entries, int32_t groups, int64_t max_prefix) {
  int dev = 0;
  cudaError_t e = note(cudaGetDevice(&dev));
  if (e != cudaSuccess || (e = device_sms(dev, sms)) != cudaSuccess) return e;
  p.S = S;
  p.tokens = tokens;
  p.q_heads = q_heads;
  p.kv_heads = kv_heads;
  p.group = q_heads / kv_heads;
  p.d = d;
  p.workers = *sms;
  p.max_entries = max_entries;
  p.groups = groups;
  p.max_prefix = max_prefix;
  const int64_t blocks = (tokens * p.group + kAttnRows - 1) / kAttnRows + (groups > 0 ? groups : S);
  p.max_units = blocks * kv_heads;
  p.max_spans = groups > 0 ? (2 * blocks + S) * kv_heads : 0;  // a prefix a unit, and a unit more or less for a sequence
  p.packed_rows = static_cast<int>((max_entries + kAttnEntries - 1) / kAttnEntries * kAttnEntries);
  p.prefix_rows = static_cast<int>((max_prefix + kAttnEntries - 1) / kAttnEntries * kAttnEntries);
  if (groups > 0 && p.prefix_rows == 0) p.prefix_rows = kAttnEntries;  // (a tile of nothing)
  return cudaSuccess;
}

// Whether a call's chunks may be long enough for packed entries: kChunkRows rows (four units) a
// sequence on average, so that packing an entry (read and written once) is
// small beside the units that read it, and packed entries within kMaxPacked bytes. (The
// workspace has room for them then; the call decides, where it knows the cache.)
constexpr int64_t kChunkRows = 256, kChunkRowsWide = 384;
constexpr int64_t kMaxPacked = int64_t{4} << 30;
bool chunked(const AttnParams& p) {
  if (p.d > kTileMaxDim || p.S < 1) return false;
  if (p.groups > 0) {
    // Behind prefixes: by the tiles that units read (a prefix's by each, own ones by each unit of a long sequence, or by
    // the one that several short ones share) and those that are packed, at the tables' capacity. Over codes, 64 sequences of 64
    // heads of 512 with up to 500 own entries behind 16384 take 176 us packed and 294 not; with 1000 behind 2048 46
    // and 51, with 2000 53 and 51; 4 sequences behind 16384 39.9 and 44.0, one 36.9 and 33.8; two chunks of up to 1500
    // tokens of 8 heads of 128 with up to 6000 own entries 203 and 357. Of 128 columns the first take 69 and 112, 100 of
    // 8 heads behind 4000 with 800 own ones 34.2 and 34.9.
    const int64_t units = (p.tokens * p.group + kAttnRows - 1) / kAttnRows;
    const int64_t tiles = p.prefix_rows / kAttnEntries, own = p.packed_rows / kAttnEntries;
    const int64_t reads = units * tiles + (units > p.S ? units : p.S) * own, packed = p.groups * tiles + p.S * own;
    if (reads < 2 * packed + 200) return false;
  } else if (p.tokens * p.group < kChunkRows * p.S) {
    return false;
  }
  const int64_t rows = packed_rows(p);
  return rows > 0 && rows < INT_MAX && rows * tile_chunks(p.d) * 128 <= kMaxPacked && p.S + p.groups < 65536 && p.kv_heads < 65536;
}

// A call of either entry point; groups is 0 without prefixes.
struct AttnCall {
  const void* q;
  int64_t q_row_stride, q_head_stride;
  const int32_t* cu_seqlens;
  int32_t S;
  int64_t tokens;
  int32_t q_heads, kv_heads, d;
  const void* data;
  const uint8_t* scales;
  int32_t format;
  const int32_t* prefix_seqs;
  int32_t groups;
  const int32_t* prefix_table;
  int32_t max_prefix_pages;
  const int32_t* prefix_entries;
  const int32_t* page_table;
  int32_t max_pages;
  int64_t num_pages;
  int32_t page_size;
  const int32_t *entries, *first;
  int32_t ratio;
  float softmax_scale;
  const float* sink;
  void* out;
  int64_t out_row_stride, out_head_stride;
  float* lse;
  void* workspace;
  size_t workspace_bytes;
  int32_t* dev_error;
};

csa_status_t run_attn(const AttnCall& c, csa_stream_t stream) {
  const int32_t S = c.S, q_heads = c.q_heads, kv_heads = c.kv_heads, d = c.d, format = c.format, groups = c.groups;
  const int32_t max_pages = c.max_pages, page_size = c.page_size;
  const int64_t tokens = c.tokens, num_pages = c.num_pages;
  const int64_t q_row_stride = c.q_row_stride, q_head_stride = c.q_head_stride;
  const int64_t out_row_stride = c.out_row_stride, out_head_stride = c.out_head_stride;
  const void *q = c.q, *data = c.data;
  void *out = c.out, *workspace = c.workspace;
  const uint8_t* scales = c.scales;
  const size_t workspace_bytes = c.workspace_bytes;
  if (max_pages < 0 || page_size < 1 || num_pages < 0 || c.ratio < 0 || q_row_stride < 0 ||
      q_head_stride < 0 || out_row_stride < 0 || out_head_stride < 0 || !std::isfinite(c.softmax_scale))
    return CSA_ERR_INVALID_VALUE;
  const int64_t max_entries = static_cast<int64_t>(max_pages) * page_size;
  const int64_t max_prefix = static_cast<int64_t>(c.max_prefix_pages) * page_size;
  const csa_status_t st = check_attn_sizes(S, tokens, q_heads, kv_heads, d, max_entries);
  if (st != CSA_OK) return st;
  if (groups > CSA_MAX_SEGMENTS || max_prefix > INT_MAX || max_entries + max_prefix > INT_MAX) return CSA_ERR_UNSUPPORTED;
  if (format < CSA_CACHE_BF16 || format > CSA_CACHE_E2M1) return CSA_ERR_UNSUPPORTED;
  if (format != CSA_CACHE_BF16 && d % CSA_CACHE_GROUP != 0) return CSA_ERR_UNSUPPORTED;
  if (num_pages > INT64_MAX / 64 / page_size / (static_cast<int64_t>(kv_heads) * d))
    return CSA_ERR_UNSUPPORTED;
  if (c.cu_seqlens == nullptr || (S > 0 && c.entries == nullptr)) return CSA_ERR_INVALID_VALUE;
  if (tokens > 0 && (q == nullptr || out == nullptr || !separate(tokens, q_heads, d, out_row_stride, out_head_stride)))
    return CSA_ERR_INVALID_VALUE;
  if (S > 0 && max_pages > 0 && c.page_table == nullptr) return CSA_ERR_INVALID_VALUE;
  if (num_pages > 0 && (data == nullptr || (format != CSA_CACHE_BF16 && scales == nullptr)))
    return CSA_ERR_INVALID_VALUE;
  if (!is_aligned(q, 2) || !is_aligned(out, 2) || !is_aligned(c.cu_seqlens, 4) ||
      !is_aligned(c.page_table, 4) || !is_aligned(c.entries, 4) || !is_aligned(c.first, 4) ||
      !is_aligned(c.sink, 4) || !is_aligned(c.lse, 4) || !is_aligned(c.dev_error, 4) ||
      !is_aligned(workspace, 16) || (format == CSA_CACHE_BF16 && !is_aligned(data, 2)))
    return CSA_ERR_INVALID_VALUE;
  if (S == 0 || tokens == 0) return CSA_OK;
  if (workspace == nullptr || workspace_bytes < kStatusBytes) return CSA_ERR_WORKSPACE;

  AttnParams p{};
  int sms = 0;
  if (plan_sizes(p, &sms, S, tokens, q_heads, kv_heads, d, max_entries, groups, max_prefix) != cudaSuccess) return CSA_ERR_CUDA;
  // a call's pointers and strides decide between the kernels, its workspace serves either
  const bool tile = d <= kTileMaxDim && d % 8 == 0 && q_row_stride % 8 == 0 && q_head_stride % 8 == 0 &&
                    out_row_stride % 8 == 0 && out_head_stride % 8 == 0 && is_aligned(q, 16) &&
                    is_aligned(out, 16) && is_aligned(data, 16);
  p.prefix_seqs = c.prefix_seqs;
  p.prefix_table = c.prefix_table;
  p.max_prefix_pages = c.max_prefix_pages;
  p.prefix_entries = c.prefix_entries;
  const int nc = tile_chunks(d);
  // bf16: tensor copies straight from the pages where a power of two of at least 8 entries
  // divides the page: smaller boxes copy slower than threads (8 entries 3.2 TB/s from L2,
  // 16 4.2, 64 and up 5.7). 48 sequences of up to 8192 entries, 8 heads of 128: 104 us against 165
  // by threads; 4 of 256: 91 against 134. At d > 256, where shared memory holds one tile,
  // the next one's copies wait for room that threads need not have (they load into registers):
  // 104 us against 79, so copies only if every share is about one tile (18.6 against 21.1 for one
  // token over 2048 entries). Codes come by threads, which have to widen them: copied first,
  // the same sequences took 32.5 instead of 32.0 us at d = 128, 45.9 instead of 45.6 at 256, and
  // 80.4 instead of 77.8 at 512.
  p.box_rows = 1;
  while (p.box_rows < kAttnEntries && page_size % (2 * p.box_rows) == 0) p.box_rows *= 2;
  const int64_t most_tiles = p.max_units * ((max_entries + max_prefix + kAttnEntries - 1) / kAttnEntries);
  const bool copies = format == CSA_CACHE_BF16 && p.box_rows >= 8 && num_pages > 0 &&
                      num_pages <= INT_MAX / page_size && (nc < 8 || groups > 0 || most_tiles <= p.workers);
  // Packing first. Up to d = 256 a tile's time is the softmax's, so packing entries that can be copied
  // from the pages gains little (3 chunks of 1024 tokens x 64 heads of 256: 450 us packed, 471 not)
  // or loses (48 of 8 tokens: 205 and 165). Codes are widened once instead of by every unit (450 and
  // 787), from 256 rows a sequence on at d = 128 (496 and 675), later above (256 rows of 256: 132
  // and 123, of 512: 255 and 227; 384 of 256: 160 and 169, of 512: 314 and 313; 512 of 256: 206 and
  // 232, of 512: 407 and 435). bf16 at d = 512: 256 rows 256 and 285, three chunks of 1024 tokens
  // 909 and 1382.
  const bool wide = format != CSA_CACHE_BF16 && d > 128;
  // Behind prefixes bf16 comes by copies at any d: the prefix's come from L2 (64 sequences of 64 heads of 512
  // behind 16384 entries: 164 us, by threads 280, packed 179; 48 with up to 8000 own entries behind 128: 46, packed
  // 103).
  const bool chunks = tile && chunked(p) && (groups > 0 ? !copies : !(copies && nc < 8) &&
                      tokens * p.group >= (wide ? kChunkRowsWide : kChunkRows) * S);
  // The places of packed entries come last: behind prefixes a call that does not pack works without them.
  if (d <= kTileMaxDim) {
    const bool packs = groups > 0 ? chunks : chunked(p);
    if (workspace_bytes < lay_out(p, sms, packs, nullptr)) return CSA_ERR_WORKSPACE;
    lay_out(p, sms, packs, static_cast<unsigned char*>(workspace));
  } else {
    p.head = static_cast<AttnHead*>(workspace);
  }
  if (!tile) p.units = nullptr;
  // A unit's own cost (q in, output out, the pipeline's start) in tiles, by which shares are evened
  // out, measured best of 1 to 5 or 6. Packed: three chunks of 1024 tokens x 64 heads of 512 910 us (at 3
  // 945, at 5 987), of 256 450 (at 1 513, at 5 468); 48 of 64 tokens x 8 heads of 128 100 (at 1
  // 112). Otherwise: 48 single tokens at d = 512 67.8 us (at 4 71.7), over codes of 256 40.4 (at 1
  // 41.3, at 6 42.1); where copies make the tiles short, 8 heads of 128, 78.3 us (at 1 98.2), and of
  // 128 tokens each 637 (at 1 815).
  p.unit_cost = copies && nc < 8 ? 5 : 2;
  if (chunks) {
    p.unit_cost = nc == 8 ? 1 : nc == 4 ? 3 : 5;
  }
  if (groups > 0) p.unit_cost = nc == 8 ? 2 : 3;
  p.q = static_cast<const uint16_t*>(q);
  p.cu = c.cu_seqlens;
  p.data = static_cast<const uint8_t*>(data);
  p.scales = scales;
  p.table = c.page_table;
  p.entries = c.entries;
  p.first = c.first;
  p.sink = c.sink;
  p.out = static_cast<uint16_t*>(out);
  p.lse = c.lse;
  p.dev_error = c.dev_error;
  p.q_row = q_row_stride;
  p.q_head = q_head_stride;
  p.out_row = out_row_stride;
  p.out_head = out_head_stride;
  p.num_pages = num_pages;
  p.max_pages = max_pages;
  p.page_size = page_size;
  p.ratio = c.ratio;
  p.scale = c.softmax_scale;
  p.wait_cycles = hooked_wait_cycles();
  p.withhold_tile = hooked_withhold();
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  void* args[] = {&p};
  int dev = 0, bps = 0;
  if (note(cudaGetDevice(&dev)) != cudaSuccess) return CSA_ERR_CUDA;
  const size_t plan_smem = sizeof(int) * (groups > 0 ? 3 * static_cast<size_t>(groups) + 2 + (plan_cached(S, groups) ? 3 * static_cast<size_t>(S) + 1 : 0)
                                                     : static_cast<size_t>(S) + 1);
  // behind prefixes: a thread for each sequence that single tokens would have in 64 rows, or twice as many as have
  // tokens there on average (4 sequences of 16384 tokens of one head of 64: 99 us, 398 with 32 threads a block; 64 of 64
  // tokens of 4 heads of 128 48 and 83)
  const int per_block = kAttnRows % p.group == 0 ? kAttnRows / p.group : kAttnRows / p.group + 2;
  int plan_lanes = 1;
  const int64_t most_blocks = p.max_units / kv_heads;
  while (plan_lanes < per_block && plan_lanes < 32 && plan_lanes * most_blocks < 2 * (most_blocks + S)) plan_lanes *= 2;
  const int64_t unit_most = (max_prefix + kAttnEntries - 1) / kAttnEntries + p.unit_cost +
                            kAttnRows * ((max_entries + kAttnEntries - 1) / kAttnEntries);
  const bool small = S <= kSmallSeqs && groups <= 32 && most_blocks * plan_lanes <= kPlanThreads && p.max_units <= kSmallUnits &&
                     p.max_units * unit_most < INT_MAX;
  const void* plan = groups == 0 ? reinterpret_cast<const void*>(attn_plan_kernel)
                     : small     ? reinterpret_cast<const void*>(attn_prefix_plan_kernel<true>)
                                 : reinterpret_cast<const void*>(attn_prefix_plan_kernel<false>);
  if (allow_shared(dev, plan) != cudaSuccess) return CSA_ERR_CUDA;
  void* plan_args[] = {&p, &plan_lanes};
  if (launch_pdl(plan, dim3(1), dim3(kPlanThreads), plan_smem, cs, plan_args) != cudaSuccess) return CSA_ERR_CUDA;
  if (tile) {
    CUtensorMap map{};
    int source = format;
    if (chunks) {
      source = kFromPacked;
      const uint64_t dims[2] = {static_cast<uint64_t>(nc) * 64,
                                static_cast<uint64_t>(packed_rows(p))};
      const uint64_t strides[1] = {static_cast<uint64_t>(nc) * 128};
      const uint32_t box[2] = {64, kAttnEntries};
      if (!encode_boxes(&map, p.packed, 2, dims, strides, box)) return CSA_ERR_CUDA;
    } else if (copies) {
      const uint64_t row = d;
      const uint64_t dims[3] = {row, static_cast<uint64_t>(kv_heads), static_cast<uint64_t>(num_pages) * page_size};
      const uint64_t strides[2] = {row * 2, row * 2 * kv_heads};
      const uint32_t box[3] = {64, 1, static_cast<uint32_t>(p.box_rows)};
      if (!encode_boxes(&map, data, 3, dims, strides, box)) return CSA_ERR_CUDA;
      source = kFromBoxes;
    }
    const TileKernels kernels = groups > 0 ? prefix_tile_kernels(nc, source, format) : tile_kernels<false>(nc, source, format);
    const void *k = kernels.tile, *join = kernels.join, *pack = kernels.pack;
    const size_t smem = kernels.smem;
    const int threads = kernels.threads;
    if (blocks_per_sm(dev, k, threads, smem, &bps) != cudaSuccess) return CSA_ERR_CUDA;
    if (bps < 1) return CSA_ERR_UNSUPPORTED;
    if (chunks) {
      // a few blocks an SM, which go on to their sequence's next entries: the table's capacity may
      // be far above what the sequences hold (behind prefixes a grid over all capacities, 33 thousand blocks for
      // 64 sequences, took 46 us)
      const int rows = pack_rows(nc, groups > 0);
      const int64_t heads = static_cast<int64_t>(S) * kv_heads, most = p.packed_rows / rows;
      int64_t want = (16 * static_cast<int64_t>(sms) + heads - 1) / heads;
      want = want < most ? want : most;
      dim3 grid(static_cast<unsigned>(want), S, kv_heads);
      int prefix_blocks = 0;
      if (groups > 0) {
        const int64_t steps = static_cast<int64_t>(groups) * kv_heads * (p.prefix_rows / rows);
        prefix_blocks = static_cast<int>(steps < 8 * sms ? steps : 8 * sms);
        want = (4 * static_cast<int64_t>(sms) + heads - 1) / heads;
        want = want < most ? want : most;
        grid = dim3(static_cast<unsigned>(prefix_blocks + want * heads));
      }
      void* pack_args[] = {&p, &prefix_blocks};
      if (launch_pdl(pack, grid, dim3(kPackThreads), 0, cs, pack_args) != cudaSuccess) return CSA_ERR_CUDA;
    }
    void* targs[] = {&p, &map};
    if (launch_pdl(k, dim3(p.workers), dim3(threads), smem, cs, targs) != cudaSuccess)
      return CSA_ERR_CUDA;
    return launch_pdl(join, dim3(kJoinBlocks * sms), dim3(kJoinThreads), 0, cs, args) == cudaSuccess
               ? CSA_OK
               : CSA_ERR_CUDA;
  }
  const int64_t warps = tokens * q_heads;
  const int64_t blocks = (warps + kScalarThreads / 32 - 1) / (kScalarThreads / 32);
  return launch_pdl(groups > 0 ? scalar_kernel_for<true>(format, d) : scalar_kernel_for<false>(format, d), dim3(static_cast<unsigned>(blocks)),
                    dim3(kScalarThreads), 0, cs, args) == cudaSuccess
             ? CSA_OK
             : CSA_ERR_CUDA;
}

}  // namespace
}  // namespace csa

using namespace csa;

extern "C" size_t csa_cache_attn_workspace_bytes(int32_t S, int64_t tokens, int32_t q_heads,
                                                 int32_t kv_heads, int32_t d, int64_t max_entries) {
  if (check_attn_sizes(S, tokens, q_heads, kv_heads, d, max_entries) != CSA_OK) return 0;
  if (d > kTileMaxDim) return kStatusBytes;
  AttnParams p{};
  int sms = 0;
  if (plan_sizes(p, &sms, S, tokens, q_heads, kv_heads, d, max_entries, 0, 0) != cudaSuccess) return 0;
  return lay_out(p, sms, chunked(p), nullptr);
}

extern "C" csa_status_t csa_cache_attn(
    const void* q, int64_t q_row_stride, int64_t q_head_stride, const int32_t* cu_seqlens, int32_t S,
    int64_t tokens, int32_t q_heads, int32_t kv_heads, int32_t d, const void* data,
    const uint8_t* scales, int32_t format, const int32_t* page_table, int32_t max_pages,
    int64_t num_pages, int32_t page_size, const int32_t* entries, const int32_t* first,
    int32_t ratio, float softmax_scale, const float* sink, void* out, int64_t out_row_stride,
    int64_t out_head_stride, float* lse, void* workspace, size_t workspace_bytes,
    int32_t* dev_error, csa_stream_t stream) {
  return run_attn({q, q_row_stride, q_head_stride, cu_seqlens, S, tokens, q_heads, kv_heads, d, data, scales, format,
                   nullptr, 0, nullptr, 0, nullptr, page_table, max_pages, num_pages, page_size, entries, first,
                   ratio, softmax_scale, sink, out, out_row_stride, out_head_stride, lse, workspace, workspace_bytes,
                   dev_error},
                  stream);
}

extern "C" size_t csa_cache_attn_prefix_workspace_bytes(int32_t S, int32_t G, int64_t tokens, int32_t q_heads,
                                                        int32_t kv_heads, int32_t d, int64_t max_entries,
                                                        int64_t max_prefix_entries) {
  if (check_attn_sizes(S, tokens, q_heads, kv_heads, d, max_entries) != CSA_OK) return 0;
  if (G < 0 || (G == 0 && S > 0) || G > CSA_MAX_SEGMENTS || max_prefix_entries < 0 || max_prefix_entries > INT_MAX ||
      max_entries + max_prefix_entries > INT_MAX)
    return 0;
  if (d > kTileMaxDim || G == 0) return kStatusBytes;
  AttnParams p{};
  int sms = 0;
  if (plan_sizes(p, &sms, S, tokens, q_heads, kv_heads, d, max_entries, G, max_prefix_entries) != cudaSuccess) return 0;
  return lay_out(p, sms, chunked(p), nullptr);
}

extern "C" csa_status_t csa_cache_attn_prefix(
    const void* q, int64_t q_row_stride, int64_t q_head_stride, const int32_t* cu_seqlens, int32_t S,
    int64_t tokens, int32_t q_heads, int32_t kv_heads, int32_t d, const void* data,
    const uint8_t* scales, int32_t format, const int32_t* prefix_seqs, int32_t G, const int32_t* prefix_table,
    int32_t max_prefix_pages, const int32_t* prefix_entries, const int32_t* page_table, int32_t max_pages,
    int64_t num_pages, int32_t page_size, const int32_t* entries, const int32_t* first,
    int32_t ratio, float softmax_scale, const float* sink, void* out, int64_t out_row_stride,
    int64_t out_head_stride, float* lse, void* workspace, size_t workspace_bytes,
    int32_t* dev_error, csa_stream_t stream) {
  if (G < 0 || max_prefix_pages < 0 || (G == 0 && S > 0)) return CSA_ERR_INVALID_VALUE;
  if (G > 0 && (prefix_seqs == nullptr || prefix_entries == nullptr || (max_prefix_pages > 0 && prefix_table == nullptr)))
    return CSA_ERR_INVALID_VALUE;
  if (!is_aligned(prefix_seqs, 4) || !is_aligned(prefix_table, 4) || !is_aligned(prefix_entries, 4))
    return CSA_ERR_INVALID_VALUE;
  return run_attn({q, q_row_stride, q_head_stride, cu_seqlens, S, tokens, q_heads, kv_heads, d, data, scales, format,
                   prefix_seqs, G, prefix_table, max_prefix_pages, prefix_entries, page_table, max_pages, num_pages,
                   page_size, entries, first, ratio, softmax_scale, sink, out, out_row_stride, out_head_stride, lse,
                   workspace, workspace_bytes, dev_error},
                  stream);
}
