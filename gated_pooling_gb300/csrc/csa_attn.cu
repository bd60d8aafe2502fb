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
  const int64_t* work = few ? s_work : p.unit_first;
  // the unit and tile that a place in the work stands for, and how many tiles lie before it
  struct Place {
    int64_t unit, tile, before;
  };
  auto place = [&](int64_t x) {
    if (x >= all) return Place{units, 0, all - units * p.unit_cost};
    int64_t l = 0, h = units;  // work[l] <= x < work[h]
    while (h - l > 1) {
      const int64_t mid = (l + h) / 2;
      if (work[mid] <= x) l = mid;
      else h = mid;
    }
    const int64_t tile = x - work[l];
    if (tile >= work[l + 1] - work[l] - p.unit_cost) return Place{l + 1, 0, work[l + 1] - (l + 1) * p.unit_cost};  // behind the unit's last tile
    return Place{l, tile, x - l * p.unit_cost};
  };
  const AttnShares share(all, p.workers);
  for (int i = threadIdx.x; i < p.workers; i += kPlanThreads) {
    const Place a = place(share(i)), b = place(share(i + 1));
    AttnStart start{};
    start.left = b.before - a.before;
    if (start.left > 0) {
      start.u = p.units[a.unit];
      start.unit = static_cast<int32_t>(a.unit);
      start.tile = static_cast<int32_t>(a.tile);
      // a unit that begins in this share and goes on in later ones
      if (b.tile > 0 && (b.unit > a.unit || a.tile == 0)) {
        const int64_t end = work[b.unit + 1] - p.unit_cost;
        AttnJoin join{};
        join.u = p.units[b.unit];
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

// Scalar kernel, any d and alignment: a warp per new token and query head, a lane the columns
// lane, lane + 32, ...; one pass over the entries with the running maximum and sum.
constexpr int kScalarThreads = 128;
template <int FORMAT, int NL>
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
  const int n = visible(pos, p.ratio, p.entries[s]);
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
    const int page = p.table[static_cast<int64_t>(s) * p.max_pages + e / p.page_size];
    if (page < 0 || page >= p.num_pages) {
      if (p.dev_error != nullptr) *p.dev_error = CSA_DEVERR_PAGE;
      continue;
    }
    const int64_t entry = (static_cast<int64_t>(page) * p.page_size + e % p.page_size) * p.kv_heads + kvh;
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
const void* scalar_kernel_for(int format, int d) {
  auto pick = [&](auto f) -> const void* {
    constexpr int F = decltype(f)::value;
    return d <= 128   ? reinterpret_cast<const void*>(attn_scalar_kernel<F, 4>)
           : d <= 512 ? reinterpret_cast<const void*>(attn_scalar_kernel<F, 16>)
                      : reinterpret_cast<const void*>(attn_scalar_kernel<F, 32>);
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

template <typename F>
auto by_chunks(int chunks, F f) {
  return chunks == 2   ? f(std::integral_constant<int, 2>{})
         : chunks == 4 ? f(std::integral_constant<int, 4>{})
                       : f(std::integral_constant<int, 8>{});
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
  const size_t pieces = 2 * static_cast<size_t>(sms), dpad = tile_chunks(p.d) * 64;
  p.part_ml = reinterpret_cast<float*>(take(pieces * 2 * kAttnRows * sizeof(float)));
  p.part_o = reinterpret_cast<float*>(take(pieces * kAttnRows * dpad * sizeof(float)));
  if (chunks)
    p.packed = reinterpret_cast<uint16_t*>(take(static_cast<size_t>(p.S) * p.kv_heads * p.packed_rows * dpad * 2));
  return at;
}

// Sizes that the workspace depends on; d beyond the tile kernel's needs the status alone.
cudaError_t plan_sizes(AttnParams& p, int* sms, int32_t S, int64_t tokens, int32_t q_heads, int32_t kv_heads,
                       int32_t d, int64_t max_entries) {
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
  p.max_units = ((tokens * p.group + kAttnRows - 1) / kAttnRows + S) * kv_heads;
  p.packed_rows = static_cast<int>((max_entries + kAttnEntries - 1) / kAttnEntries * kAttnEntries);
  return cudaSuccess;
}

// Whether a call's chunks may be long enough for packed entries: kChunkRows rows (four units) a
// sequence on average, so that packing an entry (read and written once) is
// small beside the units that read it, and packed entries within kMaxPacked bytes. (The
// workspace has room for them then; the call decides, where it knows the cache.)
constexpr int64_t kChunkRows = 256, kChunkRowsWide = 384;
constexpr int64_t kMaxPacked = int64_t{4} << 30;
bool chunked(const AttnParams& p) {
  if (p.d > kTileMaxDim || p.S < 1 || p.tokens * p.group < kChunkRows * p.S) return false;
  const int64_t rows = static_cast<int64_t>(p.S) * p.kv_heads * p.packed_rows;
  return rows > 0 && rows < INT_MAX && rows * tile_chunks(p.d) * 128 <= kMaxPacked && p.S < 65536 && p.kv_heads < 65536;
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
  if (plan_sizes(p, &sms, S, tokens, q_heads, kv_heads, d, max_entries) != cudaSuccess) return 0;
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
  if (max_pages < 0 || page_size < 1 || num_pages < 0 || ratio < 0 || q_row_stride < 0 ||
      q_head_stride < 0 || out_row_stride < 0 || out_head_stride < 0 || !std::isfinite(softmax_scale))
    return CSA_ERR_INVALID_VALUE;
  const int64_t max_entries = static_cast<int64_t>(max_pages) * page_size;
  const csa_status_t st = check_attn_sizes(S, tokens, q_heads, kv_heads, d, max_entries);
  if (st != CSA_OK) return st;
  if (format < CSA_CACHE_BF16 || format > CSA_CACHE_E2M1) return CSA_ERR_UNSUPPORTED;
  if (format != CSA_CACHE_BF16 && d % CSA_CACHE_GROUP != 0) return CSA_ERR_UNSUPPORTED;
  if (num_pages > INT64_MAX / 64 / page_size / (static_cast<int64_t>(kv_heads) * d))
    return CSA_ERR_UNSUPPORTED;
  if (cu_seqlens == nullptr || (S > 0 && entries == nullptr)) return CSA_ERR_INVALID_VALUE;
  if (tokens > 0 && (q == nullptr || out == nullptr || !separate(tokens, q_heads, d, out_row_stride, out_head_stride)))
    return CSA_ERR_INVALID_VALUE;
  if (S > 0 && max_pages > 0 && page_table == nullptr) return CSA_ERR_INVALID_VALUE;
  if (num_pages > 0 && (data == nullptr || (format != CSA_CACHE_BF16 && scales == nullptr)))
    return CSA_ERR_INVALID_VALUE;
  if (!is_aligned(q, 2) || !is_aligned(out, 2) || !is_aligned(cu_seqlens, 4) ||
      !is_aligned(page_table, 4) || !is_aligned(entries, 4) || !is_aligned(first, 4) ||
      !is_aligned(sink, 4) || !is_aligned(lse, 4) || !is_aligned(dev_error, 4) ||
      !is_aligned(workspace, 16) || (format == CSA_CACHE_BF16 && !is_aligned(data, 2)))
    return CSA_ERR_INVALID_VALUE;
  if (S == 0 || tokens == 0) return CSA_OK;
  if (workspace == nullptr || workspace_bytes < kStatusBytes) return CSA_ERR_WORKSPACE;

  AttnParams p{};
  int sms = 0;
  if (plan_sizes(p, &sms, S, tokens, q_heads, kv_heads, d, max_entries) != cudaSuccess) return CSA_ERR_CUDA;
  // a call's pointers and strides decide between the kernels, its workspace serves either
  const bool tile = d <= kTileMaxDim && d % 8 == 0 && q_row_stride % 8 == 0 && q_head_stride % 8 == 0 &&
                    out_row_stride % 8 == 0 && out_head_stride % 8 == 0 && is_aligned(q, 16) &&
                    is_aligned(out, 16) && is_aligned(data, 16);
  if (d <= kTileMaxDim) {
    if (workspace_bytes < lay_out(p, sms, chunked(p), nullptr)) return CSA_ERR_WORKSPACE;
    lay_out(p, sms, chunked(p), static_cast<unsigned char*>(workspace));
  } else {
    p.head = static_cast<AttnHead*>(workspace);
  }
  if (!tile) p.units = nullptr;
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
  const int64_t most_tiles = p.max_units * ((max_entries + kAttnEntries - 1) / kAttnEntries);
  const bool copies = format == CSA_CACHE_BF16 && p.box_rows >= 8 && num_pages > 0 &&
                      num_pages <= INT_MAX / page_size && (nc < 8 || most_tiles <= p.workers);
  // Packing first. Up to d = 256 a tile's time is the softmax's, so packing entries that can be copied
  // from the pages gains little (3 chunks of 1024 tokens x 64 heads of 256: 450 us packed, 471 not)
  // or loses (48 of 8 tokens: 205 and 165). Codes are widened once instead of by every unit (450 and
  // 787), from 256 rows a sequence on at d = 128 (496 and 675), later above (256 rows of 256: 132
  // and 123, of 512: 255 and 227; 384 of 256: 160 and 169, of 512: 314 and 313; 512 of 256: 206 and
  // 232, of 512: 407 and 435). bf16 at d = 512: 256 rows 256 and 285, three chunks of 1024 tokens
  // 909 and 1382.
  const bool wide = format != CSA_CACHE_BF16 && d > 128;
  const bool chunks = tile && chunked(p) && !(copies && nc < 8) &&
                      tokens * p.group >= (wide ? kChunkRowsWide : kChunkRows) * S;
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
  p.q = static_cast<const uint16_t*>(q);
  p.cu = cu_seqlens;
  p.data = static_cast<const uint8_t*>(data);
  p.scales = scales;
  p.table = page_table;
  p.entries = entries;
  p.first = first;
  p.sink = sink;
  p.out = static_cast<uint16_t*>(out);
  p.lse = lse;
  p.dev_error = dev_error;
  p.q_row = q_row_stride;
  p.q_head = q_head_stride;
  p.out_row = out_row_stride;
  p.out_head = out_head_stride;
  p.num_pages = num_pages;
  p.max_pages = max_pages;
  p.page_size = page_size;
  p.ratio = ratio;
  p.scale = softmax_scale;
  p.wait_cycles = hooked_wait_cycles();
  p.withhold_tile = hooked_withhold();
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  void* args[] = {&p};
  int dev = 0, bps = 0;
  if (note(cudaGetDevice(&dev)) != cudaSuccess) return CSA_ERR_CUDA;
  const size_t plan_smem = sizeof(int) * (static_cast<size_t>(S) + 1);
  const void* plan = reinterpret_cast<const void*>(attn_plan_kernel);
  if (blocks_per_sm(dev, plan, kPlanThreads, plan_smem, &bps) != cudaSuccess) return CSA_ERR_CUDA;
  if (launch_pdl(plan, dim3(1), dim3(kPlanThreads), plan_smem, cs, args) != cudaSuccess) return CSA_ERR_CUDA;
  if (tile) {
    CUtensorMap map{};
    int source = format;
    if (chunks) {
      source = kFromPacked;
      const uint64_t dims[2] = {static_cast<uint64_t>(nc) * 64,
                                static_cast<uint64_t>(S) * kv_heads * static_cast<uint64_t>(p.packed_rows)};
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
    size_t smem = 0;
    int threads = 0;
    const void *k = nullptr, *join = nullptr, *pack = nullptr;
    by_chunks(nc, [&](auto c) {
      constexpr int NC = decltype(c)::value;
      smem = TileShape<NC>::kSmemBytes;
      auto use = [&](auto src) {
        constexpr int SRC = decltype(src)::value;
        k = reinterpret_cast<const void*>(attn_tile_kernel<NC, SRC>);
        threads = TileCta<SRC>::kThreads;
        join = reinterpret_cast<const void*>(attn_join_kernel<NC>);
        return 0;
      };
      if (source == kFromPacked) {
        use(std::integral_constant<int, kFromPacked>{});
        pack = by_format(format, [](auto f) {
          return reinterpret_cast<const void*>(attn_pack_kernel<NC, decltype(f)::value>);
        });
      } else if (source == kFromBoxes) {
        use(std::integral_constant<int, kFromBoxes>{});
      } else {
        by_format(format, use);
      }
      return 0;
    });
    if (blocks_per_sm(dev, k, threads, smem, &bps) != cudaSuccess) return CSA_ERR_CUDA;
    if (bps < 1) return CSA_ERR_UNSUPPORTED;
    if (chunks) {
      // a few blocks an SM, which go on to their sequence's next entries: the table's capacity may
      // be far above what the sequences hold
      const int64_t heads = static_cast<int64_t>(S) * kv_heads, most = p.packed_rows / kPackRows;
      const int64_t want = (16 * static_cast<int64_t>(sms) + heads - 1) / heads;
      if (launch_pdl(pack, dim3(static_cast<unsigned>(want < most ? want : most), S, kv_heads), dim3(kPackThreads), 0,
                     cs, args) != cudaSuccess)
        return CSA_ERR_CUDA;
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
  return launch_pdl(scalar_kernel_for(format, d), dim3(static_cast<unsigned>(blocks)),
                    dim3(kScalarThreads), 0, cs, args) == cudaSuccess
             ? CSA_OK
             : CSA_ERR_CUDA;
}
