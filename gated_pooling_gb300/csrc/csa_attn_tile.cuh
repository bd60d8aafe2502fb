// csa_attn_tile.cuh -- cache attention on the tensor cores (d a multiple of 8 up to 512, 16-byte
// aligned rows).
//
// A unit's 64 rows (new tokens x the heads that share a cache head) go over tiles of 128
// entries; everything is computed transposed, with the entries (and then the columns of an
// entry) along the tensor cores' 128 rows:
//     S^T [128 entries, 64 rows] = K [128, d] Q^T          P^T = 2^(S^T scale log2e - m)
//     O^T [128 columns, 64 rows] += (V^T = K^T) [128 columns, 128 entries] P^T, d/128 times
// so one entry tile in shared memory, 128-byte swizzled, is both products' A operand (along its
// rows, then along its columns) and is read from memory once, and O^T (d/2 tensor-memory
// columns) leaves room for S^T at d = 512, where O with the rows along M would fill the tensor
// memory. With few rows per sequence (decoding) no part of the 128 rows is idle.
//
// Warps: 0-15 softmax (a warp reads the 32 tensor-memory lanes of its quadrant, each group of
// four warps 16 of the 64 rows), 16 issues the products, 17 the tensor copies where the tile comes
// by those (18 and 19 only complete the register group); otherwise 20-27 fetch: they follow the
// page table, widen 8- and 4-bit codes to bf16 (exact, but for bf16's own subnormals) and store
// the swizzled tile in pairs of 64-column chunks (32 KB). Two groups of four warps take alternate
// pairs: a group holds its next pair in registers while the ring is full, and one group's loads
// are under way while the other stores. At d > 256 the ring holds one tile only, so fetching is
// part of a chain with the products and the softmax; the softmax warps, idle meanwhile, fetch
// half of the tile's codes (48 sequences of up to 8192 8-bit entries of 512: 84 us without, 78 with).
//
// Softmax without a maximum per tile: the weights are taken against a running bound m that
// only moves when some score passes it by 2^8; then m becomes the true maximum and O^T and the
// sums are rescaled. Weights up to 2^8 lose nothing (bf16 and fp32 are floating), and the sums
// stay per lane until the end of the unit.
//
// Between units: the next one's q is copied in as soon as the last scores are there, so that its
// first scores are computed while the softmax warps bring this one's output out (7.3 thousand
// cycles from the last sums to the next softmax instead of 13).
//
// Shared memory's 128 bytes a cycle bound the products (6 KB for 32 cycles' worth of them at 64
// rows), HBM the decoding of a long cache.
#pragma once

#include <climits>
#include <type_traits>

#include "csa_attn.cuh"
#include "csa_tcgen05.cuh"

namespace csa {

constexpr int kTileSoftWarps = 16, kTileLoadWarps = 8;
constexpr int kSoftThreads = kTileSoftWarps * 32;
constexpr int kSoftCols = 16;  // rows of a softmax thread's group
constexpr int kTileLoaders = kTileLoadWarps * 32;
constexpr int kTileFirstLoader = kTileSoftWarps + 4;
// Where a tile comes from: threads that read the pages (in each of the cache's formats); tensor
// copies of the pages' bf16 boxes; or tensor copies of a sequence's packed entries.
enum TileSource {
  kFromBf16 = CSA_CACHE_BF16,
  kFromE4m3 = CSA_CACHE_E4M3,
  kFromE2m1 = CSA_CACHE_E2M1,
  kFromBoxes,
  kFromPacked
};
template <int SRC>
struct TileCta {
  static constexpr bool kByThreads = SRC < kFromBoxes;
  static constexpr int kThreads = (kTileFirstLoader + (kByThreads ? kTileLoadWarps : 0)) * 32;
};
// Registers a thread: 896 threads launch with 72, and 16 x 64 + 4 x 40 + 8 x 104 = 28 x 72.
constexpr int kSoftRegs = 64, kIssueRegs = 40, kLoadRegs = 104;
constexpr int kChunkBytes = kAttnEntries * 128;  // 128 entries x 64 columns
constexpr int kPairBytes = 2 * kChunkBytes;
constexpr int kSmallBytes = 11776;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kNoMax = -3.4028234e38f;  // bound of a row that has seen nothing: no score lies below it
constexpr float kRescaleAt = 8.f;    // log2 of how far a weight may pass 1

// NC: 64-column chunks of an entry (2, 4, 8).
template <int NC>
struct TileShape {
  static constexpr int kPairs = NC / 2;
  static constexpr int kRing = NC == 8 ? 4 : 5;  // pairs in shared memory
  static constexpr bool kAhead = kRing >= 2 * kPairs;  // the next tile's scores before this one's sums
  static constexpr int kQBytes = NC * kAttnRows * 128;
  static constexpr int kPBytes = kAttnEntries * 128;
  static constexpr int kTmemO = 0, kTmemS = kPairs * kAttnRows;
  static constexpr int kTmemUsed = kTmemS + 2 * kAttnRows;
  static constexpr int kTmemColumns = kTmemUsed <= 256 ? 256 : 512;
  static constexpr int kDpad = NC * 64;
  // Codes, and a ring that holds one tile only, so that nobody else has work until the next one is
  // widened: the softmax warps take the second half of its pairs.
  template <int SRC>
  static constexpr bool kHelped = (SRC == kFromE4m3 || SRC == kFromE2m1) && kRing == kPairs;
  // shared memory: ring, Q, P (the output's staging too), then the small arrays
  static constexpr int kQOff = kRing * kPairBytes;
  static constexpr int kPOff = kQOff + kQBytes;
  static constexpr int kSmallOff = kPOff + kPBytes;
  static constexpr int kSmemBytes = kSmallOff + kSmallBytes + 1024;  // and the 1024-byte alignment
};

struct TileSmall {
  int64_t row[2][2][kAttnEntries];  // by fetching group and turn: bytes to an entry in the pool, -1: none
  int64_t help_row[2][kAttnEntries];   // the same for the softmax warps that widen
  int64_t q_at[kAttnRows];          // elements to a row of q, -1: none
  int64_t out_at[2][kAttnRows];     // and of out (this unit's and the next one's, as all with [2] here)
  AttnUnit next;                    // the worker's next unit
  float sink[2][kAttnRows];
  int32_t lse_at[2][kAttnRows];
  float m[kAttnRows];  // the rows' bounds (by copies: negated, as the sums two at a time want them)
  float fac[kAttnRows];
  float red[4][kAttnRows];  // column maxima, then weight sums, by quadrant
  int lim[2][kAttnRows];
  uint32_t odd[kAttnEntries];  // tile (counted from 1) in which an entry of this place was found not to be finite
  uint64_t full[5], empty[5], scores[2], probs, summed, q_full, drain;
  uint32_t tmem;
  int stop;
};
static_assert(sizeof(TileSmall) <= kSmallBytes, "small arrays");

__device__ __forceinline__ void sts128(uint32_t addr, uint4 v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
               : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
  return v;
}

// What a fetching thread takes of a pair (128 entries x 128 columns), from loading to the
// swizzled tile. `at` is an entry's byte offset in the pool, -1 for none. A bf16 thread takes 8
// columns of 16 entries (neighbouring lanes neighbouring columns); with codes it takes 32
// columns, a scale's, of 4 entries, so that finding a place and its scale is paid once per 32
// values: a fetch of 8-bit entries in pieces of 8 took 1100 instructions a pair and thread
// instead of about 400, and was bound by them.
//
// Codes become bf16 by moving their bits: sign, exponent and mantissa go where bf16 has its own,
// which is the code's value times 2^-120 (e4m3) or 2^-126 (e2m1), its subnormals among bf16's
// subnormals, and one bf16 product with 2^120 (2^126) times the scale makes the value. Without a
// branch, for the scales up to 2^7 (2^1) whose factor is within bf16's range, and no NaN
// among the codes; anything else goes through fp32, code by code. (The conversion
// instructions, 16 lanes a cycle each, took 2.2 thousand cycles for the two pairs under way.)
// Two bytes of (w, v), each below a byte of its top bit's copies: a code at the lower end of its
// half with its sign already above it, so that one shift and one mask place both.
template <int SELECT>
__device__ __forceinline__ uint32_t signed_pair(uint32_t w, uint32_t v) {
  uint32_t x;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(x) : "r"(w), "r"(v), "n"(SELECT));
  return x;
}
template <int FORMAT>
struct Widen {
  static constexpr uint32_t kLift = FORMAT == CSA_CACHE_E4M3 ? 120 : 126;
  static __device__ __forceinline__ bool plain(uint32_t k) { return k <= 254u - kLift; }
  __nv_bfloat162 f;
  __device__ __forceinline__ explicit Widen(uint32_t k) {
    const uint32_t b = (k + kLift) << 7 | (k + kLift) << 23;
    f = *reinterpret_cast<const __nv_bfloat162*>(&b);
  }
  __device__ __forceinline__ uint32_t two(uint32_t bits) const {
    const __nv_bfloat162 v = __hmul2(*reinterpret_cast<__nv_bfloat162*>(&bits), f);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
  // 8 e4m3 codes
  __device__ __forceinline__ uint4 eight(uint32_t w, uint32_t v) const {
    auto at = [&](uint32_t x) { return two((x << 4) & 0x87F087F0u); };
    return make_uint4(at(signed_pair<0x9180>(w, 0)), at(signed_pair<0xB3A2>(w, 0)), at(signed_pair<0x9180>(v, 0)),
                      at(signed_pair<0xB3A2>(v, 0)));
  }
  // 8 e2m1 codes
  __device__ __forceinline__ uint4 eight(uint32_t w) const {
    const uint32_t lo = w << 4;  // each byte's low code to its top, as w has the high one
    auto at = [&](uint32_t x) { return two((x << 2) & 0x81C081C0u); };
    return make_uint4(at(signed_pair<0xC480>(lo, w)), at(signed_pair<0xD591>(lo, w)), at(signed_pair<0xE6A2>(lo, w)),
                      at(signed_pair<0xF7B3>(lo, w)));
  }
};
// Bits left where a word holds an e4m3 NaN.
__device__ __forceinline__ uint32_t e4m3_nans(uint32_t w) { return ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u; }
// Any codes at any scale, by fp32 (exact but for bf16's own subnormals).
__device__ __forceinline__ uint4 widen_any(uint32_t w, uint32_t v, float s) {
  uint32_t r[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = e4m3x2_to_float2(((i < 2 ? w : v) >> (16 * (i % 2))) & 0xFFFFu);
    r[i] = pack_bf16x2(f.x * s, f.y * s);
  }
  return make_uint4(r[0], r[1], r[2], r[3]);
}
__device__ __forceinline__ uint4 widen_any(uint32_t w, float s) {
  uint32_t r[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = e2m1x2_to_float2(w >> (8 * i));
    r[i] = pack_bf16x2(f.x * s, f.y * s);
  }
  return make_uint4(r[0], r[1], r[2], r[3]);
}
__device__ __forceinline__ uint32_t fma_bf16x2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}
// Weight of a sink (in log2) at the row's maximum, which it may be, an infinite one too.
__device__ __forceinline__ float sink_weight(float sink, float mx) { return sink == mx ? 1.f : fast_exp2(sink - mx); }
// 16 bytes, or zeros, into shared memory without a register.
__device__ __forceinline__ void copy16(uint32_t to, const void* from, bool some) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(some ? 16 : 0) : "memory");
}
constexpr uint32_t kNoScale = 0;  // no entry here: zeros at any scale
template <int FORMAT>
struct Take;
template <>
struct Take<CSA_CACHE_BF16> {
  static constexpr int kRows = 16, kRowStep = 8;  // entries row, row + 8, ...
  static __device__ __forceinline__ int row_bytes(int d) { return 2 * d; }
  static __device__ __forceinline__ int first_row(int t) { return t >> 4; }
  static __device__ __forceinline__ int column(int t) { return (t & 15) * 8; }
  uint4 w;
  __device__ __forceinline__ void load(const AttnParams& p, int64_t at, int col) {
    w = make_uint4(0, 0, 0, 0);
    if (at >= 0 && col < p.d) w = __ldg(reinterpret_cast<const uint4*>(p.data + at + 2 * col));
  }
  __device__ __forceinline__ void store(uint32_t pair, int row, int t) const {
    const int piece = t & 15;
    sts128(pair + (piece >> 3) * kChunkBytes + row * 128 + (((piece & 7) ^ (row & 7)) << 4), w);
  }
};
// Four pieces of 8 columns from a thread's 32. Lanes of the pair's second half (other chunk, same
// banks) take theirs in another order, so that eight neighbouring lanes use all banks.
template <typename F>
__device__ __forceinline__ void store_pieces(uint32_t pair, int row, int t, F widened) {
  const int g = t & 3;
  const uint32_t to = pair + (g >> 1) * kChunkBytes + row * 128;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int piece = (g & 1) * 4 + (i ^ (g & 2));
    sts128(to + ((piece ^ (row & 7)) << 4), widened(i));
  }
}
template <>
struct Take<CSA_CACHE_E4M3> {
  static constexpr int kRows = 4, kRowStep = 32;
  static __device__ __forceinline__ int row_bytes(int d) { return d; }
  static __device__ __forceinline__ int first_row(int t) { return t >> 2; }
  static __device__ __forceinline__ int column(int t) { return (t & 3) * 32; }
  uint4 a, b;
  uint32_t k;
  __device__ __forceinline__ void load(const AttnParams& p, int64_t at, int col) {
    const bool some = at >= 0 && col < p.d;
    a = b = make_uint4(0, 0, 0, 0);
    k = some ? __ldg(p.scales + (at >> 5) + (col >> 5)) : kNoScale;
    if (some) {
      const uint4* w = reinterpret_cast<const uint4*>(p.data + at + col);
      a = __ldg(w);
      b = __ldg(w + 1);
    }
  }
  // 8 codes
  static __device__ __forceinline__ uint4 widen(uint32_t k, uint32_t x, uint32_t y) {
    return Widen<CSA_CACHE_E4M3>::plain(k) && (e4m3_nans(x) | e4m3_nans(y)) == 0
               ? Widen<CSA_CACHE_E4M3>(k).eight(x, y)
               : widen_any(x, y, scale_value(k));
  }
  __device__ __forceinline__ void store(uint32_t pair, int row, int t) const {
    const bool swap = (t & 2) != 0;
    const uint4 u = swap ? b : a, v = swap ? a : b;
    const uint32_t nans = e4m3_nans(a.x) | e4m3_nans(a.y) | e4m3_nans(a.z) | e4m3_nans(a.w) | e4m3_nans(b.x) |
                          e4m3_nans(b.y) | e4m3_nans(b.z) | e4m3_nans(b.w);
    auto pieces = [&](auto w) {
      store_pieces(pair, row, t, [&](int i) {
        return i == 0 ? w(u.x, u.y) : i == 1 ? w(u.z, u.w) : i == 2 ? w(v.x, v.y) : w(v.z, v.w);
      });
    };
    if (Widen<CSA_CACHE_E4M3>::plain(k) && nans == 0) {
      const Widen<CSA_CACHE_E4M3> s(k);
      pieces([&](uint32_t x, uint32_t y) { return s.eight(x, y); });
    } else {
      const float s = scale_value(k);
      pieces([&](uint32_t x, uint32_t y) { return widen_any(x, y, s); });
    }
  }
};
template <>
struct Take<CSA_CACHE_E2M1> {
  static constexpr int kRows = 4, kRowStep = 32;
  static __device__ __forceinline__ int row_bytes(int d) { return d / 2; }
  static __device__ __forceinline__ int first_row(int t) { return t >> 2; }
  static __device__ __forceinline__ int column(int t) { return (t & 3) * 32; }
  uint4 a;
  uint32_t k;
  __device__ __forceinline__ void load(const AttnParams& p, int64_t at, int col) {
    const bool some = at >= 0 && col < p.d;
    k = some ? __ldg(p.scales + (at >> 4) + (col >> 5)) : kNoScale;
    a = some ? __ldg(reinterpret_cast<const uint4*>(p.data + at + (col >> 1))) : make_uint4(0, 0, 0, 0);
  }
  static __device__ __forceinline__ uint4 widen(uint32_t k, uint32_t x) {
    return Widen<CSA_CACHE_E2M1>::plain(k) ? Widen<CSA_CACHE_E2M1>(k).eight(x) : widen_any(x, scale_value(k));
  }
  __device__ __forceinline__ void store(uint32_t pair, int row, int t) const {
    const bool swap = (t & 2) != 0;
    const uint4 u = swap ? make_uint4(a.z, a.w, a.x, a.y) : a;
    auto pieces = [&](auto w) {
      store_pieces(pair, row, t, [&](int i) { return w(i == 0 ? u.x : i == 1 ? u.y : i == 2 ? u.z : u.w); });
    };
    if (Widen<CSA_CACHE_E2M1>::plain(k)) {
      const Widen<CSA_CACHE_E2M1> s(k);
      pieces([&](uint32_t x) { return s.eight(x); });
    } else {
      const float s = scale_value(k);
      pieces([&](uint32_t x) { return widen_any(x, s); });
    }
  }
};

// Waits are bounded: one that runs out sets the CTA's stop word and reports, after which every
// wait returns at once and every role runs through the rest of its (finite) loops, so that
// the barriers among its warps stay matched; the products already issued are drained before
// the tensor memory is freed. The warp that issues tensor copies issues no more of them (it could
// not tell when a slot is free, nor count what is under way) and waits for those it has issued.
__device__ __forceinline__ void tile_wait(TileSmall& sm, const AttnParams& p, uint64_t* bar, uint32_t parity) {
  if (mbar_try_wait(bar, parity)) return;
  const long long t0 = clock64();
  while (!mbar_try_wait(bar, parity)) {
    if (*reinterpret_cast<volatile int*>(&sm.stop) != 0) return;
    if (clock64() - t0 > p.wait_cycles) {
      stop_pipeline(&sm.stop, p.dev_error);
      return;
    }
  }
}
__device__ __forceinline__ bool tile_stopped(const TileSmall& sm) {
  return *reinterpret_cast<const volatile int*>(&sm.stop) != 0;
}
// test hook: the first CTA never fills this tile's place in the ring
__device__ __forceinline__ bool tile_withheld(const AttnParams& p, int unit, int tile) {
  return tile == p.withhold_tile && unit == 0 && blockIdx.x == 0;
}

// Place in the ring of pairs: slot, and the parity of its current lap.
template <int RING>
struct RingAt {
  int slot = 0;
  uint32_t lap = 0;
  __device__ __forceinline__ void next() {
    if (++slot == RING) {
      slot = 0;
      lap ^= 1u;
    }
  }
};

// A unit from the work list; volatile, so that a later reading is a new one and its fields do not
// stay in registers over a loop that has no use for them.
__device__ __forceinline__ AttnUnit read_unit(const AttnUnit* at) {
  int4 v[3];
#pragma unroll
  for (int i = 0; i < 3; ++i)
    asm volatile("ld.global.nc.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v[i].x), "=r"(v[i].y), "=r"(v[i].z), "=r"(v[i].w)
                 : "l"(reinterpret_cast<const int4*>(at) + i));
  return {v[0].x, v[0].y, v[0].z, v[0].w, v[1].x, v[1].y, v[1].z, v[1].w, v[2].x, v[2].y, v[2].z, v[2].w};
}
__device__ __forceinline__ AttnSpan read_span(const AttnSpan* at) {
  union {
    int4 v[4];
    AttnSpan s;
  } r;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    asm volatile("ld.global.nc.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r.v[i].x), "=r"(r.v[i].y), "=r"(r.v[i].z), "=r"(r.v[i].w)
                 : "l"(reinterpret_cast<const int4*>(at) + i));
  return r.s;
}

// The runs of tiles of one unit in a worker's share.
struct SegmentWalk {
  const AttnParams& p;
  int unit, t0, t1;
  int64_t left;
  AttnUnit u;
  __device__ __forceinline__ SegmentWalk(const AttnParams& pp, int worker) : p(pp) {
    const AttnStart* at = p.starts + worker;
    u = read_unit(&at->u);
    const longlong2 v = __ldg(reinterpret_cast<const longlong2*>(at) + 3);
    unit = static_cast<int>(v.x);
    t0 = static_cast<int>(v.x >> 32);
    left = v.y;
    bound();
  }
  __device__ __forceinline__ void bound() { t1 = left < u.tiles - t0 ? t0 + static_cast<int>(left) : u.tiles; }
  __device__ __forceinline__ bool valid() const { return left > 0; }
  __device__ __forceinline__ void next() {
    left -= t1 - t0;
    ++unit;
    t0 = 0;
    if (left > 0) {
      u = read_unit(p.units + unit);
      bound();
    }
  }
  __device__ __forceinline__ bool last() const { return left == t1 - t0; }
};

// The walk with what a tile's entries are: the unit's sequence, or behind prefixes the span that the
// tile lies in, which enter() finds (tiles in order; some may be passed over). (Spans and pages looked up a
// span ahead took the same time.)
template <bool PREFIX>
struct TileWalk : SegmentWalk {
  __device__ __forceinline__ TileWalk(const AttnParams& pp, int worker) : SegmentWalk(pp, worker) {}
  __device__ __forceinline__ bool enter(int) { return false; }
  __device__ __forceinline__ int at(int tile) const { return tile; }  // among the list of entries that it belongs to
  __device__ __forceinline__ int run_end() const { return t1; }
  __device__ __forceinline__ int seen() const { return u.seen; }
  __device__ __forceinline__ int seen_all() const { return u.seen_all; }
  __device__ __forceinline__ const int32_t* table() const { return p.table + static_cast<int64_t>(u.s) * p.max_pages; }
  __device__ __forceinline__ int packed() const { return (u.s * p.kv_heads + u.kvh) * p.packed_rows; }
};
template <>
struct TileWalk<true> : SegmentWalk {
  const AttnSpan* next_span;
  const int32_t* span_table;
  int first, end, span_seen, span_all, span_packed;  // the span's tiles, and what is asked for at each of them
  __device__ __forceinline__ TileWalk(const AttnParams& pp, int worker) : SegmentWalk(pp, worker) { start(); }
  // before a unit's first tile
  __device__ __forceinline__ void start() {
    next_span = p.spans + u.span;
    end = 0;
  }
  __device__ __forceinline__ void next() {
    SegmentWalk::next();
    start();
  }
  __device__ __forceinline__ AttnSpan span() const { return read_span(next_span - 1); }
  // whether the tile lies in another span than the one before
  __device__ __forceinline__ bool enter(int tile) {
    bool moved = false;
    while (tile >= end) {
      const AttnSpan v = read_span(next_span++);
      first = v.tile;
      end = v.tile + v.tiles;
      span_seen = v.seen;
      span_all = v.seen_all;
      span_table = v.table;
      span_packed = v.packed;
      moved = true;
    }
    return moved;
  }
  __device__ __forceinline__ int at(int tile) const { return tile - first; }
  __device__ __forceinline__ int run_end() const { return min(t1, end); }
  __device__ __forceinline__ int seen() const { return span_seen; }
  __device__ __forceinline__ int seen_all() const { return span_all; }
  __device__ __forceinline__ const int32_t* table() const { return span_table; }
  __device__ __forceinline__ int packed() const { return span_packed; }
};
// What row `row` of a unit (`some`: it is one of the group's) sees of a span's entries.
__device__ __forceinline__ int span_limit(const AttnParams& p, const AttnUnit& u, const AttnSpan& v, int r) {
  const int row = u.block * kAttnRows + r;
  if (row >= u.rows) return v.seen;
  const int token = u.token + row / p.group;
  if (v.own != 0) {
    if (r < v.row0 || r >= v.row1) return 0;
    return max(0, visible(static_cast<int64_t>(v.first) + (token - v.token), p.ratio, v.n) - v.before);
  }
  if (v.seen_all >= v.seen) return v.seen;
  int lo = v.token, hi = v.first + 1;  // the token's sequence: cu[lo] <= token < cu[hi], the last such one
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (__ldg(p.cu + mid) <= token) lo = mid;
    else hi = mid;
  }
  const int64_t pos = static_cast<int64_t>(p.first != nullptr ? __ldg(p.first + lo) : 0) + (token - __ldg(p.cu + lo));
  return visible(pos, p.ratio, v.seen);
}

// ------------------------------------------------------------------------------ the fetchers
template <int NC, int SRC, bool PREFIX>
__device__ void tile_fetch(const AttnParams& p, TileSmall& sm, uint32_t base) {
  using SH = TileShape<NC>;
  using P = Take<SRC>;
  constexpr int kGroup = kTileLoaders / 2;
  constexpr int kStep = SH::kPairs == 1 ? 2 : 1;  // tiles from one of a group's to its next
  const int lt = threadIdx.x - kTileFirstLoader * 32;
  const int group = lt / kGroup, gt = lt % kGroup;
  const int row_bytes = P::row_bytes(p.d);

  TileWalk<PREFIX> w(p, blockIdx.x);
  int tile = w.t0, pair = 0, buf = 0;
  RingAt<SH::kRing> ring;
  bool fresh = true;  // the tile's rows are still to be looked up
  auto next_pair = [&]() {
    ring.next();
    if (++pair < SH::kPairs) return;
    pair = 0;
    fresh = true;
    if (++tile == w.t1) {
      w.next();
      tile = w.t0;
    }
  };
  // from one of the group's pairs to its next
  constexpr int kPairStep = SH::template kHelped<SRC> ? SH::kPairs : 2;
  // this thread's page of tile `ahead` of unit `unit`, read early
  int page = -1, ahead = -1, unit = -1;
  auto read_page = [&](int tl) {
    const int e = w.at(tl) * kAttnEntries + gt;
    ahead = tl;
    unit = w.unit;
    page = e < w.seen() ? __ldg(w.table() + e / p.page_size) : -1;
  };
  auto entry_at = [&](int e) {
    return ((static_cast<int64_t>(page) * p.page_size + e % p.page_size) * p.kv_heads + w.u.kvh) * row_bytes;
  };
  auto rows = [&]() {
    w.enter(tile);
    if (ahead != tile || unit != w.unit) read_page(tile);
    const int e = w.at(tile) * kAttnEntries + gt;
    int64_t at = -1;
    if (e < w.seen()) {
      if (page >= 0 && page < p.num_pages) at = entry_at(e);
      else if (p.dev_error != nullptr) *p.dev_error = CSA_DEVERR_PAGE;
    }
    buf ^= 1;
    sm.row[group][buf][gt] = at;
    named_barrier(6 + group, kGroup);
    fresh = false;
    if (tile + kStep < w.run_end()) read_page(tile + kStep);
  };

  if (group == 1 && w.valid()) next_pair();
  while (w.valid()) {
    if (fresh) rows();
    P v[P::kRows];
    const int64_t* at = &sm.row[group][buf][P::first_row(gt)];
    const int col = pair * 128 + P::column(gt);
    if constexpr (SH::template kHelped<SRC>) {
      // the softmax warps' half on its way into L2, a line by one lane
      const int far = (pair + SH::kPairs / 2) * 128;
      if ((gt & 3) == 0 && far < p.d)
#pragma unroll
        for (int i = 0; i < P::kRows; ++i)
          if (at[i * P::kRowStep] >= 0)
            asm volatile("prefetch.global.L2 [%0];" ::"l"(p.data + at[i * P::kRowStep] + P::row_bytes(far)));
    }
#pragma unroll
    for (int i = 0; i < P::kRows; ++i) v[i].load(p, at[i * P::kRowStep], col);
    tile_wait(sm, p, &sm.empty[ring.slot], ring.lap ^ 1u);
#pragma unroll
    for (int i = 0; i < P::kRows; ++i)
      v[i].store(base + ring.slot * kPairBytes, P::first_row(gt) + i * P::kRowStep, gt);
    fence_proxy_async_smem();
    __syncwarp();
    if ((threadIdx.x & 31) == 0 && !tile_withheld(p, w.unit, tile)) mbar_arrive(&sm.full[ring.slot]);
    next_pair();
#pragma unroll
    for (int i = 1; i < kPairStep; ++i)
      if (w.valid()) next_pair();
  }
}

// The softmax warps' part of fetching (kHelped): the second half of a tile's pairs, each by 256 of
// them.
template <int SRC, typename W>
__device__ __forceinline__ void help_places(const AttnParams& p, TileSmall& sm, const W& w, int tile, uint32_t t) {
  const int tid = threadIdx.x;
  if (tid >= kAttnEntries) return;
  const int e = w.at(tile) * kAttnEntries + tid;
  int64_t at = -1;
  if (e < w.seen()) {
    const int page = __ldg(w.table() + e / p.page_size);
    if (page >= 0 && page < p.num_pages)
      at = ((static_cast<int64_t>(page) * p.page_size + e % p.page_size) * p.kv_heads + w.u.kvh) *
           Take<SRC>::row_bytes(p.d);
  }
  sm.help_row[t & 1u][tid] = at;
}
template <int NC, int SRC, typename W>
__device__ __forceinline__ void tile_help(const AttnParams& p, TileSmall& sm, uint32_t base, const W& w, int tile,
                                          uint32_t t, bool moved) {
  using P = Take<SRC>;
  constexpr int kHalf = kSoftThreads / 2, kRows = 2, kRowStep = kAttnEntries / kRows;
  const int tid = threadIdx.x, half = tid / kHalf, ht = tid % kHalf;
  if (moved || tile == w.t0) help_places<SRC>(p, sm, w, tile, t);
  named_barrier(5, kSoftThreads);
  const int pair = TileShape<NC>::kPairs / 2 + half, row = P::first_row(ht), col = pair * 128 + P::column(ht);
  P v[kRows];
#pragma unroll
  for (int i = 0; i < kRows; ++i) v[i].load(p, sm.help_row[t & 1u][row + i * kRowStep], col);
  tile_wait(sm, p, &sm.empty[pair], (t & 1u) ^ 1u);
#pragma unroll
  for (int i = 0; i < kRows; ++i) v[i].store(base + pair * kPairBytes, row + i * kRowStep, ht);
  fence_proxy_async_smem();
  __syncwarp();
  if ((tid & 31) == 0) mbar_arrive(&sm.full[pair]);
  if (tile + 1 < w.run_end()) help_places<SRC>(p, sm, w, tile + 1, t + 1);
}

// ------------------------------------------------------------- the warp that issues tensor copies
// From the pages: lane i copies box i mod n of chunk i / n of each pair, n = 128 / box_rows of them.
// A box behind the last entry that the unit sees is not copied, and rows behind it in a copied
// box are whatever the pool holds there: masked in the scores, and made finite where they are
// not before the second product. From packed entries: a pair's two chunks by a lane each.
template <int NC, int SRC, bool PREFIX>
__device__ void tile_copy(const AttnParams& p, TileSmall& sm, uint32_t base, const CUtensorMap* map) {
  using SH = TileShape<NC>;
  const int lane = threadIdx.x & 31;
  RingAt<SH::kRing> ring;
  uint32_t places = 0;                     // of the ring, one after another, that this warp has filled
  uint32_t skipped_from = 0, skipped = 0;  // (test hook) those that it left empty: [skipped_from, skipped)
  // the next place is free, and the CTA has not stopped (one answer for the warp)
  auto room = [&]() {
    tile_wait(sm, p, &sm.empty[ring.slot], ring.lap ^ 1u);
    return !__any_sync(0xFFFFFFFFu, tile_stopped(sm));
  };
  bool go = true;
  if constexpr (SRC == kFromPacked) {
    for (TileWalk<PREFIX> w(p, blockIdx.x); go && w.valid(); w.next()) {
      for (int tile = w.t0; go && tile < w.t1; ++tile) {
        w.enter(tile);
        const int row = w.packed() + w.at(tile) * kAttnEntries;
        const bool withheld = tile_withheld(p, w.unit, tile);
        for (int c = 0; c < SH::kPairs && (go = room()); ++c, ring.next()) {
          ++places;
          if (withheld) {
            if (skipped == 0) skipped_from = places - 1;
            skipped = places;
            continue;
          }
          if (lane == 0) mbar_arrive_expect_tx(&sm.full[ring.slot], kPairBytes);
          __syncwarp();
          if (lane < 2)
            box_load2(base + ring.slot * kPairBytes + lane * kChunkBytes, map, c * 128 + lane * 64, row,
                      &sm.full[ring.slot]);
        }
      }
    }
  } else {
    const int n = kAttnEntries / p.box_rows, chunk = lane / n, box = lane % n;
    for (TileWalk<PREFIX> w(p, blockIdx.x); go && w.valid(); w.next()) {
      for (int tile = w.t0; go && tile < w.t1; ++tile) {
        w.enter(tile);
        const int e = w.at(tile) * kAttnEntries + box * p.box_rows;
        bool on = chunk < 2 && e < w.seen();
        int slot = 0;
        if (on) {
          const int page = __ldg(w.table() + e / p.page_size);
          on = page >= 0 && page < p.num_pages;
          if (on) slot = page * p.page_size + e % p.page_size;
          else if (p.dev_error != nullptr) *p.dev_error = CSA_DEVERR_PAGE;
        }
        const uint32_t bytes = __popc(__ballot_sync(0xFFFFFFFFu, on)) * p.box_rows * 128;
        const bool withheld = tile_withheld(p, w.unit, tile);
        for (int c = 0; c < SH::kPairs && (go = room()); ++c, ring.next()) {
          ++places;
          if (withheld) {
            if (skipped == 0) skipped_from = places - 1;
            skipped = places;
            continue;
          }
          if (lane == 0) mbar_arrive_expect_tx(&sm.full[ring.slot], bytes);
          __syncwarp();
          if (on)
            box_load3(base + ring.slot * kPairBytes + chunk * kChunkBytes + box * p.box_rows * 128, map,
                      c * 128 + chunk * 64, w.u.kvh, slot, &sm.full[ring.slot]);
        }
      }
    }
  }
  // A stop may come at any time from now on, after which nobody else waits for a copy: this warp stays
  // until those of the ring's last lap have landed. (Each earlier one was waited for before its place was
  // free again.)
  for (uint32_t k = places > SH::kRing ? places - SH::kRing : 0; k < places; ++k)
    if (k < skipped_from || k >= skipped)
      mbar_wait_bounded(&sm.full[k % SH::kRing], (k / SH::kRing) & 1u, kWaitCycles);
}

// ------------------------------------------------- the products' warp (all lanes take part)
template <int NC>
__device__ void tile_products(const AttnParams& p, TileSmall& sm, uint32_t base, uint32_t tmem) {
  using SH = TileShape<NC>;
  constexpr uint32_t kScoreDesc = mma_desc(128, kAttnRows, 0, 0);
  constexpr uint32_t kSumDesc = mma_desc(128, kAttnRows, 1, 1);
  // descriptors count in 16 bytes: a step adds to their address field
  const uint64_t by_row = smem_desc(base, 16, 1024), by_column = smem_desc(base, kChunkBytes, 1024);
  const uint64_t q = smem_desc(base + SH::kQOff, 16, 1024), probs = smem_desc(base + SH::kPOff, 16, 1024);
  RingAt<SH::kRing> rs, ro;  // next pair of the score products, and of the sums
  uint32_t t = 0;            // tiles whose scores have been issued
  auto scores = [&]() {
    const uint32_t d = tmem + SH::kTmemS + (t & 1) * kAttnRows;
#pragma unroll 1
    for (int c = 0; c < SH::kPairs; ++c, rs.next()) {
      tile_wait(sm, p, &sm.full[rs.slot], rs.lap);
      tc_fence_after();
      const uint64_t a = by_row + rs.slot * (kPairBytes >> 4), b = q + 2 * c * (kAttnRows * 128 >> 4);
#pragma unroll
      for (int k = 0; k < 8; ++k)  // 16 columns a step, 4 to a chunk
        tc_mma(d, a + (((k >> 2) * kChunkBytes + (k & 3) * 32) >> 4),
               b + (((k >> 2) * kAttnRows * 128 + (k & 3) * 32) >> 4), kScoreDesc, c > 0 || k > 0);
    }
    tc_commit(&sm.scores[t & 1]);
    ++t;
  };
  uint32_t done = 0, seg = 0;  // tiles summed, segments
  for (SegmentWalk w(p, blockIdx.x); w.valid(); w.next(), ++seg) {
    const int tiles = w.t1 - w.t0;
    tile_wait(sm, p, &sm.q_full, seg & 1u);
    tc_fence_after();
    scores();
    for (int j = 0; j < tiles; ++j) {
      if (SH::kAhead && j + 1 < tiles) scores();
      tile_wait(sm, p, &sm.probs, done & 1u);
      tc_fence_after();
#pragma unroll 1
      for (int c = 0; c < SH::kPairs; ++c, ro.next()) {
        const uint64_t a = by_column + ro.slot * (kPairBytes >> 4);
#pragma unroll
        for (int k = 0; k < 8; ++k)  // 16 entries a step
          tc_mma(tmem + SH::kTmemO + c * kAttnRows, a + k * (2048 >> 4), probs + k * (2048 >> 4), kSumDesc,
                 j > 0 || k > 0);
        tc_commit(&sm.empty[ro.slot]);
      }
      tc_commit(&sm.summed);
      ++done;
      if (!SH::kAhead && j + 1 < tiles) scores();
    }
  }
  // whatever was issued is over before the tensor memory goes
  tc_commit(&sm.drain);
  mbar_wait_bounded(&sm.drain, 0, kWaitCycles);
}

// Makes the infinities and NaN of entry e0 of tile t 0; whether it had any. Four threads do this for an
// entry, one a group: one that comes late finds the others' mark.
template <int NC>
__device__ __forceinline__ bool clear_odd(TileSmall& sm, unsigned char* smem, uint32_t t, int e0) {
  volatile uint32_t* const mark = &sm.odd[e0];
  bool found = false;
#pragma unroll 1
  for (int pass = 0; pass < 2; ++pass) {
#pragma unroll 1
    for (int i = 0; i < NC * 64; ++i) {
      const uint32_t pair = t * TileShape<NC>::kPairs + (i >> 7);
      unsigned char* at = smem + pair % TileShape<NC>::kRing * kPairBytes + (i >> 6 & 1) * kChunkBytes + e0 * 128;
      volatile uint16_t* v = reinterpret_cast<volatile uint16_t*>(at) + (i & 63);
      if ((*v & 0x7F80u) == 0x7F80u) {
        found = true;
        if (pass == 1) *v = 0;
      }
    }
    __threadfence_block();
    if (!found) found = *mark == t + 1u;
    if (!found) break;
    *mark = t + 1u;
    __threadfence_block();
  }
  return found;
}

// A row that has seen an infinity or NaN has one in its sums (0 * inf where its weight was 0): out and lse,
// or its piece's weight sum, become NaN throughout. (All softmax warps, rarely.)
template <int NC>
__device__ __forceinline__ void spread_nans(const AttnParams& p, TileSmall& sm, uint32_t sums, int par, bool whole,
                                            int64_t piece) {
  const int tid = threadIdx.x, lane = tid & 31, quad = (tid >> 5) & 3, c0 = (tid >> 7) * kSoftCols;
  tc_fence_after();
  uint32_t odd = 0;  // rows of the group
#pragma unroll 1
  for (int b = 0; b < TileShape<NC>::kPairs; ++b) {
    float v[kSoftCols];
    tmem_load16(sums + b * kAttnRows, v);
#pragma unroll
    for (int c = 0; c < kSoftCols; ++c) odd |= (fabsf(v[c]) <= 3.4028234e38f ? 0u : 1u) << c;
  }
  tc_fence_before();
  odd = __reduce_or_sync(0xFFFFFFFFu, odd);
  if (lane == 0) sm.red[quad][c0] = __uint_as_float(odd);
  named_barrier(1 + (tid >> 7), 128);
#pragma unroll
  for (int q = 0; q < 4; ++q) odd |= __float_as_uint(sm.red[q][c0]);
  const float nan = __uint_as_float(0x7FFFFFFFu);
#pragma unroll 1
  for (int c = 0; c < kSoftCols; ++c) {
    const int row = c0 + c;
    if ((odd >> c & 1u) == 0 || sm.out_at[par][row] < 0) continue;
    if (whole) {
      for (int col = quad * 32 + lane; col < p.d; col += 128) p.out[sm.out_at[par][row] + col] = 0x7FFF;
      if (p.lse != nullptr && quad == 0 && lane == 0) p.lse[sm.lse_at[par][row]] = nan;
    } else if (quad == 0 && lane == 0) {
      p.part_ml[piece * 2 * kAttnRows + kAttnRows + row] = nan;
    }
  }
}

// ------------------------------------------------------------------------- the softmax warps
template <int NC, int SRC, bool PREFIX>
__device__ void tile_softmax(const AttnParams& p, TileSmall& sm, unsigned char* smem, uint32_t base, uint32_t tmem) {
  using SH = TileShape<NC>;
  // Scores and sums two at a time where registers do for it (the same bits; 64 tokens behind 16384 packed entries of
  // 512 176.3 -> 173.5 us; by threads, in 72 registers, 48 tokens 68.9 -> 70.0).
  constexpr bool kTwos = !TileCta<SRC>::kByThreads;
  const int tid = threadIdx.x, lane = tid & 31, quad = (tid >> 5) & 3, group = tid >> 7;
  const int c0 = group * kSoftCols;     // the rows (columns of S^T) of this group of four warps
  const int e0 = quad * 32 + lane;      // the entry (row of S^T) of this thread
  const uint32_t lanes = tmem + (static_cast<uint32_t>(quad * 32) << 16);
  // (a scale of 0, under which every score is equal, becomes the least one: no finite score exceeds 2^-20
  // under it, and masked ones stay infinite)
  const float sl2 = p.scale == 0.f ? 1.4e-45f : p.scale * kLog2e;
  uint32_t t = 0;  // tiles so far
  auto barrier_group = [&]() { named_barrier(1 + group, 128); };

  // where each row of a unit's q, out and lse lies, what it sees, its sink (rows behind the last one
  // are zeros, see what the last one sees, and are never stored)
  auto set_up = [&](const AttnUnit& u, int par) {
    const int row = u.block * kAttnRows + tid, token = row / p.group;
    const bool some = row < u.rows;
    const int head = u.kvh * p.group + (row - token * p.group);
    const int64_t at = static_cast<int64_t>(u.token) + token;
    if constexpr (!PREFIX) sm.lim[par][tid] = some ? visible(static_cast<int64_t>(u.first) + token, p.ratio, u.n) : u.seen;
    sm.q_at[tid] = some ? at * p.q_row + head * p.q_head : -1;
    sm.out_at[par][tid] = some ? at * p.out_row + head * p.out_head : -1;
    sm.lse_at[par][tid] = some ? static_cast<int32_t>(at * p.q_heads + head) : -1;
    sm.sink[par][tid] = some && p.sink != nullptr ? __ldg(p.sink + head) : -INFINITY;
  };
  auto copy_q = [&]() {
    constexpr int kPer = NC * 8;  // 16-byte pieces of a row; NC pieces a thread
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int at = tid + i * kSoftThreads, r = at / kPer, c = at % kPer;
      const int64_t q_at = sm.q_at[r];
      const bool some = q_at >= 0 && c * 8 < p.d;
      copy16(base + SH::kQOff + (c >> 3) * (kAttnRows * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4),
             p.q + (some ? q_at + c * 8 : 0), some);
    }
  };
  auto q_copied = [&]() {
    asm volatile("cp.async.wait_all;" ::: "memory");
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.q_full);
  };
  int par = 0;
  if (tid < kAttnEntries) sm.odd[tid] = 0;
  TileWalk<PREFIX> w(p, blockIdx.x);
  bool idle = false;  // behind prefixes: the group's rows see nothing of the span
  int lim_at = 0;  // which of the two lists of limits holds: the unit's, or behind prefixes the span's
  if (w.valid()) {
    if (tid < kAttnRows) {
      set_up(w.u, 0);
      sm.m[tid] = kTwos ? -kNoMax : kNoMax;
    }
    named_barrier(5, kSoftThreads);
    copy_q();
    q_copied();
  }
  for (; w.valid(); par ^= 1) {
    if constexpr (!PREFIX) lim_at = par;
    const bool whole = w.t0 == 0 && w.t1 == w.u.tiles, more = !w.last();
    if (more && tid >= kSoftThreads - 3) {  // the next unit on its way
      const int i = tid - (kSoftThreads - 3);
      reinterpret_cast<int4*>(&sm.next)[i] = __ldg(reinterpret_cast<const int4*>(p.units + w.unit + 1) + i);
    }
    float l[kSoftCols];
#pragma unroll
    for (int c = 0; c < kSoftCols; ++c) l[c] = 0.f;

    for (int j = w.t0; j < w.t1; ++j, ++t) {
      const bool moved = w.enter(j);
      if constexpr (SH::template kHelped<SRC>) tile_help<NC, SRC>(p, sm, base, w, j, t, moved);
      if constexpr (PREFIX) {
        // the span's limits for the group's rows, in the list that no warp of the group reads any more (all
        // have passed a barrier since the span before the last one)
        if (moved) {
          lim_at ^= 1;
          // an own entry's sequence may have no row in this group: no weight then (some group has rows, and
          // clears what is not finite)
          const AttnSpan v = w.span();
          idle = v.own != 0 && (c0 + kSoftCols <= v.row0 || c0 >= v.row1);
          if (!idle) {
            if (quad == 0 && lane < kSoftCols) sm.lim[lim_at][c0 + lane] = span_limit(p, w.u, v, c0 + lane);
            barrier_group();
          }
        }
      }
      const uint32_t row = base + SH::kPOff + e0 * 128;
      if (PREFIX && idle) {
        if (j > w.t0) tile_wait(sm, p, &sm.summed, (t - 1u) & 1u);  // (so the scores' barrier is not passed a lap ahead either)
#pragma unroll
        for (int c = 0; c < 2; ++c) sts128(row + (((group * 2 + c) ^ (e0 & 7)) << 4), make_uint4(0, 0, 0, 0));
      } else {
        const int e = w.at(j) * kAttnEntries + e0;
        const bool masked = (w.at(j) + 1) * static_cast<int64_t>(kAttnEntries) > w.seen_all();
        const uint32_t s_at = lanes + SH::kTmemS + (t & 1u) * kAttnRows + c0;
        tile_wait(sm, p, &sm.scores[t & 1u], (t >> 1) & 1u);
        tc_fence_after();
        float s[kSoftCols];
        bool odd = false;  // some row of the tile does not see all of it, and a score of this entry is not finite
        auto take = [&]() {
          tmem_load16(s_at, s);
          if (masked) {
#pragma unroll
            for (int c = 0; c < kSoftCols; ++c) {
              odd = odd || !(fabsf(s[c]) <= 3.4028234e38f);
              if (e >= sm.lim[lim_at][c0 + c]) s[c] = sl2 < 0.f ? INFINITY : -INFINITY;  // -inf once scaled
            }
          }
        };
        auto scale = [&]() {
#pragma unroll
          for (int c = 0; c < kSoftCols; c += 4) {
            if constexpr (kTwos) {
              const ulonglong2 m = *reinterpret_cast<const ulonglong2*>(&sm.m[c0 + c]);
              const uint64_t a = f2_fma(f2_pack(s[c], s[c + 1]), f2_pack(sl2, sl2), m.x);
              const uint64_t b = f2_fma(f2_pack(s[c + 2], s[c + 3]), f2_pack(sl2, sl2), m.y);
              s[c] = f2_lo(a);
              s[c + 1] = f2_hi(a);
              s[c + 2] = f2_lo(b);
              s[c + 3] = f2_hi(b);
            } else {
              const float4 m = *reinterpret_cast<const float4*>(&sm.m[c0 + c]);
              s[c] = fmaf(s[c], sl2, -m.x);
              s[c + 1] = fmaf(s[c + 1], sl2, -m.y);
              s[c + 2] = fmaf(s[c + 2], sl2, -m.z);
              s[c + 3] = fmaf(s[c + 3], sl2, -m.w);
            }
          }
        };
        take();
        scale();
        float top = fmaxf(s[0], s[1]);
#pragma unroll
        for (int c = 2; c < kSoftCols; c += 2) top = fmax3(top, s[c], s[c + 1]);
        if (named_barrier_or(1 + group, 128, top > kRescaleAt)) {
          // new bounds: the true maxima so far, rounded down. A score less its row's maximum is then what the
          // rounding left, never below 0; far from zero (2^27 and more) that may pass any weight, and is
          // cut off (a difference of one step of the fp32 score that it stands for).
          take();
          float mine = kNoMax;
#pragma unroll
          for (int c = 0; c < kSoftCols; ++c) {
            const float v = warp_max_f32(__fmul_rd(s[c], sl2));
            if (lane == c) mine = v;
          }
          if (lane < kSoftCols) sm.red[quad][c0 + lane] = mine;
          barrier_group();
          if (quad == 0 && lane < kSoftCols) {
            const int c = c0 + lane;
            const float old = kTwos ? -sm.m[c] : sm.m[c];
            float m = fmaxf(fmaxf(sm.red[0][c], sm.red[1][c]), fmaxf(sm.red[2][c], sm.red[3][c]));
            m = fmaxf(old, m);
            sm.fac[c] = fast_exp2(old - m);
            sm.m[c] = kTwos ? -m : m;
          }
          barrier_group();
#pragma unroll
          for (int c = 0; c < kSoftCols; ++c) l[c] *= sm.fac[c0 + c];
          if (j > w.t0) {
            tile_wait(sm, p, &sm.summed, (t - 1u) & 1u);
            tc_fence_after();
#pragma unroll 1
            for (int b = 0; b < SH::kPairs; ++b) {
              const uint32_t at = lanes + SH::kTmemO + b * kAttnRows + c0;
              tmem_load16(at, s);
#pragma unroll
              for (int c = 0; c < kSoftCols; ++c) s[c] *= sm.fac[c0 + c];
              tmem_store16(at, s);
            }
          }
          take();
          scale();
#pragma unroll
          for (int c = 0; c < kSoftCols; ++c) s[c] = min_nan(s[c], kRescaleAt);
        }
        // weights; their sums before rounding
        uint32_t w2[kSoftCols / 2];
#pragma unroll
        for (int c = 0; c < kSoftCols; c += 2) {
          const float a = fast_exp2(s[c]), b = fast_exp2(s[c + 1]);
          if constexpr (kTwos) {
            const uint64_t sum = f2_add(f2_pack(l[c], l[c + 1]), f2_pack(a, b));
            l[c] = f2_lo(sum);
            l[c + 1] = f2_hi(sum);
          } else {
            l[c] += a;
            l[c + 1] += b;
          }
          w2[c / 2] = pack_bf16x2(a, b);
        }
        if (j > w.t0) tile_wait(sm, p, &sm.summed, (t - 1u) & 1u);  // P is free
#pragma unroll
        for (int c = 0; c < 2; ++c)
          sts128(row + (((group * 2 + c) ^ (e0 & 7)) << 4), make_uint4(w2[4 * c], w2[4 * c + 1], w2[4 * c + 2], w2[4 * c + 3]));
        if (masked && __any_sync(0xFFFFFFFFu, odd)) {
          // 0 * NaN would reach the rows that do not see this entry: its non-finite values become 0, and the
          // weights of the rows that see it (whose scores are not finite either) NaN
          tmem_load16(s_at, s);
          if (odd && clear_odd<NC>(sm, smem, t, e0))
#pragma unroll
            for (int c = 0; c < kSoftCols; ++c)
              if (e < sm.lim[lim_at][c0 + c] && !(fabsf(s[c]) <= 3.4028234e38f)) {
                l[c] = __uint_as_float(0x7FFFFFFFu);
                asm volatile("st.shared.b16 [%0], %1;" ::"r"(row + (((group * 2 + (c >> 3)) ^ (e0 & 7)) << 4) + 2 * (c & 7)),
                             "h"(static_cast<uint16_t>(0x7FFF))
                             : "memory");
              }
        }
      }
      fence_proxy_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.probs);
      if (j == w.t0 && more) {
        // the next unit's places, and its rows of q on their way into L2
        named_barrier(5, kSoftThreads);
        if (tid < kAttnRows) set_up(sm.next, par ^ 1);
        const int r = tid / NC, row = sm.next.block * kAttnRows + r;
        const int col = (tid % NC) * 64;
        if (r < kAttnRows && row < sm.next.rows && col < p.d) {
          const int token = row / p.group;
          const uint16_t* at = p.q + (static_cast<int64_t>(sm.next.token) + token) * p.q_row +
                               (sm.next.kvh * p.group + (row - token * p.group)) * p.q_head + col;
          asm volatile("prefetch.global.L2 [%0];" ::"l"(at));
        }
      }
    }

    if (more) {
      // q's place is free, the last scores being there: the next unit's rows come, and its first
      // scores follow, while this one's sums go out
      named_barrier(5, kSoftThreads);
      copy_q();
    }
    // the unit's (or its piece's) sums are complete
    tile_wait(sm, p, &sm.summed, (t - 1u) & 1u);
    tc_fence_after();
    // the lanes' sums of each column: halves change hands until a lane has one column
#pragma unroll
    for (int k = 8; k > 0; k >>= 1) {
      const bool upper = (lane & (2 * k)) != 0;
#pragma unroll
      for (int c = 0; c < k; ++c) {
        const float give = upper ? l[c] : l[c + k], keep = upper ? l[c + k] : l[c];
        l[c] = keep + __shfl_xor_sync(0xFFFFFFFFu, give, 2 * k);
      }
    }
    l[0] += __shfl_xor_sync(0xFFFFFFFFu, l[0], 1);
    if ((lane & 1) == 0) sm.red[quad][c0 + (lane >> 1)] = l[0];
    barrier_group();
    const int64_t piece = 2 * static_cast<int64_t>(blockIdx.x) + (w.t0 == 0 ? 1 : 0);
    if (quad == 0 && lane < kSoftCols) {
      const int c = c0 + lane;
      const float z = (sm.red[0][c] + sm.red[1][c]) + (sm.red[2][c] + sm.red[3][c]), m = kTwos ? -sm.m[c] : sm.m[c];
      if (!whole) {
        float* ml = p.part_ml + piece * 2 * kAttnRows;
        ml[c] = m;
        ml[kAttnRows + c] = z;
      } else {
        const float sink_e = sm.sink[par][c], sink = sink_e * kLog2e;
        const float mx = fmaxf(z > 0.f || z != z ? m : -INFINITY, sink);
        const float old = mx == -INFINITY ? 0.f : fast_exp2(m - mx);
        const float den = mx == -INFINITY ? 0.f : z * old + sink_weight(sink, mx);
        sm.fac[c] = mx == -INFINITY ? 0.f : old / den;
        if (p.lse != nullptr && sm.lse_at[par][c] >= 0) p.lse[sm.lse_at[par][c]] = z == 0.f ? sink_e : (mx + log2f(den)) * kLn2;
      }
      sm.m[c] = kTwos ? -kNoMax : kNoMax;  // for the next unit
    }
    if (more) q_copied();
    barrier_group();
    uint32_t probe = 0;  // two bf16, one NaN once one of this thread's sums is (or, harmlessly, at huge ones)
    if (whole) {
      // O^T times the rows' factors, as bf16 rows: a warp's 32 columns of its 16 rows at a time are
      // transposed by 8 x 8 matrices through its 1 KB of P's place (two rows to 128 bytes, their 16-byte
      // pieces at other places from pair to pair), and go out in 16-byte pieces
      const int c = c0 + 2 * (lane & 3);
      const float f0 = sm.fac[c], f1 = sm.fac[c + 1], f2 = sm.fac[c + 8], f3 = sm.fac[c + 9];
      const uint32_t stage = base + SH::kPOff + (tid >> 5) * 1024;
      auto place = [&](int r, int piece) {
        return stage + (r >> 1) * 128 + (((r & 1) * 4 + (piece ^ ((r >> 1) & 3))) << 4);
      };
      const int to_row = ((lane >> 4) << 3) + (lane & 7), to_piece = (lane >> 3) & 1;
#pragma unroll 1
      for (int b = 0; b < SH::kPairs; ++b) {
        float v[2][8];
        tmem_load_fragments(lanes + SH::kTmemO + b * kAttnRows + c0, v);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t a = pack_bf16x2(v[h][0] * f0, v[h][1] * f1), b2 = pack_bf16x2(v[h][2] * f0, v[h][3] * f1);
          const uint32_t c2 = pack_bf16x2(v[h][4] * f2, v[h][5] * f3), d = pack_bf16x2(v[h][6] * f2, v[h][7] * f3);
          store_transposed(place(to_row, to_piece + h * 2), a, b2, c2, d);
          probe = fma_bf16x2(c2, d, fma_bf16x2(a, b2, probe));
        }
        __syncwarp();
        const int col = b * 128 + quad * 32 + (lane & 3) * 8;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int r = h * 8 + (lane >> 2);
          const int64_t at = sm.out_at[par][c0 + r];
          if (at >= 0 && col < p.d) *reinterpret_cast<uint4*>(p.out + at + col) = lds128(place(r, lane & 3));
        }
        __syncwarp();
      }
      tc_fence_before();
    } else {
      // four rows of a column in 16 bytes, a warp's 32 columns side by side
      float4* o = reinterpret_cast<float4*>(p.part_o + piece * kAttnRows * SH::kDpad);
#pragma unroll 1
      for (int b = 0; b < SH::kPairs; ++b) {
        float v[kSoftCols];
        tmem_load16(lanes + SH::kTmemO + b * kAttnRows + c0, v);
        float product = 0.f;
#pragma unroll
        for (int c = 0; c < kSoftCols; c += 2) product = fmaf(v[c], v[c + 1], product);
        probe |= product != product ? 0x7FFFu : 0u;
#pragma unroll
        for (int c = 0; c < kSoftCols; c += 4)
          if (sm.out_at[par][c0 + c] >= 0)
            o[((b * 4 + quad) * (kAttnRows / 4) + (c0 + c) / 4) * 32 + lane] =
                make_float4(v[c], v[c + 1], v[c + 2], v[c + 3]);
      }
      tc_fence_before();
    }
    w.left -= w.t1 - w.t0;
    ++w.unit;
    w.t0 = 0;
    if (more) {
      w.u = sm.next;
      w.bound();
      if constexpr (PREFIX) w.start();
    }
    // (sm.next and P's place are free again)
    if (named_barrier_or(5, kSoftThreads, (probe & 0x7FFFu) > 0x7F80u || (probe >> 16 & 0x7FFFu) > 0x7F80u))
      spread_nans<NC>(p, sm, lanes + SH::kTmemO + c0, par, whole, piece);
  }
}

// Chunks: the entries that a sequence's last token sees, as bf16 rows in order, zeros up to the next
// multiple of 128 rows and of 64 NC columns, so that the tile kernel's copies are whole boxes
// whatever the format, the page size and the heads. Every unit of the sequence (one per 64
// rows) reads them again; packing reads and writes them once. Block (x, s, cache head): 32
// entries at a time, a thread 8 columns at a time. Behind prefixes a row of blocks: prefix_blocks for all
// prefixes, then the same number for each sequence and cache head.
constexpr int kPackThreads = 256;
// Entries at a time: 32, behind prefixes 32 to 128 of 64 KB in all, so that a thread has eight pieces under way
// (32 of 128 columns each, two pieces a thread, took 21.5 us for 31 thousand entries of 4 heads).
__host__ __device__ constexpr int pack_rows(int nc, bool prefix) { return prefix ? 256 / nc : 32; }
template <int NC, int FORMAT, bool PREFIX>
__global__ void __launch_bounds__(kPackThreads) attn_pack_kernel(const __grid_constant__ AttnParams p, int prefix_blocks) {
  constexpr int kPer = NC * 8;  // pieces of 8 columns
  pdl_wait();
  if (p.head->status != 0) return;
  // kRows entries from e0 on of a run of n, whose first lies in row row0 of the packed ones: each row's place in the
  // pool once, by a thread each, then the pieces
  constexpr int kRows = pack_rows(NC, PREFIX), kPieces = kRows * kPer / kPackThreads;  // a thread's
  constexpr int kAtOnce = kPieces < (PREFIX ? 8 : 4) ? kPieces : PREFIX ? 8 : 4;
  static_assert(kPieces % kAtOnce == 0 && kPieces * kPackThreads == kRows * kPer && kAttnEntries % kRows == 0 &&
                kRows <= kPackThreads);
  __shared__ int64_t s_entry[kRows];
  auto pack = [&](const int32_t* table, int64_t row0, int kvh, int n, int e0) {
    uint16_t* to = p.packed + (row0 + e0) * (NC * 64);
    __syncthreads();
    if (threadIdx.x < kRows) {
      const int e = e0 + threadIdx.x;
      int64_t entry = -1;
      if (e < n) {
        const int page = __ldg(table + e / p.page_size);
        if (page >= 0 && page < p.num_pages) entry = (static_cast<int64_t>(page) * p.page_size + e % p.page_size) * p.kv_heads + kvh;
        else if (p.dev_error != nullptr) *p.dev_error = CSA_DEVERR_PAGE;
      }
      s_entry[threadIdx.x] = entry;
    }
    __syncthreads();
#pragma unroll 1
    for (int i0 = threadIdx.x; i0 < kRows * kPer; i0 += kAtOnce * kPackThreads) {
      // codes, then rows: each step's loads side by side
      uint4 v[kAtOnce];
      uint32_t scale[kAtOnce];
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k) {
        const int i = i0 + k * kPackThreads, col = (i % kPer) * 8;
        const int64_t entry = s_entry[i / kPer];
        v[k] = make_uint4(0, 0, 0, 0);
        scale[k] = kNoScale;
        if (entry >= 0 && col < p.d) {
          if constexpr (FORMAT == CSA_CACHE_BF16) {
            v[k] = __ldg(reinterpret_cast<const uint4*>(p.data + (entry * p.d + col) * 2));
          } else {
            scale[k] = __ldg(p.scales + entry * (p.d / CSA_CACHE_GROUP) + col / CSA_CACHE_GROUP);
            if constexpr (FORMAT == CSA_CACHE_E4M3) {
              const uint2 w = __ldg(reinterpret_cast<const uint2*>(p.data + entry * p.d + col));
              v[k].x = w.x;
              v[k].y = w.y;
            } else {
              v[k].x = __ldg(reinterpret_cast<const uint32_t*>(p.data + entry * (p.d / 2) + col / 2));
            }
          }
        }
      }
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k) {
        const int i = i0 + k * kPackThreads;
        if constexpr (FORMAT == CSA_CACHE_E4M3) v[k] = Take<FORMAT>::widen(scale[k], v[k].x, v[k].y);
        if constexpr (FORMAT == CSA_CACHE_E2M1) v[k] = Take<FORMAT>::widen(scale[k], v[k].x);
        *reinterpret_cast<uint4*>(to + (i / kPer) * (NC * 64) + (i % kPer) * 8) = v[k];
      }
    }
  };
  auto rows_of = [](int n) { return max(kAttnEntries, (n + kAttnEntries - 1) / kAttnEntries * kAttnEntries); };
  int seq = blockIdx.y, kvh = blockIdx.z, x = blockIdx.x, wide = gridDim.x;
  if (PREFIX && x < prefix_blocks) {
    // all prefixes and cache heads, in steps of the table's capacity, over the first blocks
    const int steps = p.prefix_rows / kRows;
    for (int64_t i = x; i < static_cast<int64_t>(p.groups) * p.kv_heads * steps; i += prefix_blocks) {
      const int part = static_cast<int>(i / steps), e0 = static_cast<int>(i - static_cast<int64_t>(part) * steps) * kRows;
      const int g = part / p.kv_heads, n = __ldg(p.prefix_entries + g);
      if (e0 >= rows_of(n) || __ldg(p.cu + __ldg(p.prefix_seqs + g + 1)) == __ldg(p.cu + __ldg(p.prefix_seqs + g))) continue;
      pack(p.prefix_table + static_cast<int64_t>(g) * p.max_prefix_pages, static_cast<int64_t>(part) * p.prefix_rows,
           part - g * p.kv_heads, n, e0);
    }
    return;
  }
  if constexpr (PREFIX) {  // a sequence's cache heads: as many blocks each as there are room for
    wide = (gridDim.x - prefix_blocks) / (p.S * p.kv_heads);
    const int part = (x - prefix_blocks) / wide;
    x = (x - prefix_blocks) - part * wide;
    seq = part / p.kv_heads;
    kvh = part - seq * p.kv_heads;
  }
  const int rows = sequence_rows(p, seq);
  if (rows == 0) return;
  int before = 0;
  if constexpr (PREFIX) {
    int lo = 0, hi = p.groups;  // the sequence's group
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (__ldg(p.prefix_seqs + mid) <= seq) lo = mid;
      else hi = mid;
    }
    before = __ldg(p.prefix_entries + lo);
  }
  const int64_t first = p.first != nullptr ? __ldg(p.first + seq) : 0;
  const int n = max(0, visible(first + rows / p.group - 1, p.ratio, before + __ldg(p.entries + seq)) - before);
  if (PREFIX && n == 0) return;
  const int64_t row0 = (static_cast<int64_t>(seq) * p.kv_heads + kvh) * p.packed_rows +
                       (PREFIX ? static_cast<int64_t>(p.groups) * p.kv_heads * p.prefix_rows : 0);
  const int end = rows_of(n);
  for (int e0 = x * kRows; e0 < end; e0 += wide * kRows)
    pack(p.table + static_cast<int64_t>(seq) * p.max_pages, row0, kvh, n, e0);
}

template <int NC, int SRC, bool PREFIX>
__global__ void __launch_bounds__(TileCta<SRC>::kThreads, 1)
    attn_tile_kernel(const __grid_constant__ AttnParams p, const __grid_constant__ CUtensorMap map) {
  using SH = TileShape<NC>;
  using CTA = TileCta<SRC>;
  extern __shared__ unsigned char raw[];
  unsigned char* smem = raw + ((1024u - (smem_addr(raw) & 1023u)) & 1023u);
  TileSmall& sm = *reinterpret_cast<TileSmall*>(smem + SH::kSmallOff);
  const uint32_t base = smem_addr(smem);
  const int warp = threadIdx.x >> 5;
  if (warp == 0) tmem_alloc(&sm.tmem, SH::kTmemColumns);
  if (threadIdx.x == 32) {
    for (int i = 0; i < SH::kRing; ++i) {
      const bool helped = SH::template kHelped<SRC> && i >= SH::kPairs / 2;
      mbar_init(&sm.full[i], helped ? kTileSoftWarps / 2 : CTA::kByThreads ? kTileLoadWarps / 2 : 1);
      mbar_init(&sm.empty[i], 1);
    }
    mbar_init(&sm.scores[0], 1);
    mbar_init(&sm.scores[1], 1);
    mbar_init(&sm.probs, kTileSoftWarps);
    mbar_init(&sm.summed, 1);
    mbar_init(&sm.q_full, kTileSoftWarps);
    mbar_init(&sm.drain, 1);
    sm.stop = 0;
    fence_mbar_init();
  }
  if constexpr (PREFIX && SRC == kFromBoxes) {
    // rows that no box covers count as seen by nobody, but what shared memory holds of other kernels may look
    // like infinities and NaN, which the softmax warps would have to clear one by one (7 us a tile)
    for (uint32_t at = threadIdx.x * 16; at < SH::kRing * kPairBytes; at += CTA::kThreads * 16) sts128(base + at, make_uint4(0, 0, 0, 0));
    fence_proxy_async_smem();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem;
  pdl_wait();
  const bool run = p.head->status == 0;
  if constexpr (CTA::kByThreads) {
    if (warp >= kTileFirstLoader) {
      regs_up<kLoadRegs>();
      if (run) tile_fetch<NC, SRC, PREFIX>(p, sm, base);
    } else if (warp >= kTileSoftWarps) {
      regs_down<kIssueRegs>();
      if (run && warp == kTileSoftWarps) tile_products<NC>(p, sm, base, tmem);
    } else {
      regs_down<kSoftRegs>();
      if (run) tile_softmax<NC, SRC, PREFIX>(p, sm, smem, base, tmem);
    }
  } else if (run) {
    if (warp == kTileSoftWarps) tile_products<NC>(p, sm, base, tmem);
    else if (warp == kTileSoftWarps + 1) tile_copy<NC, SRC, PREFIX>(p, sm, base, &map);
    else if (warp < kTileSoftWarps) tile_softmax<NC, SRC, PREFIX>(p, sm, smem, base, tmem);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 0) tmem_free(tmem, SH::kTmemColumns);
}

// Joins the pieces of the units that workers share. What it costs is a chain of loads (the list,
// the pieces' maxima and weight sums, their sums) and instructions: a warp takes four rows and 64
// columns, four pieces' loads under way at once and the first four's before their weights are
// known; lane 8 r + k works out row r's weight of piece k. A unit of many pieces (a long sequence
// by itself) is split over a block's warps, which take four pieces each in turn and meet in shared
// memory. The order of the sums is fixed. (Redundant work in the warps took 33 of 720 us for 150 units of
// 64 rows x 512 in two pieces each, 12 of 701 so.)
constexpr int kJoinThreads = 256, kJoinWarps = kJoinThreads / 32, kJoinBlocks = 3;  // blocks an SM
constexpr int kFewPieces = 8;
template <int NC>
__global__ void __launch_bounds__(kJoinThreads, kJoinBlocks) attn_join_kernel(const __grid_constant__ AttnParams p) {
  constexpr int kQuads = kAttnRows / 4;           // fours of rows
  constexpr int kTasks = kQuads * NC;             // of a unit: four rows, 64 columns
  constexpr int kFewItems = kTasks / kJoinWarps;  // blocks of a unit of few pieces; kTasks of one of many
  constexpr int kPiece = kAttnRows * NC * 64 / 4, kFlight = 4;
  __shared__ float4 s_sum[kJoinWarps][2][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane >> 3, kk = lane & 7;
  pdl_wait();
  const int4 head = *reinterpret_cast<const int4*>(p.head);
  if (head.x != 0) return;
  const int few_items = head.y * kFewItems, items = few_items + head.z * kTasks;  // (of at most one unit a worker)
  for (int item = blockIdx.x; item < items; item += gridDim.x) {
    const bool few = item < few_items;
    const int rest = few ? item : item - few_items;
    const int task = few ? rest % kFewItems * kJoinWarps + warp : rest % kTasks;
    const AttnJoin& J = p.joins[few ? rest / kFewItems : p.workers - 1 - rest / kTasks];
    const int quad = task % kQuads, chunk = task / kQuads;
    const AttnUnit u = J.u;
    const int first = J.worker, n = J.pieces;
    const int row0 = u.block * kAttnRows + quad * 4, row = row0 + r;
    if (row0 >= u.rows) continue;  // (all of a block's warps, where they share a task)
    auto slot = [&](int k) { return 2 * static_cast<int64_t>(first + k) + (k == 0 ? 1 : 0); };
    const float4* o = reinterpret_cast<const float4*>(p.part_o) + (chunk * 2 * kQuads + quad) * 32 + lane;
    const float* ml = p.part_ml + quad * 4 + r;
    const int step = few ? kFlight : kFlight * kJoinWarps;
    int k0 = few ? 0 : warp * kFlight;
    float4 v[kFlight][2];
    float m0;  // piece k0 + kk's bound
    auto fetch = [&]() {
#pragma unroll
      for (int k = 0; k < kFlight; ++k)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          v[k][h] = k0 + k < n ? o[slot(k0 + k) * kPiece + h * (kQuads * 32)] : make_float4(0.f, 0.f, 0.f, 0.f);
      m0 = k0 + kk < n ? ml[slot(k0 + kk) * 2 * kAttnRows] : kNoMax;
    };
    fetch();
    const int token = row / p.group, head_of = u.kvh * p.group + (row - token * p.group);
    const int64_t at = static_cast<int64_t>(u.token) + token, out_at = at * p.out_row + head_of * p.out_head;
    const float sink_e = p.sink != nullptr && row < u.rows ? __ldg(p.sink + head_of) : -INFINITY;
    float mx = fmaxf(sink_e * kLog2e, -INFINITY), den = 0.f;  // (a sink of NaN is no maximum)
    bool some = false;
    for (int k = kk; k < n; k += 8) {
      const float* x = ml + slot(k) * 2 * kAttnRows;
      const float m = x[0], z = x[kAttnRows];
      if (!(z <= 0.f)) {
        mx = fmaxf(mx, m);
        some = true;
      }
    }
    some = (__ballot_sync(0xFFFFFFFFu, some) >> (8 * r) & 0xFFu) != 0;
#pragma unroll
    for (int s = 4; s > 0; s >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, s));
    for (int k = kk; k < n; k += 8) {
      const float* x = ml + slot(k) * 2 * kAttnRows;
      den += mx == -INFINITY ? 0.f : fast_exp2(x[0] - mx) * x[kAttnRows];
    }
#pragma unroll
    for (int s = 4; s > 0; s >>= 1) den += __shfl_xor_sync(0xFFFFFFFFu, den, s);
    const float all = mx == -INFINITY ? 1.f : den + sink_weight(sink_e * kLog2e, mx), inverse = 1.f / all;
    float4 acc[2] = {};
    while (true) {
      const float f = mx == -INFINITY ? 0.f : fast_exp2(m0 - mx);
#pragma unroll
      for (int k = 0; k < kFlight; ++k) {
        const float fx = __shfl_sync(0xFFFFFFFFu, f, k), fy = __shfl_sync(0xFFFFFFFFu, f, 8 + k);
        const float fz = __shfl_sync(0xFFFFFFFFu, f, 16 + k), fw = __shfl_sync(0xFFFFFFFFu, f, 24 + k);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          acc[h].x = fmaf(fx, v[k][h].x, acc[h].x);
          acc[h].y = fmaf(fy, v[k][h].y, acc[h].y);
          acc[h].z = fmaf(fz, v[k][h].z, acc[h].z);
          acc[h].w = fmaf(fw, v[k][h].w, acc[h].w);
        }
      }
      k0 += step;
      if (k0 >= n) break;
      fetch();
    }
    if (!few) {
      s_sum[warp][0][lane] = acc[0];
      s_sum[warp][1][lane] = acc[1];
      __syncthreads();
      if (warp < 2) {
        acc[0] = s_sum[0][warp][lane];
#pragma unroll
        for (int k = 1; k < kJoinWarps; ++k) {
          const float4 w = s_sum[k][warp][lane];
          acc[0].x += w.x, acc[0].y += w.y, acc[0].z += w.z, acc[0].w += w.w;
        }
      }
      __syncthreads();
      if (warp >= 2) continue;
    }
    const int col = chunk * 64 + (few ? 0 : warp * 32) + lane;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float f = __shfl_sync(0xFFFFFFFFu, inverse, 8 * i);
      uint16_t* to = p.out + __shfl_sync(0xFFFFFFFFu, out_at, 8 * i) + col;
      const float a = i == 0 ? acc[0].x : i == 1 ? acc[0].y : i == 2 ? acc[0].z : acc[0].w;
      const float b = i == 0 ? acc[1].x : i == 1 ? acc[1].y : i == 2 ? acc[1].z : acc[1].w;
      if (row0 + i < u.rows) {
        if (col < p.d) to[0] = Element<CSA_DTYPE_BF16>::from_float(a * f);
        if (few && col + 32 < p.d) to[32] = Element<CSA_DTYPE_BF16>::from_float(b * f);
      }
    }
    if (p.lse != nullptr && chunk == 0 && (few || warp == 0) && kk == 0 && row < u.rows)
      p.lse[at * p.q_heads + head_of] = some ? (mx + log2f(all)) * kLn2 : sink_e;
  }
}

// The kernels of a call: chunks of 64 columns, where a tile comes from, the cache's format.
struct TileKernels {
  const void *tile, *join, *pack;
  int threads;
  size_t smem;
};
template <typename F>
auto by_chunks(int chunks, F f) {
  return chunks == 2   ? f(std::integral_constant<int, 2>{})
         : chunks == 4 ? f(std::integral_constant<int, 4>{})
                       : f(std::integral_constant<int, 8>{});
}
template <bool PREFIX>
TileKernels tile_kernels(int nc, int source, int format) {
  return by_chunks(nc, [&](auto c) {
    constexpr int NC = decltype(c)::value;
    TileKernels r{};
    r.smem = TileShape<NC>::kSmemBytes;
    r.join = reinterpret_cast<const void*>(attn_join_kernel<NC>);
    auto use = [&](auto src) {
      constexpr int SRC = decltype(src)::value;
      r.tile = reinterpret_cast<const void*>(attn_tile_kernel<NC, SRC, PREFIX>);
      r.threads = TileCta<SRC>::kThreads;
    };
    switch (source) {
      case kFromPacked: use(std::integral_constant<int, kFromPacked>{}); break;
      case kFromBoxes: use(std::integral_constant<int, kFromBoxes>{}); break;
      case kFromBf16: use(std::integral_constant<int, kFromBf16>{}); break;
      case kFromE4m3: use(std::integral_constant<int, kFromE4m3>{}); break;
      default: use(std::integral_constant<int, kFromE2m1>{}); break;
    }
    r.pack = format == CSA_CACHE_BF16   ? reinterpret_cast<const void*>(attn_pack_kernel<NC, CSA_CACHE_BF16, PREFIX>)
             : format == CSA_CACHE_E4M3 ? reinterpret_cast<const void*>(attn_pack_kernel<NC, CSA_CACHE_E4M3, PREFIX>)
                                        : reinterpret_cast<const void*>(attn_pack_kernel<NC, CSA_CACHE_E2M1, PREFIX>);
    return r;
  });
}
// Those behind shared prefixes (csa_attn_prefix.cu: they compile beside the others).
TileKernels prefix_tile_kernels(int nc, int source, int format);

}  // namespace csa
