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
// four warps 16 of the 64 rows), 16 issues the products (17-19 only complete its register
// group), 20-27 fetch: they follow the page table,
// widen 8- and 4-bit codes to bf16 (exact, but for bf16's own subnormals) and store the swizzled tile; a pair of
// 64-column chunks (32 KB) is the unit of the ring, and the next pair's loads are in flight
// in registers while one is stored.
//
// Softmax without a maximum per tile: the weights are taken against a running bound m that
// only moves when some score passes it by 2^8; then m becomes the true maximum and O^T and the
// sums are rescaled. Weights up to 2^8 lose nothing (bf16 and fp32 are floating), and the sums
// stay per lane until the end of the unit.
//
// Shared memory's 128 bytes a cycle bound the products (6 KB for 32 cycles' worth of them at 64
// rows), HBM the decoding of a long cache.
#pragma once

#include <climits>

#include "csa_attn.cuh"
#include "csa_tcgen05.cuh"

namespace csa {

constexpr int kTileSoftWarps = 16, kTileLoadWarps = 8;
constexpr int kSoftThreads = kTileSoftWarps * 32;
constexpr int kSoftCols = 16;  // rows of a softmax thread's group
constexpr int kTileLoaders = kTileLoadWarps * 32;
constexpr int kTileFirstLoader = kTileSoftWarps + 4;
constexpr int kTileThreads = (kTileFirstLoader + kTileLoadWarps) * 32;
// Registers a thread: 896 threads launch with 72, and 16 x 72 + 4 x 40 + 8 x 88 = 28 x 72.
constexpr int kIssueRegs = 40, kLoadRegs = 88;
constexpr int kChunkBytes = kAttnEntries * 128;  // 128 entries x 64 columns
constexpr int kPairBytes = 2 * kChunkBytes;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kNoMax = -1e30f;     // bound of a row that has seen nothing
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
  // shared memory: ring, Q (the output's staging too), P, then the small arrays
  static constexpr int kQOff = kRing * kPairBytes;
  static constexpr int kPOff = kQOff + kQBytes;
  static constexpr int kSmallOff = kPOff + kPBytes;
  static constexpr int kSmemBytes = kSmallOff + 4096 + 1024;  // and the 1024-byte alignment
};

struct TileSmall {
  int64_t row[2][kAttnEntries];  // entry rows of a tile in the pool, -1: none
  float m[kAttnRows];
  float fac[kAttnRows];
  float red[4][kAttnRows];  // column maxima, then weight sums, by quadrant
  int lim[kAttnRows];
  uint64_t full[5], empty[5], scores[2], probs, summed, q_full, q_free, drain;
  uint32_t tmem;
  int stop;
};
static_assert(sizeof(TileSmall) <= 4096, "small arrays");

// 8 columns of an entry as they lie in the cache, and their scale byte.
template <int FORMAT>
struct Piece;
template <>
struct Piece<CSA_CACHE_BF16> {
  uint4 w;
  __device__ __forceinline__ void load(const AttnParams& p, int64_t row, int col) {
    w = make_uint4(0, 0, 0, 0);
    if (row >= 0 && col < p.d)
      w = __ldg(reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(p.data) + row * p.d + col));
  }
  __device__ __forceinline__ uint4 bf16() const { return w; }
};
__device__ __forceinline__ uint32_t scaled_bf16x2(float2 v, float s) { return pack_bf16x2(v.x * s, v.y * s); }
template <>
struct Piece<CSA_CACHE_E4M3> {
  uint2 w;
  uint32_t k;
  __device__ __forceinline__ void load(const AttnParams& p, int64_t row, int col) {
    w = make_uint2(0, 0);
    k = 127;
    if (row >= 0 && col < p.d) {
      w = __ldg(reinterpret_cast<const uint2*>(p.data + row * p.d + col));
      k = __ldg(p.scales + row * (p.d / CSA_CACHE_GROUP) + col / CSA_CACHE_GROUP);
    }
  }
  __device__ __forceinline__ uint4 bf16() const {
    const float s = scale_value(k);
    return make_uint4(scaled_bf16x2(e4m3x2_to_float2(w.x & 0xFFFF), s), scaled_bf16x2(e4m3x2_to_float2(w.x >> 16), s),
                      scaled_bf16x2(e4m3x2_to_float2(w.y & 0xFFFF), s), scaled_bf16x2(e4m3x2_to_float2(w.y >> 16), s));
  }
};
template <>
struct Piece<CSA_CACHE_E2M1> {
  uint32_t w, k;
  __device__ __forceinline__ void load(const AttnParams& p, int64_t row, int col) {
    w = 0;
    k = 127;
    if (row >= 0 && col < p.d) {
      w = __ldg(reinterpret_cast<const uint32_t*>(p.data + row * (p.d / 2) + col / 2));
      k = __ldg(p.scales + row * (p.d / CSA_CACHE_GROUP) + col / CSA_CACHE_GROUP);
    }
  }
  __device__ __forceinline__ uint4 bf16() const {
    const float s = scale_value(k);
    return make_uint4(scaled_bf16x2(e2m1x2_to_float2(w), s), scaled_bf16x2(e2m1x2_to_float2(w >> 8), s),
                      scaled_bf16x2(e2m1x2_to_float2(w >> 16), s), scaled_bf16x2(e2m1x2_to_float2(w >> 24), s));
  }
};

__device__ __forceinline__ void sts128(uint32_t addr, uint4 v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
               : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
  return v;
}

// Waits are bounded: one that runs out sets the CTA's stop word and reports, after which every
// wait returns at once and every role runs through the rest of its (finite) loops, so that
// the barriers among its warps stay matched; the products already issued are drained before
// the tensor memory is freed. Nothing else is ever in flight.
__device__ __forceinline__ void tile_wait(TileSmall& sm, const AttnParams& p, uint64_t* bar, uint32_t parity) {
  if (mbar_try_wait(bar, parity)) return;
  const long long t0 = clock64();
  while (!mbar_try_wait(bar, parity)) {
    if (*reinterpret_cast<volatile int*>(&sm.stop) != 0) return;
    if (clock64() - t0 > kWaitCycles) {
      stop_pipeline(&sm.stop, p.dev_error);
      return;
    }
  }
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

// The runs of tiles of one unit in a CTA's share.
struct SegmentWalk {
  const AttnParams& p;
  int unit, t0, t1, left;  // (a CTA's share stays below 2^31 tiles: checked on the host)
  AttnUnit u;
  __device__ __forceinline__ SegmentWalk(const AttnParams& pp) : p(pp) {
    const AttnStart* at = p.starts + blockIdx.x;
    take(reinterpret_cast<const int4*>(&at->u));
    const int4 v = __ldg(reinterpret_cast<const int4*>(at) + 3);
    unit = v.x;
    t0 = v.y;
    left = v.z;
    bound();
  }
  __device__ __forceinline__ void take(const int4* at) {
    const int4 a = __ldg(at), b = __ldg(at + 1), c = __ldg(at + 2);
    u = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w, c.x, c.y, {0, 0}};
  }
  __device__ __forceinline__ void bound() { t1 = left < u.tiles - t0 ? t0 + left : u.tiles; }
  __device__ __forceinline__ bool valid() const { return left > 0; }
  __device__ __forceinline__ void next() {
    left -= t1 - t0;
    ++unit;
    t0 = 0;
    if (left > 0) {
      take(reinterpret_cast<const int4*>(p.units + unit));
      bound();
    }
  }
};

// ------------------------------------------------------------------------------ the fetchers
template <int NC, int FORMAT>
__device__ void tile_fetch(const AttnParams& p, TileSmall& sm, uint32_t base) {
  using SH = TileShape<NC>;
  const int lt = threadIdx.x - kTileFirstLoader * 32;
  const int piece = lt & 15, rg = lt >> 4;  // 8 columns of the pair's 128; rows rg, rg + 16, ...
  const uint32_t dst = (piece >> 3) * kChunkBytes + rg * 128 + (((piece & 7) ^ (rg & 7)) << 4);

  SegmentWalk w(p);
  if (!w.valid()) return;
  int tile = w.t0, pair = 0, buf = 0, seg = 0;
  bool q_due = false;  // the current segment's q is still to be stored

  // The tile's rows in the pool, by the first 128 threads, then a barrier of all. The page numbers
  // are read one tile ahead within a unit.
  int page = -1, ahead = -1;  // this thread's page of tile `ahead`
  auto read_page = [&](int tl) {
    const int e = tl * kAttnEntries + lt;
    ahead = tl;
    page = lt < kAttnEntries && e < w.u.seen
               ? __ldg(p.table + static_cast<int64_t>(w.u.s) * p.max_pages + e / p.page_size)
               : -1;
  };
  auto rows = [&](bool new_unit) {
    if (new_unit || ahead != tile) read_page(tile);
    if (lt < kAttnEntries) {
      const int e = tile * kAttnEntries + lt;
      int64_t r = -1;
      if (e < w.u.seen) {
        if (page >= 0 && page < p.num_pages)
          r = (static_cast<int64_t>(page) * p.page_size + e % p.page_size) * p.kv_heads + w.u.kvh;
        else if (p.dev_error != nullptr)
          *p.dev_error = CSA_DEVERR_PAGE;
      }
      sm.row[buf][lt] = r;
    }
    named_barrier(6, kTileLoaders);
    if (tile + 1 < w.t1) read_page(tile + 1);
  };
  auto load = [&](Piece<FORMAT>(&v)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i].load(p, sm.row[buf][i * 16 + rg], pair * 128 + piece * 8);
  };
  auto arrive = [&](uint64_t* bar) {
    fence_proxy_async_smem();
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
  };
  RingAt<SH::kRing> ring;
  auto store = [&](const Piece<FORMAT>(&v)[8]) {
    tile_wait(sm, p, &sm.empty[ring.slot], ring.lap ^ 1u);
    const uint32_t at = base + ring.slot * kPairBytes + dst;
#pragma unroll
    for (int i = 0; i < 8; ++i) sts128(at + i * 16 * 128, v[i].bf16());
    arrive(&sm.full[ring.slot]);
    ring.next();
  };
  // the unit's rows of q, zeros behind the last row and column
  auto load_q = [&](int kvh, int block, int token, int all) {
    if (seg > 0) tile_wait(sm, p, &sm.q_free, static_cast<uint32_t>(seg - 1) & 1u);
    constexpr int kPer = NC * 8;  // 16-byte pieces of a row
#pragma unroll 2
    for (int i = lt; i < kAttnRows * kPer; i += kTileLoaders) {
      const int r = i / kPer, c = i % kPer, row = block * kAttnRows + r;
      uint4 v = make_uint4(0, 0, 0, 0);
      if (row < all && c * 8 < p.d) {
        const int tok = row / p.group, head = kvh * p.group + row % p.group;
        v = __ldg(reinterpret_cast<const uint4*>(p.q + (static_cast<int64_t>(token) + tok) * p.q_row +
                                                 head * p.q_head + c * 8));
      }
      sts128(base + SH::kQOff + (c >> 3) * (kAttnRows * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4), v);
    }
    arrive(&sm.q_full);
    ++seg;
  };
  // moves on to the next pair; false at the end of the CTA's share
  auto advance = [&]() {
    if (++pair < SH::kPairs) return true;
    pair = 0;
    bool new_unit = false;
    if (++tile == w.t1) {
      w.next();
      if (!w.valid()) return false;
      tile = w.t0;
      new_unit = q_due = true;
    }
    buf ^= 1;
    rows(new_unit);
    return true;
  };
  // q of a segment goes in after its first tile's pairs (the fetch of these need not wait for
  // the previous segment's output to leave the buffer); the first segment's at once
  Piece<FORMAT> va[8], vb[8];
  rows(true);
  load(va);
  load_q(w.u.kvh, w.u.block, w.u.token, w.u.rows);
  bool more = true;
  auto step = [&](Piece<FORMAT>(&cur)[8], Piece<FORMAT>(&nxt)[8]) {
    const bool q_after = q_due && pair == SH::kPairs - 1;
    const int kvh = w.u.kvh, block = w.u.block, token = w.u.token, all = w.u.rows;
    if (q_after) q_due = false;
    more = advance();
    if (more) load(nxt);
    store(cur);
    if (q_after) load_q(kvh, block, token, all);
  };
  while (true) {
    step(va, vb);
    if (!more) break;
    step(vb, va);
    if (!more) break;
  }
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
  for (SegmentWalk w(p); w.valid(); w.next(), ++seg) {
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

// ------------------------------------------------------------------------- the softmax warps
template <int NC>
__device__ void tile_softmax(const AttnParams& p, TileSmall& sm, unsigned char* smem, uint32_t base, uint32_t tmem) {
  using SH = TileShape<NC>;
  const int tid = threadIdx.x, lane = tid & 31, quad = (tid >> 5) & 3, group = tid >> 7;
  const int c0 = group * kSoftCols;     // the rows (columns of S^T) of this group of four warps
  const int e0 = quad * 32 + lane;      // the entry (row of S^T) of this thread
  const uint32_t lanes = tmem + (static_cast<uint32_t>(quad * 32) << 16);
  // (a scale of 0, under which every score is equal, becomes one that no score can show)
  const float sl2 = p.scale == 0.f ? 1.17549435e-38f : p.scale * kLog2e;
  uint32_t t = 0;  // tiles so far
  auto barrier_group = [&]() { named_barrier(1 + group, 128); };

  for (SegmentWalk w(p); w.valid(); w.next()) {
    const AttnUnit u = w.u;
    const int row0 = u.block * kAttnRows;
    // what each row sees; rows behind the last one see everything (they are never stored)
    if (tid < kAttnRows) {
      sm.lim[tid] = row0 + tid < u.rows
                        ? visible(static_cast<int64_t>(u.first) + (row0 + tid) / p.group, p.ratio, u.n)
                        : INT_MAX;
      sm.m[tid] = kNoMax;
    }
    named_barrier(5, kSoftThreads);
    float l[kSoftCols];
#pragma unroll
    for (int c = 0; c < kSoftCols; ++c) l[c] = 0.f;

    for (int j = w.t0; j < w.t1; ++j, ++t) {
      const int e = j * kAttnEntries + e0;
      const bool masked = (j + 1) * static_cast<int64_t>(kAttnEntries) > u.seen_all;
      const uint32_t s_at = lanes + SH::kTmemS + (t & 1u) * kAttnRows + c0;
      tile_wait(sm, p, &sm.scores[t & 1u], (t >> 1) & 1u);
      tc_fence_after();
      float s[kSoftCols];
      bool odd = false;  // a masked score of this entry is not finite
      auto take = [&](bool subtract) {
        tmem_load16(s_at, s);
        if (masked) {
#pragma unroll
          for (int c = 0; c < kSoftCols; ++c)
            if (e >= sm.lim[c0 + c]) {
              odd = odd || !(fabsf(s[c]) <= 3.4028234e38f);
              s[c] = sl2 < 0.f ? INFINITY : -INFINITY;  // -inf once scaled
            }
        }
#pragma unroll
        for (int c = 0; c < kSoftCols; c += 4) {
          const float4 m = subtract ? *reinterpret_cast<const float4*>(&sm.m[c0 + c]) : make_float4(0.f, 0.f, 0.f, 0.f);
          s[c] = fmaf(s[c], sl2, -m.x);
          s[c + 1] = fmaf(s[c + 1], sl2, -m.y);
          s[c + 2] = fmaf(s[c + 2], sl2, -m.z);
          s[c + 3] = fmaf(s[c + 3], sl2, -m.w);
        }
      };
      take(true);
      float top = fmaxf(s[0], s[1]);
#pragma unroll
      for (int c = 2; c < kSoftCols; c += 2) top = fmax3(top, s[c], s[c + 1]);
      if (named_barrier_or(1 + group, 128, top > kRescaleAt)) {
        // new bounds: the true maxima so far
        take(false);
        float mine = kNoMax;
#pragma unroll
        for (int c = 0; c < kSoftCols; ++c) {
          const float v = warp_max_f32(s[c]);
          if (lane == c) mine = v;
        }
        if (lane < kSoftCols) sm.red[quad][c0 + lane] = mine;
        barrier_group();
        if (quad == 0 && lane < kSoftCols) {
          const int c = c0 + lane;
          const float old = sm.m[c];
          float m = fmaxf(fmaxf(sm.red[0][c], sm.red[1][c]), fmaxf(sm.red[2][c], sm.red[3][c]));
          m = fmaxf(old, m);
          sm.fac[c] = fast_exp2(old - m);
          sm.m[c] = m;
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
        take(true);
      }
      // weights; their sums before rounding
      uint32_t w2[kSoftCols / 2];
#pragma unroll
      for (int c = 0; c < kSoftCols; c += 2) {
        const float a = fast_exp2(s[c]), b = fast_exp2(s[c + 1]);
        l[c] += a;
        l[c + 1] += b;
        w2[c / 2] = pack_bf16x2(a, b);
      }
      if (j > w.t0) tile_wait(sm, p, &sm.summed, (t - 1u) & 1u);  // P is free
      const uint32_t row = base + SH::kPOff + e0 * 128;
#pragma unroll
      for (int c = 0; c < 2; ++c)
        sts128(row + (((group * 2 + c) ^ (e0 & 7)) << 4), make_uint4(w2[4 * c], w2[4 * c + 1], w2[4 * c + 2], w2[4 * c + 3]));
      if (odd) {
        // 0 * NaN would reach the rows that do not see this entry: its non-finite values become
        // 0 before the second product (the rows that see it have a non-finite score)
#pragma unroll 1
        for (int b = 0; b < NC; ++b) {
          const int slot = static_cast<int>((t * SH::kPairs + (b >> 1)) % SH::kRing);
          unsigned char* at = smem + slot * kPairBytes + (b & 1) * kChunkBytes + e0 * 128;
#pragma unroll 1
          for (int i = 0; i < 64; ++i) {
            uint16_t* v = reinterpret_cast<uint16_t*>(at) + i;
            if ((*v & 0x7F80u) == 0x7F80u) *v = 0;
          }
        }
      }
      fence_proxy_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.probs);
    }

    // the unit's (or its piece's) sums are complete
    tile_wait(sm, p, &sm.summed, (t - 1u) & 1u);
    tc_fence_after();
    float mine = 0.f;
#pragma unroll
    for (int c = 0; c < kSoftCols; ++c) {
      float v = l[c];
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
      if (lane == c) mine = v;
    }
    if (lane < kSoftCols) sm.red[quad][c0 + lane] = mine;
    barrier_group();
    const bool whole = w.t0 == 0 && w.t1 == u.tiles;
    const int64_t piece = 2 * static_cast<int64_t>(blockIdx.x) + (w.t0 == 0 ? 1 : 0);
    if (quad == 0 && lane < kSoftCols) {
      const int c = c0 + lane;
      const float z = (sm.red[0][c] + sm.red[1][c]) + (sm.red[2][c] + sm.red[3][c]), m = sm.m[c];
      if (!whole) {
        float* ml = p.part_ml + piece * 2 * kAttnRows;
        ml[c] = m;
        ml[kAttnRows + c] = z;
      } else {
        const int row = row0 + c;
        const int head = u.kvh * p.group + row % p.group;
        const float sink_e = p.sink != nullptr && row < u.rows ? p.sink[head] : -INFINITY;
        const float sink = sink_e * kLog2e;
        const float mx = fmaxf(z > 0.f || z != z ? m : -INFINITY, sink);
        const float old = mx == -INFINITY ? 0.f : fast_exp2(m - mx);
        const float den = mx == -INFINITY ? 0.f : z * old + fast_exp2(sink - mx);
        sm.fac[c] = mx == -INFINITY ? 0.f : old / den;
        if (p.lse != nullptr && row < u.rows)
          p.lse[(static_cast<int64_t>(u.token) + row / p.group) * p.q_heads + head] =
              z == 0.f ? sink_e : (mx + log2f(den)) * kLn2;
      }
    }
    barrier_group();
    if (whole) {
      // O^T times the rows' factors, as bf16 rows in q's buffer, then out in 16-byte pieces
      uint16_t* stage = reinterpret_cast<uint16_t*>(smem + SH::kQOff);
#pragma unroll 1
      for (int b = 0; b < SH::kPairs; ++b) {
        float v[kSoftCols];
        tmem_load16(lanes + SH::kTmemO + b * kAttnRows + c0, v);
#pragma unroll
        for (int c = 0; c < kSoftCols; ++c)
          stage[(c0 + c) * SH::kDpad + b * 128 + e0] = Element<CSA_DTYPE_BF16>::from_float(v[c] * sm.fac[c0 + c]);
      }
      tc_fence_before();
      barrier_group();
      constexpr int kPer = NC * 8;
#pragma unroll 1
      for (int i = (tid & 127); i < kSoftCols * kPer; i += 128) {
        const int r = c0 + i / kPer, c = i % kPer, row = row0 + r;
        if (row < u.rows && c * 8 < p.d) {
          const uint4 v = lds128(base + SH::kQOff + r * (SH::kDpad * 2) + c * 16);
          *reinterpret_cast<uint4*>(p.out + (static_cast<int64_t>(u.token) + row / p.group) * p.out_row +
                                    (u.kvh * p.group + row % p.group) * p.out_head + c * 8) = v;
        }
      }
    } else {
      float* o = p.part_o + piece * kAttnRows * SH::kDpad;
#pragma unroll 1
      for (int b = 0; b < SH::kPairs; ++b) {
        float v[kSoftCols];
        tmem_load16(lanes + SH::kTmemO + b * kAttnRows + c0, v);
#pragma unroll
        for (int c = 0; c < kSoftCols; ++c) o[(c0 + c) * SH::kDpad + b * 128 + e0] = v[c];
      }
      tc_fence_before();
    }
    named_barrier(5, kSoftThreads);  // the small arrays and the staging are free again
    if (lane == 0) mbar_arrive(&sm.q_free);
  }
}

template <int NC, int FORMAT>
__global__ void __launch_bounds__(kTileThreads, 1) attn_tile_kernel(const __grid_constant__ AttnParams p) {
  using SH = TileShape<NC>;
  extern __shared__ unsigned char raw[];
  unsigned char* smem = raw + ((1024u - (smem_addr(raw) & 1023u)) & 1023u);
  TileSmall& sm = *reinterpret_cast<TileSmall*>(smem + SH::kSmallOff);
  const uint32_t base = smem_addr(smem);
  const int warp = threadIdx.x >> 5;
  if (warp == 0) tmem_alloc(&sm.tmem, SH::kTmemColumns);
  if (threadIdx.x == 32) {
    for (int i = 0; i < SH::kRing; ++i) {
      mbar_init(&sm.full[i], kTileLoadWarps);
      mbar_init(&sm.empty[i], 1);
    }
    mbar_init(&sm.scores[0], 1);
    mbar_init(&sm.scores[1], 1);
    mbar_init(&sm.probs, kTileSoftWarps);
    mbar_init(&sm.summed, 1);
    mbar_init(&sm.q_full, kTileLoadWarps);
    mbar_init(&sm.q_free, kTileSoftWarps);
    mbar_init(&sm.drain, 1);
    sm.stop = 0;
    fence_mbar_init();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem;
  pdl_wait();
  const bool run = *p.status == 0;
  if (warp >= kTileFirstLoader) {
    regs_up<kLoadRegs>();
    if (run) tile_fetch<NC, FORMAT>(p, sm, base);
  } else if (warp >= kTileSoftWarps) {
    regs_down<kIssueRegs>();
    if (run && warp == kTileSoftWarps) tile_products<NC>(p, sm, base, tmem);
  } else if (run) {
    tile_softmax<NC>(p, sm, smem, base, tmem);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 0) tmem_free(tmem, SH::kTmemColumns);
}

// Joins the pieces of the units that CTAs share: block (i, y) the rows y*8 .. y*8+7 of the unit
// whose first piece is CTA i's last one. A warp per row.
template <int NC>
__global__ void __launch_bounds__(256) attn_join_kernel(const __grid_constant__ AttnParams p) {
  using SH = TileShape<NC>;
  pdl_wait();
  if (*p.status != 0) return;
  const int64_t all_tiles = *p.tiles;
  const int ctas = static_cast<int>(all_tiles < p.ctas ? all_tiles : p.ctas);
  const int i = blockIdx.x;
  if (i + 1 >= ctas) return;
  const AttnStart& nx = p.starts[i + 1];
  if (nx.tile == 0) return;                                             // ends with its share
  if (p.unit_first[nx.unit] < attn_share(all_tiles, p.ctas, i)) return;  // begins before it
  const int64_t end = p.unit_first[nx.unit + 1];
  int last = i + 1;  // last CTA with a piece
  while (last + 1 < ctas && attn_share(all_tiles, p.ctas, last + 1) < end) ++last;
  const AttnUnit u = p.units[nx.unit];
  const int r = blockIdx.y * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  const int row = u.block * kAttnRows + r;
  if (row >= u.rows) return;
  const int head = u.kvh * p.group + row % p.group;
  const int64_t token = static_cast<int64_t>(u.token) + row / p.group;

  auto slot = [&](int k) { return 2 * static_cast<int64_t>(k) + (k == i ? 1 : 0); };
  const float sink_e = p.sink != nullptr ? p.sink[head] : -INFINITY, sink = sink_e * kLog2e;
  float mx = sink;
  bool some = false;
  for (int k = i; k <= last; ++k) {
    const float* ml = p.part_ml + slot(k) * 2 * kAttnRows;
    if (!(ml[kAttnRows + r] <= 0.f)) {
      mx = fmaxf(mx, ml[r]);
      some = true;
    }
  }
  float den = mx == -INFINITY ? 0.f : fast_exp2(sink - mx);
  float acc[SH::kDpad / 32];
#pragma unroll
  for (int c = 0; c < SH::kDpad / 32; ++c) acc[c] = 0.f;
  if (mx != -INFINITY) {
    for (int k = i; k <= last; ++k) {
      const float* ml = p.part_ml + slot(k) * 2 * kAttnRows;
      const float f = fast_exp2(ml[r] - mx);
      den += f * ml[kAttnRows + r];
      const float4* o = reinterpret_cast<const float4*>(p.part_o + (slot(k) * kAttnRows + r) * SH::kDpad);
#pragma unroll
      for (int c = 0; c < SH::kDpad / 128; ++c) {
        const float4 v = o[c * 32 + lane];
        acc[4 * c] += f * v.x;
        acc[4 * c + 1] += f * v.y;
        acc[4 * c + 2] += f * v.z;
        acc[4 * c + 3] += f * v.w;
      }
    }
  }
  const float inv = mx == -INFINITY ? 0.f : 1.f / den;
  uint16_t* out = p.out + token * p.out_row + head * p.out_head;
#pragma unroll
  for (int c = 0; c < SH::kDpad / 128; ++c) {
    const int col = (c * 32 + lane) * 4;
    if (col < p.d)
      *reinterpret_cast<uint2*>(out + col) = make_uint2(pack_bf16x2(acc[4 * c] * inv, acc[4 * c + 1] * inv),
                                                        pack_bf16x2(acc[4 * c + 2] * inv, acc[4 * c + 3] * inv));
  }
  if (p.lse != nullptr && lane == 0)
    p.lse[token * p.q_heads + head] = some ? (mx + log2f(den)) * kLn2 : sink_e;
}

}  // namespace csa
