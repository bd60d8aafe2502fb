// csa_attn.cuh -- what the kernels of the cache attention share: the call's parameters, the
// visibility rule, and the work list that the plan kernel leaves in the workspace.
#pragma once

#include <climits>
#include <stdint.h>

#include "csa_compressor.h"
#include "csa_element.cuh"

namespace csa {

constexpr int kAttnRows = 64;      // (token, head) rows of a unit
constexpr int kAttnEntries = 128;  // entries of a tile

// A unit is up to 64 consecutive rows (token, head of the group) of one sequence and cache head; its
// work is a run of tiles of 128 entries, at least one. The work of all units in order is split
// evenly over the workers, a CTA each (AttnShares).
struct alignas(16) AttnUnit {
  int32_t s, kvh, block, tiles;
  int32_t token, rows;  // the sequence's first token, and its rows
  int32_t first;        // position of that token
  int32_t n;            // the sequence's entries
  int32_t seen_all;     // entries that every row of the unit sees
  int32_t seen;         // entries that some row sees
  int32_t pad[2];
};
struct alignas(16) AttnStart {  // a worker's share: its first unit, the tile there, and how many tiles
  AttnUnit u;
  int32_t unit, tile;
  int64_t left;
};
struct alignas(16) AttnJoin {  // a unit whose tiles several workers share, from `worker` on
  AttnUnit u;
  int32_t worker, pieces;
  int32_t pad[2];
};
struct alignas(16) AttnHead {
  int32_t status;  // 0, or why the call's lengths were refused
  int32_t few, many;  // shared units, of few pieces and of many
  int32_t pad;
};
static_assert(sizeof(AttnUnit) == 48 && sizeof(AttnStart) == 64 && sizeof(AttnJoin) == 64 && sizeof(AttnHead) == 16,
              "read in 16-byte pieces");

struct AttnParams {
  const uint16_t* q;
  const int32_t* cu;
  const uint8_t* data;
  const uint8_t* scales;
  const int32_t* table;
  const int32_t* entries;
  const int32_t* first;
  const float* sink;
  uint16_t* out;
  float* lse;
  int32_t* dev_error;
  // workspace
  AttnHead* head;
  AttnStart* starts;    // [workers]
  AttnJoin* joins;      // [workers]: those of few pieces from its start, of many from its end
  AttnUnit* units;      // [max_units]
  int64_t* unit_first;  // [max_units + 1]: where each unit's work begins
  float* part_o;        // [2 workers][64 x dpad]: sums of the pieces of shared units
  float* part_ml;       // [2 workers][2][64]: their maxima (in log2) and weight sums
  uint16_t* packed;     // chunks: the sequences' entries as bf16 rows [S][kv_heads][packed_rows][dpad]
  int64_t q_row, q_head, out_row, out_head;
  int64_t tokens, num_pages, max_entries, max_units;
  int S, q_heads, kv_heads, group, d, max_pages, page_size, ratio;
  int workers, unit_cost;
  int packed_rows;  // rows of a sequence's cache head in `packed`, a multiple of 128
  int box_rows;     // entries of a tensor copy's box from the pages
  float scale;  // softmax_scale
  int withhold_tile;      // test hook: tile of the first CTA's first unit that never comes, -1: none
  long long wait_cycles;  // bound of each wait on a barrier in shared memory, in SM clock cycles
};

// Entries that the token at position pos sees, of a sequence's n.
__device__ __forceinline__ int visible(int64_t pos, int ratio, int n) {
  if (ratio == 0) return n;
  if (pos < 0) return 0;
  const uint64_t done = pos < 0xFFFFFFFFll ? static_cast<uint32_t>(pos + 1) / static_cast<uint32_t>(ratio)
                                           : static_cast<uint64_t>(pos + 1) / static_cast<uint32_t>(ratio);
  return done < static_cast<uint64_t>(n) ? static_cast<int>(done) : n;
}
// Rows of a sequence and cache head (below 2^31 - 256: tokens * q_heads is).
__device__ __forceinline__ int sequence_rows(const AttnParams& p, int s) {
  return (__ldg(p.cu + s + 1) - __ldg(p.cu + s)) * p.group;
}
// A unit of sequence s from its place.
__device__ __forceinline__ AttnUnit make_unit(const AttnParams& p, int s, int kvh, int block) {
  AttnUnit u{};
  u.s = s;
  u.kvh = kvh;
  u.block = block;
  u.token = __ldg(p.cu + s);
  u.rows = sequence_rows(p, s);
  u.first = p.first != nullptr ? __ldg(p.first + s) : 0;
  u.n = __ldg(p.entries + s);
  const int last = min(block * kAttnRows + kAttnRows, u.rows) - 1;
  u.seen_all = visible(static_cast<int64_t>(u.first) + block * kAttnRows / p.group, p.ratio, u.n);
  u.seen = visible(static_cast<int64_t>(u.first) + last / p.group, p.ratio, u.n);
  u.tiles = u.seen <= kAttnEntries ? 1 : (u.seen - 1) / kAttnEntries + 1;
  return u;
}

// Worker i's share of the work, a unit counting its tiles and unit_cost more (loading q, bringing
// the output out): [share(i), share(i + 1)) of n = min(work, workers) equal ones.
struct AttnShares {
  int64_t work, q;
  int n, r;
  __host__ __device__ __forceinline__ AttnShares(int64_t w, int workers) : work(w) {
    n = w < workers ? static_cast<int>(w) : workers;
    const int d = n > 0 ? n : 1;
    q = w < INT_MAX ? static_cast<int>(w) / d : w / d;
    r = static_cast<int>(w - q * d);
  }
  __host__ __device__ __forceinline__ int64_t operator()(int i) const {
    return i >= n ? work : q * i + static_cast<int>(static_cast<uint32_t>(r) * static_cast<uint32_t>(i) / static_cast<uint32_t>(n));
  }
  // the worker whose share x < work lies in, or one next to it
  __device__ __forceinline__ int near(int64_t x) const {
    return min(n - 1, static_cast<int>(static_cast<float>(x) * (static_cast<float>(n) / static_cast<float>(work))));
  }
};

}  // namespace csa
