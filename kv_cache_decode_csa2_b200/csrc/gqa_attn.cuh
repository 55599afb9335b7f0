// What the kernels of grouped-query attention over the FP4 cache share: the
// arguments, which rows a query sees, and how the work of a launch is cut
// into CTAs.
//
// The work of a launch is one sequence of tiles: for every item (a query, or
// a block of queries, with a group of KV heads) the kTile-row steps of the
// cache that it sees.  Each of n_cta CTAs takes an equal run of tiles, so
// sequences of any lengths load the device evenly and one long sequence uses
// all of it.  A run covers whole items and at most two parts of items that
// other CTAs share; each part leaves (max, sum, O) in the workspace and the
// combine kernel joins an item's parts in CTA order, so results do not depend
// on timing.
#pragma once

#include "csa2_device.cuh"
#include "internal.h"

namespace csa2 {

constexpr int kPageStep = 64;      // pages are multiples of this many rows

struct GqaArgs {
  const uint16_t* q;               // bf16 [nq][Hq][D]
  uint16_t* out;                   // bf16 [nq][Hq][D]
  float* lse;                      // [nq][Hq] or nullptr
  const uint8_t* base[4];          // K codes, K scales, V codes, V scales
  int64_t rb[4];
  RowMap map[4];
  int32_t page_shift[4];           // log2 of the rows per page (-1: not a power of two)
  int32_t one_map;                 // all four planes place rows alike
  const int32_t* seq_of_query;
  const int32_t* query_pos;
  int32_t nq, Hkv, G, window, n_sink;
  float scale_log2;
  int32_t n_cta;                   // CTAs of the main kernel
  int32_t vh;                      // virtual heads: (KV head, run of up to 8 NT query heads)
  int32_t subs;                    // runs per KV head
  int32_t per_cta;                 // virtual heads per CTA
  int32_t groups;                  // CTA groups per query: ceil(vh / per_cta)
  int64_t* starts;                 // [nq + 1] tiles of one group before each query; tiles per CTA
  float* part_o;                   // [2 n_cta][rows][D] unnormalised O of a part
  float2* part_ml;                 // [2 n_cta][rows] (offset max in log2 units, sum)
  int32_t* status;
};

// The tiles of T rows that a query at position pos sees rows of: tile x starts
// at row x T, from `sink` on `gap` rows later (the rows between the sinks and
// the window).
struct TileRange {
  int32_t sink, gap, count;
  __device__ __forceinline__ int32_t row(int32_t x, int T) const { return x * T + (x >= sink ? gap : 0); }
};
template <int T>
__device__ __forceinline__ TileRange tile_range(int32_t pos, int32_t window, int32_t n_sink) {
  if (pos < 0) return TileRange{0, 0, 0};
  const int32_t last = pos / T;
  const int32_t first = window > 0 && pos >= window ? (pos - window + 1) / T : 0;
  const int32_t sink = n_sink > 0 ? (n_sink - 1) / T + 1 : 0;
  if (first <= sink) return TileRange{0, 0, last + 1};      // no tile between them
  return TileRange{sink, (first - sink) * T, sink + last + 1 - first};
}

// The rows a query sees, relative to a tile: r <= hi && (r >= lo || r < sk).
struct Seen {
  int32_t hi, lo, sk;
  __device__ __forceinline__ bool row(int32_t r) const { return r <= hi && (r >= lo || r < sk); }
  __device__ __forceinline__ bool all(int32_t n) const { return n - 1 <= hi && (lo <= 0 || n <= sk); }
  __device__ __forceinline__ Seen from(int32_t p0) const { return Seen{hi - p0, lo - p0, sk - p0}; }
};
__device__ __forceinline__ Seen seen_rows(int32_t pos, int32_t window, int32_t n_sink) {
  return Seen{pos, window > 0 && pos >= window ? pos - window + 1 : 0, n_sink};
}

}  // namespace csa2
