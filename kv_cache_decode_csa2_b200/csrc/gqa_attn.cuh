// What the kernels of grouped-query attention over the FP4 cache share: the
// arguments, which rows a query sees, and how the work of a launch is cut
// into CTAs.
//
// The work of a launch is one sequence of units: for every item (a query, or
// a block of queries, with a group of KV heads) the kUnit-row steps of the
// cache that it sees.  Each of n_cta CTAs takes an equal run of units, so
// sequences of any lengths load the device evenly and one long sequence uses
// all of it.  A run covers whole items and at most two parts of items that
// other CTAs share; each part leaves (max, sum, O) in the workspace and the
// combine kernel joins an item's parts in CTA order, so results do not depend
// on timing.
#pragma once

#include "csa2_device.cuh"
#include "internal.h"

namespace csa2 {

constexpr int kUnit = 64;          // cache rows per unit; pages are whole units

struct GqaArgs {
  const uint16_t* q;               // bf16 [nq][Hq][D]
  uint16_t* out;                   // bf16 [nq][Hq][D]
  float* lse;                      // [nq][Hq] or nullptr
  const uint8_t* base[4];          // K codes, K scales, V codes, V scales
  int64_t rb[4];
  RowMap map[4];
  int32_t page_shift[4];           // log2 of the units per page (-1: not a power of two)
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
  int64_t* starts;                 // [nq + 1] units of one group before each query; the total
  float* part_o;                   // [2 n_cta][rows][D] unnormalised O of a part
  float2* part_ml;                 // [2 n_cta][rows] (offset max in log2 units, sum)
  int32_t* status;
};

// The units of a query at position pos: those from 0 to pos, or, where the
// sinks and the window leave a gap, the sinks' units and then the window's.
struct UnitRange {
  int32_t sink_units, first, count;   // unit u: u < sink_units ? u : first + u - sink_units
  __device__ __forceinline__ int32_t row(int32_t u) const {
    return (u < sink_units ? u : first + (u - sink_units)) * kUnit;
  }
};
__device__ __forceinline__ UnitRange unit_range(int32_t pos, int32_t window, int32_t n_sink) {
  UnitRange r{0, 0, 0};
  if (pos < 0) return r;
  const int32_t last = pos / kUnit;
  const int32_t wstart = window > 0 && pos >= window ? pos - window + 1 : 0;
  const int32_t sink_units = n_sink > 0 ? (n_sink - 1) / kUnit + 1 : 0;
  const int32_t first = wstart / kUnit;
  if (first <= sink_units) {          // no unit between them: one run
    r.count = last + 1;
    return r;
  }
  r.sink_units = sink_units;
  r.first = first;
  r.count = sink_units + last + 1 - first;
  return r;
}
__device__ __forceinline__ bool sees(int32_t row, int32_t pos, int32_t window, int32_t n_sink) {
  return row <= pos && (window <= 0 || row > pos - window || row < n_sink);
}
// Whether any of rows [row, row + n) is seen.
__device__ __forceinline__ bool sees_any(int32_t row, int32_t n, int32_t pos, int32_t window, int32_t n_sink) {
  return row <= pos && (window <= 0 || row + (n - 1) > pos - window || row < n_sink);
}

}  // namespace csa2
