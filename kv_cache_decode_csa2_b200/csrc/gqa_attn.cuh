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
#include "fp4_device.cuh"
#include "internal.h"

namespace csa2 {

constexpr int kPageStep = 64;      // pages are multiples of this many rows

// The item that a CTA's run starts in the middle of.
struct GqaJoint {
  int64_t i0, i1;                  // the item's tiles (i0 < 0: it did not begin in the CTA before, or there is none)
  int64_t run;                     // tiles per CTA
  int32_t q0, n_q, grp;            // its queries and which of their items it is
};

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
  int32_t limit;                   // positions from here on have no row in any sequence
  float scale_log2;
  int32_t n_cta;                   // CTAs of the main kernel
  int32_t q_tile;                  // queries per item of the block kernel (0: the split kernel, one query per item)
  int32_t vh;                      // virtual heads: (KV head, run of up to 8 NT query heads)
  int32_t subs;                    // runs per KV head
  int32_t per_cta;                 // virtual heads per CTA
  int32_t groups;                  // items per query or block: ceil(vh / per_cta)
  GqaJoint* joints;                // [n_cta] what each CTA shares with the one before it
  float* part_o;                   // [2 n_cta][rows][D] unnormalised O of a part
  float2* part_ml;                 // [2 n_cta][rows] (reference, sum of weights)
  int32_t* status;
};

// Positions are held below this: 256 runs of a block then have fewer than 2^31 tiles.
constexpr int64_t kMaxPositions = 1 << 29;
// The position that query i works with: one past its plane's rows is taken as
// the last there is (and reported by looks_empty), so that neither the work
// nor a neighbour's rows depend on it.
__device__ __forceinline__ int32_t position(const GqaArgs& a, int64_t i) {
  return min(__ldg(a.query_pos + i), a.limit - 1);
}

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
  // whether any of rows a to b is seen
  __device__ __forceinline__ bool some(int32_t a, int32_t b) const {
    const int32_t e = min(b, hi);
    return max(a, lo) <= e || a <= min(e, sk - 1);
  }
  __device__ __forceinline__ bool all(int32_t n) const { return n - 1 <= hi && (lo <= 0 || n <= sk); }
  __device__ __forceinline__ Seen from(int32_t p0) const { return Seen{hi - p0, lo - p0, sk - p0}; }
};
__device__ __forceinline__ Seen seen_rows(int32_t pos, int32_t window, int32_t n_sink) {
  return Seen{pos, window > 0 && pos >= window ? pos - window + 1 : 0, n_sink};
}

// Weights are 2^(L - r): L the logit in log2 units, r the row's reference,
// kOffset below the largest L so far, until an L is more than kLazy above that.
// (The largest weight is then 2^kOffset, which f16 holds exactly: rows that one
// weight dominates are half as far off as with a whole number for r.)
//
// While r is up to kFine, L - r is one fused multiply-add of a product of q and
// k with its scale; an L rounded by itself is off by less than 2^-3 there.  Past
// that a fused product differs from the rounded one by more and more, from 2^27
// on by more than the offset, which is then lost beside L as well: the largest
// exponent could be anything (infinite weights, an endless search for the
// maximum).  So past kFine every L is rounded first, which makes L - r exact
// for what counts, and past kExact, where r cannot hold the offset, it goes
// without (a logit's own error is 1 there, and a weight below 2^-25 nothing).
constexpr float kLazy = 5.f;
constexpr float kOffset = 10.f;
constexpr float kFine = 1 << 20, kExact = 1 << 24;
__device__ __forceinline__ float reference(float largest) {       // -inf: no row yet
  return fabsf(largest) <= kExact ? largest - kOffset : largest;
}
__device__ __forceinline__ bool past_fine(float r) { return fabsf(r) > kFine && r != -INFINITY; }
__device__ __forceinline__ float exponent(float s, float scale, float r) {
  return past_fine(r) ? __fsub_rn(__fmul_rn(s, scale), r) : fmaf(s, scale, -r);
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
// Eight codes to four f16 pairs, in order.  The bytes are taken apart by name
// (mov.b32), which the conversion reads in place: 81 values per clock and SM
// with the multiply by the scale, against 43 with shifts and masks.
__device__ __forceinline__ void e2m1x8_to_f16(uint32_t w, uint32_t (&o)[4]) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "mov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(o[0]), "=r"(o[1]), "=r"(o[2]), "=r"(o[3])
      : "r"(w));
}
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t two) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)two));
  return r;
}
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// The page of row p in a plane (0 where it is contiguous, -1 past the table).
__device__ __forceinline__ int32_t page_of(const RowMap& m, int32_t shift, int32_t p) {
  return shift >= 0 ? p >> shift : p / m.page_rows;
}
__device__ __forceinline__ int32_t load_page(const RowMap& m, int32_t shift, int32_t seq, int32_t p) {
  if (!m.page_table) return 0;
  const int32_t pg = page_of(m, shift, p);
  return seq < 0 || pg >= m.max_pages ? -1 : __ldg(m.page_table + (int64_t)seq * m.max_pages + pg);
}
// Physical row of position p, a multiple of kPageStep; `have` falls to the
// number of rows of its step that the plane holds for the sequence (a page may
// be missing, a last page or the last sequence's share cut short).
__device__ __forceinline__ int64_t step_rows(const RowMap& m, int32_t shift, int32_t seq, int32_t p, int32_t page,
                                             int32_t& have) {
  int64_t r, room;
  if (m.page_table) {
    r = (int64_t)page * m.page_rows + (p - page_of(m, shift, p) * m.page_rows);
    room = page < 0 ? 0 : m.n_rows - r;
  } else {
    r = (int64_t)seq * m.seq_rows + p;
    room = seq < 0 ? 0 : m.n_rows - r;
    if (m.seq_rows > 0) room = min(room, m.seq_rows - p);
  }
  have = room >= have ? have : room > 0 ? (int32_t)room : 0;
  return r;
}

// a / b of two counts, most of which fit 32 bits (a 64-bit division is long).
__device__ __forceinline__ int64_t div_run(int64_t a, int64_t b) {
  return (a | b) >> 32 ? a / b : (int64_t)((uint32_t)a / (uint32_t)b);
}

// Joins the parts that CTAs left (gqa_attn.cu), of at most `items` items;
// launched behind either kernel.
cudaError_t launch_gqa_combine(const GqaArgs& a, int32_t D, int32_t run_heads, int64_t items, cudaStream_t st);
// The queries of a CTA: blockIdx.x, n_cta queries on, ...  Thread i looks at
// the i-th: reports a position past every row and says whether one sees none.
// (Read where the kernel starts; the answers meet at a barrier it has anyway.)
template <int N>
__device__ __forceinline__ bool looks_empty(const GqaArgs& a) {
  bool empty = false;
#pragma unroll 1
  for (int32_t q = blockIdx.x + a.n_cta * threadIdx.x; q < a.nq; q += a.n_cta * N) {
    const int32_t p = __ldg(a.query_pos + q);
    if (p >= a.limit) record_error(a.status, CSA2_ERR_INDEX_RANGE);
    empty = empty || p < 0;
  }
  return empty;
}
// The outputs of those that see no row, by all N threads.
template <int N>
__device__ __forceinline__ void write_empties(const GqaArgs& a, int32_t D) {
  const int64_t Hq = (int64_t)a.Hkv * a.G;
  for (int64_t q = blockIdx.x; q < a.nq; q += a.n_cta) {
    if (__ldg(a.query_pos + q) >= 0) continue;
    for (int64_t i = threadIdx.x; i < Hq * D / 8; i += N)
      reinterpret_cast<uint4*>(a.out + q * Hq * D)[i] = make_uint4(0, 0, 0, 0);
    if (a.lse)
      for (int64_t i = threadIdx.x; i < Hq; i += N) a.lse[q * Hq + i] = -INFINITY;
  }
}
// Blocks of queries on the tensor cores (gqa_block.cu): the fields of a that
// describe the work, the CTAs at most and the rows of a part; the launch.
constexpr int kBlockRows = 256;    // query rows of an item: two MMA heights
void gqa_block_shape(GqaArgs& a);
cudaError_t launch_gqa_block(GqaArgs& a, int32_t D, cudaStream_t st);

}  // namespace csa2
