// Grouped-query attention over the FP4 cache, a few query heads per KV head:
//   o = sum_j p_j v_j / sum_j p_j,  p_j = exp(scale q.k_j - m)
// over the rows j that the query sees (all up to its own position, or a
// window and the first rows), in one pass with a running maximum m.
//
// Bound by HBM: a row is D (1/2 + 1/32) bytes each of K and V per KV head,
// read once for all the query heads that share it.  A warp owns one KV head
// (up to 8 NT of its query heads) and walks 16-row tiles:
//   S^T [16 rows][heads] = K Q^T,   O^T [D][heads] += V^T P^T
// on m16n8k16 MMAs whose M side is the cache, so 8 heads fill an MMA and no
// row of it is padding.  Codes go from global memory to the MMA operand in
// registers: the contraction order is free, so lane t of a row's quad owns a
// contiguous quarter of the head dimension (one 16-byte load, one scale), and
// of V^T lane g owns a contiguous eighth of it in four rows, two of which are
// interleaved nibble by nibble so that one E2M1 conversion makes the operand
// pair.  code x scale is exact in f16 (at most 6 significant bits, 2^-10 to
// 2688).  A query row is scaled by a power of two into f16, which keeps all
// of bf16's 8 bits for values down to 2^-28 of the row's largest.
//
// The maximum is lazy: m moves only when a logit exceeds it by 5 (log2), and
// weights are 2^(s - m + 10) <= 2^15.  A row's largest is then at least 2^10,
// so in f16 a weight keeps 11 bits down to 2^-24 of the largest and vanishes
// only below 2^-35: a million rows of small weights beside one large sink
// still count.  Sums are fp32 of the unrounded weights.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "fp4_device.cuh"
#include "gqa_attn.cuh"

namespace csa2 {

namespace {

constexpr int kGqaThreads = 256;
constexpr int kGqaWarps = kGqaThreads / 32;
constexpr float kLazy = 5.f;          // how far a logit may exceed the maximum in use (log2)
constexpr float kOffset = 10.f;       // weights are 2^(s - m + kOffset)

__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Transposes an 8 x 8 matrix of 16-bit values held as two per lane.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
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

// A warp's ring of tiles in shared memory.  A tile is 16 rows of one KV head:
// K codes as they are (a lane reads its quarter row), V codes with rows 0, 2, 4,
// 6 next to one another, then 1, 3, 5, 7 and so on (the rows a quad reads at
// once fill the banks; at D = 128 every other pair of rows has its halves
// swapped for the same end), and four bytes of scales per row.
constexpr int kStages = 4;
template <int D>
struct GqaRing {
  static constexpr int kRow = D / 2;
  static constexpr int k = 0, v = 16 * kRow, sc = 32 * kRow;
  static constexpr int stage = 32 * kRow + 128;
  static constexpr int warp = kStages * stage;
};
template <int D>
__device__ __forceinline__ int v_at(int row, int byte) {       // of a byte of V row `row` in its tile
  const int slot = ((row >> 1) & 3) + 4 * ((row & 1) + 2 * (row >> 3));
  return slot * (D / 2) + (D == 128 ? byte ^ (((slot >> 1) & 1) << 5) : byte);
}

// Copies 16 bytes to shared memory, or zeroes them.
__device__ __forceinline__ void copy16(uint32_t dst, const uint8_t* src, bool take) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(take ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// The page of unit u in a plane (0 where it is contiguous, -1 past the table).
__device__ __forceinline__ int32_t page_of(const RowMap& m, int32_t shift, int32_t u) {
  return shift >= 0 ? u >> shift : u / (m.page_rows / kUnit);
}
__device__ __forceinline__ int32_t unit_page(const RowMap& m, int32_t shift, int32_t seq, int32_t u) {
  if (!m.page_table) return 0;
  const int32_t pg = page_of(m, shift, u);
  return seq < 0 || pg >= m.max_pages ? -1 : __ldg(m.page_table + (int64_t)seq * m.max_pages + pg);
}
// First physical row of unit u, whose rows up to `last` (a position) are
// wanted; -1 when they are not all in the plane.
__device__ __forceinline__ int64_t unit_base(const RowMap& m, int32_t shift, int32_t seq, int32_t u, int32_t page,
                                             int32_t last) {
  const int32_t n = min(kUnit - 1, last - u * kUnit);
  int64_t r;
  if (m.page_table) {
    r = page < 0 ? -1 : (int64_t)page * m.page_rows + (u * kUnit - page_of(m, shift, u) * m.page_rows);
  } else {
    r = seq < 0 || (m.seq_rows > 0 && u * kUnit + n >= m.seq_rows) ? -1 : (int64_t)seq * m.seq_rows + (int64_t)u * kUnit;
  }
  return r >= 0 && r + n < m.n_rows ? r : -1;
}

// Where a lane's parts of the tiles come from: it copies 16 bytes of one or
// two rows of K and of V, and loads one row's scales (K in lanes 0 to 15, V
// above).  Pages are looked up a unit ahead.
template <int D>
struct GqaSource {
  static constexpr int kPer = D / 32;             // lanes per row
  const GqaArgs& a;
  int32_t seq, pos, head, lane;
  int32_t unit = -1, ahead = -1;                  // whose rows k, v, s are; whose pages are loaded
  int32_t page[3];
  const uint8_t *k, *v, *s;                       // this lane's parts of row 0 of the unit
  uint32_t srb;                                   // row stride of its scale plane
  bool ok = false;
  __device__ __forceinline__ GqaSource(const GqaArgs& args, int32_t sq, int32_t p, int32_t h, int l)
      : a(args), seq(sq), pos(p), head(h), lane(l), srb((uint32_t)args.rb[s_plane()]) {}
  __device__ __forceinline__ int s_plane() const { return lane < 16 ? 1 : 3; }
  __device__ __forceinline__ void look_up(int32_t u) {
    ahead = u;
    page[0] = unit_page(a.map[0], a.page_shift[0], seq, u);
    if (!a.one_map) {
      page[1] = unit_page(a.map[2], a.page_shift[2], seq, u);
      page[2] = unit_page(a.map[s_plane()], a.page_shift[s_plane()], seq, u);
    }
  }
  // Moves to unit u; `then` (or -1) is the one after it.
  __device__ __forceinline__ void go(int32_t u, int32_t then) {
    if (ahead != u) look_up(u);
    unit = u;
    const int64_t rk = unit_base(a.map[0], a.page_shift[0], seq, u, page[0], pos);
    const int64_t rv = a.one_map ? rk : unit_base(a.map[2], a.page_shift[2], seq, u, page[1], pos);
    const int64_t rs = a.one_map ? rk : unit_base(a.map[s_plane()], a.page_shift[s_plane()], seq, u, page[2], pos);
    ok = !__any_sync(0xffffffffu, rk < 0 || rv < 0 || rs < 0);
    if (!ok && lane == 0) record_error(a.status, CSA2_ERR_INDEX_RANGE);
    const int row = lane / kPer, byte = (lane % kPer) * 16;
    k = a.base[0] + (rk + row) * a.rb[0] + head * (D / 2) + byte;
    v = a.base[2] + (rv + row) * a.rb[2] + head * (D / 2) + byte;
    const int sp = s_plane();
    s = a.base[sp] + (rs + (lane & 15)) * a.rb[sp] + head * (D / 32);
    if (then >= 0) look_up(then);
  }
  // Starts the copies of tile i of the unit into `stage`; returns its scales.
  __device__ __forceinline__ uint32_t copy(int i, uint32_t stage) const {
    const int p0 = unit * kUnit + 16 * i, row = lane / kPer, byte = (lane % kPer) * 16;
    const bool full = sees_all(p0);
#pragma unroll
    for (int x = 0; x < 16; x += 32 / kPer) {
      const bool take = full || sees(p0 + row + x, pos, a.window, a.n_sink);
      const uint32_t at = 16 * i + x;
      copy16(stage + GqaRing<D>::k + (row + x) * (D / 2) + byte, k + (uint64_t)at * (uint32_t)a.rb[0], take);
      copy16(stage + GqaRing<D>::v + v_at<D>(row + x, byte), v + (uint64_t)at * (uint32_t)a.rb[2], take);
    }
    if (!full && !sees(p0 + (lane & 15), pos, a.window, a.n_sink)) return 0;
    const uint8_t* p = s + (uint64_t)(uint32_t)(16 * i) * srb;
    return D == 128 ? __ldg(reinterpret_cast<const uint32_t*>(p)) : (uint32_t)__ldg(reinterpret_cast<const uint16_t*>(p));
  }
  __device__ __forceinline__ bool sees_all(int32_t p0) const {
    return p0 + 15 <= pos && (a.window <= 0 || p0 > pos - a.window || p0 + 15 < a.n_sink);
  }
};

__device__ __forceinline__ uint32_t lds32(uint32_t at) {
  uint32_t r;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(r) : "r"(at));
  return r;
}
__device__ __forceinline__ uint32_t lds8(uint32_t at) {
  uint32_t r;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(r) : "r"(at));
  return r;
}
template <int N>
__device__ __forceinline__ void lds_words(uint32_t at, uint32_t (&w)[N]) {
  if constexpr (N == 4)
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(at));
  else if constexpr (N == 2)
    asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(at));
  else
    w[0] = lds32(at);
}

// Running state of a warp: NT runs of 8 heads.  A lane holds heads 2t and
// 2t + 1 of each run.
template <int D, int NT>
struct GqaState {
  float o[NT][D / 16][4];     // O^T: dims g D/8 + 2j (+ 1), heads 2t and 2t + 1
  float mo[NT][2];            // maximum in use minus kOffset, log2 units (-inf: no row yet)
  float l[NT][2];             // this lane's part of the sum of weights
};

// One tile: S^T = K Q^T, the weights, O^T += V^T P^T.  `full`: every row is seen.
template <int D, int NT>
__device__ __forceinline__ void tile_step(const GqaArgs& a, GqaState<D, NT>& st, uint32_t stage,
                                          const uint32_t (&qf)[NT][D / 16][2], const float (&qs)[NT][2], bool full,
                                          int32_t p0, int32_t pos, int g, int t) {
  using R = GqaRing<D>;
  float s[NT][4];
#pragma unroll
  for (int n = 0; n < NT; ++n) s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.f;
  {
    uint32_t k0[D / 32], k1[D / 32];
    lds_words(stage + R::k + g * R::kRow + t * (D / 8), k0);
    lds_words(stage + R::k + (g + 8) * R::kRow + t * (D / 8), k1);
    const uint32_t sk0 = e4m3x2_to_f16x2(lds8(stage + R::sc + g * 4 + t * (D / 4) / 32) * 0x101u);
    const uint32_t sk1 = e4m3x2_to_f16x2(lds8(stage + R::sc + (g + 8) * 4 + t * (D / 4) / 32) * 0x101u);
#pragma unroll
    for (int w = 0; w < D / 32; ++w) {
      uint32_t x0[4], x1[4];
      e2m1x8_to_f16(k0[w], x0);
      e2m1x8_to_f16(k1[w], x1);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t af[4] = {mul_f16x2(x0[2 * h], sk0), mul_f16x2(x1[2 * h], sk1), mul_f16x2(x0[2 * h + 1], sk0),
                                mul_f16x2(x1[2 * h + 1], sk1)};
#pragma unroll
        for (int n = 0; n < NT; ++n) mma_f16(s[n], af, qf[n][2 * w + h][0], qf[n][2 * w + h][1]);
      }
    }
  }
  // x = the logit above the maximum in use, plus kOffset
  const bool see0 = full || sees(p0 + g, pos, a.window, a.n_sink);
  const bool see1 = full || sees(p0 + g + 8, pos, a.window, a.n_sink);
  float x[NT][4];
  bool more = false;
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[n][i] = (i < 2 ? see0 : see1) ? fmaf(s[n][i], qs[n][i & 1], -st.mo[n][i & 1]) : -INFINITY;
      more |= x[n][i] > kOffset + kLazy;
    }
  if (__any_sync(0xffffffffu, more)) {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float f[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float m = fmaxf(see0 ? s[n][e] * qs[n][e] : -INFINITY, see1 ? s[n][2 + e] * qs[n][e] : -INFINITY);
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        const float mo = fmaxf(st.mo[n][e], m - kOffset);
        f[e] = st.mo[n][e] == -INFINITY ? 0.f : ex2(st.mo[n][e] - mo);
        st.mo[n][e] = mo;
        st.l[n][e] *= f[e];
        x[n][e] = see0 ? fmaf(s[n][e], qs[n][e], -mo) : -INFINITY;
        x[n][2 + e] = see1 ? fmaf(s[n][2 + e], qs[n][e], -mo) : -INFINITY;
      }
#pragma unroll
      for (int j = 0; j < D / 16; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) st.o[n][j][i] *= f[i & 1];
    }
  }
  uint32_t pf[NT][2];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    float p[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = ex2(x[n][i]);
    st.l[n][0] += p[0] + p[2];
    st.l[n][1] += p[1] + p[3];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const __half2 h = __floats2half2_rn(p[2 * i], p[2 * i + 1]);
      pf[n][i] = transpose8x8(*reinterpret_cast<const uint32_t*>(&h));
    }
  }
  uint32_t v[4][D / 64], sv[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = 2 * t + (i & 1) + 8 * (i >> 1);
    lds_words(stage + R::v + v_at<D>(row, g * (D / 16)), v[i]);
    sv[i] = lds8(stage + R::sc + 64 + row * 4 + g * (D / 8) / 32);
  }
  const uint32_t sv0 = e4m3x2_to_f16x2(sv[0] | sv[1] << 8), sv1 = e4m3x2_to_f16x2(sv[2] | sv[3] << 8);
#pragma unroll
  for (int w = 0; w < D / 64; ++w) {
    constexpr uint32_t kLow = 0x0F0F0F0Fu;
    const uint32_t lo01 = (v[0][w] & kLow) | ((v[1][w] << 4) & ~kLow), hi01 = ((v[0][w] >> 4) & kLow) | (v[1][w] & ~kLow);
    const uint32_t lo23 = (v[2][w] & kLow) | ((v[3][w] << 4) & ~kLow), hi23 = ((v[2][w] >> 4) & kLow) | (v[3][w] & ~kLow);
    uint32_t x0[4], x1[4], x2[4], x3[4];
    e2m1x8_to_f16(lo01, x0);
    e2m1x8_to_f16(hi01, x1);
    e2m1x8_to_f16(lo23, x2);
    e2m1x8_to_f16(hi23, x3);
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      const uint32_t af[4] = {mul_f16x2(x0[b], sv0), mul_f16x2(x1[b], sv0), mul_f16x2(x2[b], sv1), mul_f16x2(x3[b], sv1)};
#pragma unroll
      for (int n = 0; n < NT; ++n) mma_f16(st.o[n][4 * w + b], af, pf[n][0], pf[n][1]);
    }
  }
}

// The query heads of a run as MMA operands, and their logit scales (log2
// units) for the heads a lane holds.  Head n 8 + g, dims t D/4 + 4k + {0..3}.
template <int D, int NT>
__device__ __forceinline__ void load_query(const GqaArgs& a, const uint16_t* q, int heads, int g, int t,
                                           uint32_t (&qf)[NT][D / 16][2], float (&qs)[NT][2]) {
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int h = n * 8 + g;
    uint32_t w[D / 8];
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      const uint4 u = h < heads ? __ldg(reinterpret_cast<const uint4*>(q + (int64_t)h * D + t * (D / 4)) + i)
                                : make_uint4(0, 0, 0, 0);
      w[4 * i] = u.x, w[4 * i + 1] = u.y, w[4 * i + 2] = u.z, w[4 * i + 3] = u.w;
    }
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < D / 8; ++i) top = max(top, max(w[i] & 0x7FFFu, (w[i] >> 16) & 0x7FFFu));
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
    // the largest magnitude into [2^14, 2^15); rows below 2^-107 are scaled as that
    const int e = max((int)(top >> 7), 20);
    const float up = __uint_as_float((uint32_t)(268 - e) << 23);             // 2^(141 - e)
    float down = __uint_as_float((uint32_t)max(e - 14, 1) << 23) * a.scale_log2;   // 2^(e - 141)
#pragma unroll
    for (int i = 0; i < D / 8; ++i) {
      const __half2 hh = __floats2half2_rn(__uint_as_float(w[i] << 16) * up, __uint_as_float(w[i] & 0xFFFF0000u) * up);
      qf[n][i / 2][i & 1] = *reinterpret_cast<const uint32_t*>(&hh);
    }
#pragma unroll
    for (int x = 0; x < 2; ++x) qs[n][x] = __shfl_sync(0xffffffffu, down, (2 * t + x) * 4);
  }
}

// Sum over the block of one value per thread, and the sum of the threads
// before this one.
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t* sh, int64_t* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t s = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t n = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += n;
  }
  if (lane == 31) sh[warp] = s;
  __syncthreads();
  int64_t before = 0, all = 0;
#pragma unroll
  for (int i = 0; i < kGqaWarps; ++i) {
    if (i < warp) before += sh[i];
    all += sh[i];
  }
  *total = all;
  return before + s - v;
}

template <int D>
__device__ __forceinline__ void store_bf16(uint16_t* dst, const float* v, float w) {   // D/8 values
#pragma unroll
  for (int i = 0; i < D / 64; ++i) {
    uint32_t p[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(v[8 * i + 2 * j] * w, v[8 * i + 2 * j + 1] * w);
      p[j] = *reinterpret_cast<const uint32_t*>(&b);
    }
    reinterpret_cast<uint4*>(dst)[i] = make_uint4(p[0], p[1], p[2], p[3]);
  }
}

template <int D, int NT>
__global__ void __launch_bounds__(kGqaThreads, NT == 1 ? 2 : 1) gqa_split_kernel(const __grid_constant__ GqaArgs a) {
  extern __shared__ __align__(128) uint8_t gqa_s[];    // the warps' rings; then [warps][8 NT][D + 2] floats to join
  __shared__ int64_t scan_s[kGqaWarps];
  __shared__ int32_t item_s;
  __shared__ int64_t item_start_s;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  pdl_trigger();

  // ---- where this CTA's run of units starts
  int64_t total;
  {
    const int per = (a.nq + kGqaThreads - 1) / kGqaThreads;
    const int i0 = min(tid * per, a.nq), i1 = min(i0 + per, a.nq);
    int64_t n = 0;
    for (int i = i0; i < i1; ++i) n += unit_range(__ldg(a.query_pos + i), a.window, a.n_sink).count;
    int64_t start = block_scan(n, scan_s, &total);
    const int64_t all = total * a.groups, run = (all + a.n_cta - 1) / a.n_cta;
    const int64_t u = (int64_t)blockIdx.x * run;
    if (blockIdx.x == 0 || (start * a.groups <= u && u < (start + n) * a.groups)) {
      for (int i = i0; i < i1; ++i) {
        const int64_t c = unit_range(__ldg(a.query_pos + i), a.window, a.n_sink).count;
        if (blockIdx.x == 0) a.starts[i] = start;
        if (start * a.groups <= u && u < (start + c) * a.groups) {
          item_s = i;
          item_start_s = start;
        }
        start += c;
      }
    }
    if (blockIdx.x == 0 && tid == 0) a.starts[a.nq] = total;
    __syncthreads();
    if (u >= all) return;
  }
  const int64_t all = total * a.groups, run = (all + a.n_cta - 1) / a.n_cta;
  const int64_t u_begin = (int64_t)blockIdx.x * run, u_end = min(u_begin + run, all);
  const int Hq = a.Hkv * a.G;

  int qi = item_s;
  int64_t q_start = item_start_s * a.groups;       // first unit of the query, over its groups
  for (int64_t u = u_begin; u < u_end;) {
    const int32_t pos = __ldg(a.query_pos + qi);
    const UnitRange ur = unit_range(pos, a.window, a.n_sink);
    if (u >= q_start + (int64_t)ur.count * a.groups) {     // on to the next query (or past empty ones)
      q_start += (int64_t)ur.count * a.groups;
      ++qi;
      continue;
    }
    const int grp = (int)((u - q_start) / ur.count);
    const int64_t i_start = q_start + (int64_t)grp * ur.count, i_end = i_start + ur.count;
    const int32_t c0 = (int32_t)(u - i_start), c1 = (int32_t)(min(u_end, i_end) - i_start);
    const int32_t seq = a.seq_of_query ? __ldg(a.seq_of_query + qi) : qi;

    // ---- this warp's head and tiles
    const int vh0 = grp * a.per_cta, n_vh = min(a.per_cta, a.vh - vh0);
    const int share = kGqaWarps / n_vh;            // warps per virtual head
    const int vh = vh0 + warp / share, sub = warp % share;
    const bool busy = warp < n_vh * share;
    const int head = vh / a.subs, r0 = (vh % a.subs) * 8 * NT;
    const int heads = min(8 * NT, a.G - r0);
    GqaState<D, NT> st;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      st.mo[n][0] = st.mo[n][1] = -INFINITY;
      st.l[n][0] = st.l[n][1] = 0.f;
#pragma unroll
      for (int j = 0; j < D / 16; ++j) st.o[n][j][0] = st.o[n][j][1] = st.o[n][j][2] = st.o[n][j][3] = 0.f;
    }
    if (busy) {
      uint32_t qf[NT][D / 16][2];
      float qs[NT][2];
      load_query<D, NT>(a, a.q + ((int64_t)qi * Hq + head * a.G + r0) * D, heads, g, t, qf, qs);
      // tiles c0 * 4 + sub, + share, ... that hold a row to see: kStages - 1 of
      // them in flight while one is worked on
      constexpr int TPU = kUnit / 16;
      const int32_t t1 = c1 == ur.count ? (c1 - 1) * TPU + pos % kUnit / 16 + 1 : c1 * TPU;   // none past pos
      const uint32_t ring = smem_u32(gqa_s) + warp * GqaRing<D>::warp;
      auto unit_of = [&](int32_t x) { return ur.row(x / TPU) / kUnit; };
      auto next = [&](int32_t x) {
        if (a.window > 0) while (x < t1 && !sees_any(ur.row(x / TPU) + (x % TPU) * 16, 16, pos, a.window, a.n_sink)) x += share;
        return x;
      };
      GqaSource<D> src(a, seq, pos, head, lane);
      int32_t load = next(c0 * TPU + sub), work = load;
      uint32_t sc = 0, bad = 0;                    // scales on their way; stages whose rows are not there
      int ls = 0, ws = 0;
      auto start = [&]() {                         // starts the next tile's copies; its stage's scales come back
        if (load < t1) {
          const int32_t u = unit_of(load);
          if (u != src.unit) {
            const int32_t then = (load / TPU + 1) * TPU;
            src.go(u, then < t1 ? unit_of(then) : -1);
          }
          bad = src.ok ? bad & ~(1u << ls) : bad | (1u << ls);
          sc = src.ok ? src.copy(load % TPU, ring + ls * GqaRing<D>::stage) : 0;
          load = next(load + share);
        }
        copies_commit();
      };
      auto put_scales = [&]() {
        asm volatile("st.shared.b32 [%0], %1;" ::"r"(ring + ls * GqaRing<D>::stage + GqaRing<D>::sc + lane * 4), "r"(sc)
                     : "memory");
        ls = ls + 1 == kStages ? 0 : ls + 1;
      };
#pragma unroll
      for (int i = 0; i < kStages - 2; ++i) start(), put_scales();
      start();
      while (work < t1) {
        copies_wait<kStages - 2>();
        __syncwarp();                              // the tile is there, and its predecessor's stage is free
        put_scales();
        start();
        const int32_t p0 = ur.row(work / TPU) + (work % TPU) * 16;
        if (!((bad >> ws) & 1u))
          tile_step<D, NT>(a, st, ring + ws * GqaRing<D>::stage, qf, qs, src.sees_all(p0), p0, pos, g, t);
        ws = ws + 1 == kStages ? 0 : ws + 1;
        work = next(work + share);
      }
      copies_wait<0>();
      __syncwarp();
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) st.l[n][e] += __shfl_xor_sync(0xffffffffu, st.l[n][e], o);
    }
    // ---- warps of the same head join
    if (share > 1) {
      constexpr int W = D + 2;                     // O, maximum, sum
      float* merge_s = reinterpret_cast<float*>(gqa_s);
      __syncthreads();                             // the rings are done with
      if (busy && sub > 0) {
        float* m = merge_s + (size_t)warp * 8 * NT * W;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float* hm = m + (n * 8 + 2 * t + e) * W;
            if (g == 0) hm[D] = st.mo[n][e], hm[D + 1] = st.l[n][e];
#pragma unroll
            for (int j = 0; j < D / 16; ++j) {
              hm[g * (D / 8) + 2 * j] = st.o[n][j][e];
              hm[g * (D / 8) + 2 * j + 1] = st.o[n][j][2 + e];
            }
          }
      }
      __syncthreads();
      if (busy && sub == 0) {
        for (int w = 1; w < share; ++w) {
          const float* m = merge_s + (size_t)(warp + w) * 8 * NT * W;
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float* hm = m + (n * 8 + 2 * t + e) * W;
              const float mo = fmaxf(st.mo[n][e], hm[D]);
              const float f0 = st.mo[n][e] == -INFINITY ? (st.l[n][e] != st.l[n][e] ? st.l[n][e] : 0.f) : ex2(st.mo[n][e] - mo);
              const float f1 = hm[D] == -INFINITY ? (hm[D + 1] != hm[D + 1] ? hm[D + 1] : 0.f) : ex2(hm[D] - mo);
              st.mo[n][e] = mo;
              st.l[n][e] = st.l[n][e] * f0 + hm[D + 1] * f1;
#pragma unroll
              for (int j = 0; j < D / 16; ++j) {
                st.o[n][j][e] = st.o[n][j][e] * f0 + hm[g * (D / 8) + 2 * j] * f1;
                st.o[n][j][2 + e] = st.o[n][j][2 + e] * f0 + hm[g * (D / 8) + 2 * j + 1] * f1;
              }
            }
        }
      }
      __syncthreads();
    }
    // ---- the whole item: its output; else this CTA's part of it
    if (busy && sub == 0) {
      const bool before = i_start < u_begin, after = i_end > u_end;
      const int rows = a.per_cta * 8 * NT;
      const int64_t slot = 2 * (int64_t)blockIdx.x + (before ? 0 : 1);
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int r = n * 8 + 2 * t + e;
          if (r >= heads) continue;
          float v[D / 8];
#pragma unroll
          for (int j = 0; j < D / 16; ++j) v[2 * j] = st.o[n][j][e], v[2 * j + 1] = st.o[n][j][2 + e];
          if (!before && !after) {
            const int64_t at = (int64_t)qi * Hq + head * a.G + r0 + r;
            store_bf16<D>(a.out + at * D + g * (D / 8), v, st.l[n][e] == 0.f ? 0.f : 1.f / st.l[n][e]);
            if (a.lse && g == 0)
              a.lse[at] = st.l[n][e] == 0.f ? -INFINITY : (st.mo[n][e] + log2f(st.l[n][e])) * 0.69314718055994531f;
          } else {
            const int64_t at = slot * rows + (vh - vh0) * 8 * NT + r;
#pragma unroll
            for (int j = 0; j < D / 32; ++j)
              reinterpret_cast<float4*>(a.part_o + at * D + g * (D / 8))[j] =
                  make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
            if (g == 0) a.part_ml[at] = make_float2(st.mo[n][e], st.l[n][e]);
          }
        }
    }
    u = i_start + c1;
  }
}

// Joins the parts of every item that several CTAs share, and writes the
// outputs of queries that see no row.  One block per (query, virtual head).
constexpr int kCombThreads = 128;
constexpr int kCombWarps = kCombThreads / 32;
template <int D>
__global__ void __launch_bounds__(kCombThreads) gqa_combine_kernel(const __grid_constant__ GqaArgs a, int32_t run_heads) {
  __shared__ float acc_s[kCombWarps][D];
  __shared__ float m_s[kCombWarps], l_s[kCombWarps];
  const int r = blockIdx.x, qi = blockIdx.y;           // query head, query
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int32_t pos = __ldg(a.query_pos + qi);
  const int32_t count = unit_range(pos, a.window, a.n_sink).count;
  const int64_t at = (int64_t)qi * (a.Hkv * a.G) + r;
  pdl_wait();
  if (count == 0) {
    for (int i = threadIdx.x; i < D / 2; i += kCombThreads) reinterpret_cast<uint32_t*>(a.out + at * D)[i] = 0u;
    if (threadIdx.x == 0 && a.lse) a.lse[at] = -INFINITY;
    return;
  }
  const int vh = (r / a.G) * a.subs + (r % a.G) / run_heads, grp = vh / a.per_cta;
  const int64_t all = __ldcg(a.starts + a.nq) * a.groups, run = (all + a.n_cta - 1) / a.n_cta;
  const int64_t i0 = __ldcg(a.starts + qi) * a.groups + (int64_t)grp * count, i1 = i0 + count;
  const int64_t first = i0 / run, last = (i1 - 1) / run;
  if (first == last) return;                           // one CTA had the whole item
  const int rows = a.per_cta * run_heads, row = (vh - grp * a.per_cta) * run_heads + (r % a.G) % run_heads;
  auto part = [&](int64_t c) { return (2 * c + (c == first ? 1 : 0)) * rows + row; };
  float M = -INFINITY;
  for (int64_t c = first + threadIdx.x; c <= last; c += kCombThreads) M = fmaxf(M, __ldcg(&a.part_ml[part(c)]).x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  if (lane == 0) m_s[warp] = M;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kCombWarps; ++w) M = fmaxf(M, m_s[w]);
  constexpr int V = D / 32;                            // values per lane
  float acc[V], l = 0.f;
#pragma unroll
  for (int i = 0; i < V; ++i) acc[i] = 0.f;
#pragma unroll 4
  for (int64_t c = first + warp; c <= last; c += kCombWarps) {
    const int64_t p = part(c);
    const float2 ml = __ldcg(&a.part_ml[p]);
    const float f = ml.x == -INFINITY ? (ml.y != ml.y ? ml.y : 0.f) : ex2(ml.x - M);
    const float* o = a.part_o + p * D + lane * V;
    l += f * ml.y;
    if constexpr (V == 4) {
      const float4 v = __ldcg(reinterpret_cast<const float4*>(o));
      acc[0] += f * v.x, acc[1] += f * v.y, acc[2] += f * v.z, acc[3] += f * v.w;
    } else {
      const float2 v = __ldcg(reinterpret_cast<const float2*>(o));
      acc[0] += f * v.x, acc[1] += f * v.y;
    }
  }
#pragma unroll
  for (int i = 0; i < V; ++i) acc_s[warp][lane * V + i] = acc[i];
  if (lane == 0) l_s[warp] = l;
  __syncthreads();
  l = 0.f;
#pragma unroll
  for (int w = 0; w < kCombWarps; ++w) l += l_s[w];
  const float inv = l == 0.f ? 0.f : 1.f / l;
  for (int i = threadIdx.x; i < D; i += kCombThreads) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kCombWarps; ++w) v += acc_s[w][i];
    reinterpret_cast<__nv_bfloat16*>(a.out)[at * D + i] = __float2bfloat16_rn(v * inv);
  }
  if (threadIdx.x == 0 && a.lse) a.lse[at] = l == 0.f ? -INFINITY : (M + log2f(l)) * 0.69314718055994531f;
}

constexpr int kMaxCtas = 2 * 160;      // main-kernel CTAs at most: the workspace is sized without a device

template <int D, int NT>
cudaError_t launch_gqa_t(GqaArgs& a, cudaStream_t st) {
  static SetupMask done{0};
  constexpr size_t rings = (size_t)kGqaWarps * GqaRing<D>::warp, join = (size_t)kGqaWarps * 8 * NT * (D + 2) * 4;
  constexpr size_t smem = rings > join ? rings : join;
  cudaError_t e = ensure_smem(gqa_split_kernel<D, NT>, (int)smem, done);
  if (e != cudaSuccess) return e;
  a.n_cta = sm_count() * (NT == 1 ? 2 : 1);
  if (a.n_cta > kMaxCtas) a.n_cta = kMaxCtas;
  gqa_split_kernel<D, NT><<<a.n_cta, kGqaThreads, smem, st>>>(a);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch_k(gqa_combine_kernel<D>, dim3(a.Hkv * a.G, a.nq), dim3(kCombThreads), 0, st, false, true, a,
                  (int32_t)(8 * NT));
}

// How query heads map to warps: runs of 8 NT heads of a KV head, up to 8 runs per CTA.
void gqa_heads(GqaArgs& a, int32_t Hkv, int32_t G, int* nt) {
  *nt = G <= 8 ? 1 : 2;
  a.Hkv = Hkv;
  a.G = G;
  a.subs = (G + 8 * *nt - 1) / (8 * *nt);
  a.vh = Hkv * a.subs;
  a.groups = (a.vh + kGqaWarps - 1) / kGqaWarps;
  a.per_cta = (a.vh + a.groups - 1) / a.groups;
}

void carve_gqa(GqaArgs& a, Carver& c, int32_t nq, int32_t D, int nt) {
  const size_t parts = 2 * (size_t)kMaxCtas * a.per_cta * 8 * nt;
  a.starts = c.take<int64_t>((size_t)nq + 1);
  a.part_o = c.take<float>(parts * D);
  a.part_ml = c.take<float2>(parts);
}

}  // namespace

size_t gqa_scratch_bytes(int32_t nq, int32_t Hq, int32_t Hkv, int32_t D) {
  GqaArgs a{};
  int nt;
  gqa_heads(a, Hkv, Hq / Hkv, &nt);
  Carver c(nullptr);
  carve_gqa(a, c, nq, D, nt);
  return c.used + 256;
}

cudaError_t launch_gqa_attn(const uint16_t* q, const csa2_kv_cache& kv, const int32_t* seq_of_query,
                            const int32_t* query_pos, int32_t nq, int32_t Hq, int32_t window, int32_t n_sink,
                            float scale, bool group_queries, uint16_t* out, float* lse, void* ws, int32_t* status,
                            cudaStream_t st) {
  (void)group_queries;
  GqaArgs a{};
  int nt;
  gqa_heads(a, kv.Hkv, Hq / kv.Hkv, &nt);
  Carver c(ws);
  carve_gqa(a, c, nq, kv.D, nt);
  a.q = q, a.out = out, a.lse = lse;
  const csa2_rows* views[4] = {&kv.k_codes, &kv.k_scales, &kv.v_codes, &kv.v_scales};
  a.one_map = 1;
  for (int i = 0; i < 4; ++i) {
    a.base[i] = static_cast<const uint8_t*>(views[i]->base);
    a.rb[i] = views[i]->row_bytes;
    a.map[i] = to_rowmap(*views[i]);
    if (!same_rows(*views[0], *views[i])) a.one_map = 0;
    const int32_t units = views[i]->page_table ? views[i]->page_rows / kUnit : 1;
    a.page_shift[i] = -1;
    for (int b = 0; b < 31; ++b)
      if (units == 1 << b) a.page_shift[i] = b;
  }
  a.seq_of_query = seq_of_query;
  a.query_pos = query_pos;
  a.nq = nq;
  a.window = window;
  a.n_sink = window > 0 ? n_sink : 0;
  a.scale_log2 = scale * 1.4426950408889634f;
  a.status = status;
  if (kv.D == 128) return nt == 1 ? launch_gqa_t<128, 1>(a, st) : launch_gqa_t<128, 2>(a, st);
  return nt == 1 ? launch_gqa_t<64, 1>(a, st) : launch_gqa_t<64, 2>(a, st);
}

}  // namespace csa2
