// Grouped-query attention over the FP4 cache, a few query heads per KV head:
//   o = sum_j p_j v_j / sum_j p_j,  p_j = exp(scale q.k_j - m)
// over the rows j that the query sees (all up to its own position, or a
// window and the first rows), in one pass with a running maximum m.
//
// The least it can do is read the rows: D (1/2 + 1/32) bytes each of K and V
// per KV head, once for all the query heads that share it.  A warp owns one
// KV head (up to 8 NT of its query heads) and walks 32-row tiles:
//   S^T [rows][heads] = K Q^T,   O^T [D][heads] += V^T P^T
// on m16n8k16 MMAs whose M side is the cache, so 8 heads fill an MMA and no
// row of it is padding (tcgen05 would have 8 columns beside 128 rows, and both
// operands through shared memory).  Codes come by 16-byte asynchronous copies
// into a ring of the warp's own, three tiles deep, and go from there to the
// MMA operand in registers: the contraction order is free, so lane t of a
// row's quad owns a contiguous quarter of the head dimension (one scale), and
// of V^T lane g owns a contiguous eighth of it in four rows, two of which are
// interleaved nibble by nibble so that one E2M1 conversion makes the operand
// pair.  code x scale is exact in f16 (at most 6 significant bits, 2^-10 to
// 2688).  A query row is scaled by a power of two into f16, which keeps all
// of bf16's 8 bits for values down to 2^-28 of the row's largest.
//
// Measured on 64 query and 8 KV heads, D = 128: one query over 1,048,576 rows
// 281 to 308 us from GPU to GPU (3.7 to 4.1 TB/s, 0.57 to 0.62 of the copy
// rate), 32 queries over 572,000 rows 167 to 176 us (3.5 to 3.7 TB/s); at D = 64,
// 238 and 140 us.  No unit is full (ALU pipe 55%, issue slots 62%, DRAM 44%,
// tensor pipe 21%): four warps per scheduler wait for their own instructions
// before, for the half-rate pipe of conversions, permutes and f16 products and
// for the issue slot, 1.6, 0.9 and 1.1 warps per issue.  Against
// what stood when each was tried, 16-row tiles took 383 us for 326, V of a
// tile beside K of the next 348 for 322, two chains of MMAs per logit tile 299
// for 292, and 80 registers for a third CTA per SM 429 for 292 (spills).
//
// The maximum is lazy: m moves only when a logit exceeds it by 5 (log2), and
// weights are 2^(s - m + 10) <= 2^15 (logits past 2^20: gqa_attn.cuh).  A row's
// largest is then at least 2^10, so in f16 a weight keeps 11 bits down to 2^-24
// of the largest and vanishes only below 2^-35: a million rows of small weights
// beside one large sink still count.  Sums are fp32 of the unrounded weights.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "fp4_device.cuh"
#include "gqa_attn.cuh"

namespace csa2 {

namespace {

constexpr int kGqaThreads = 256;
constexpr int kMaxCtas = 2 * 160;     // main-kernel CTAs at most: the workspace is sized without a device
constexpr int kGqaWarps = kGqaThreads / 32;
__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Transposes an 8 x 8 matrix of 16-bit values held as two per lane.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
// A warp's ring of tiles in shared memory.  A tile is kRows rows of one KV
// head: K codes as they are (a lane reads its quarter row), V codes of every 16
// rows with rows 0, 2, 4, 6 next to one another, then 1, 3, 5, 7 and so on (the
// rows a quad reads at once fill the banks; at D = 128 every other pair of rows
// has its halves swapped for the same end), and four bytes of scales per row.
constexpr int kRows = 32;
constexpr int kStages = 3;
static_assert(kRows == 32 && kStages == 3, "a lane per row of scales, written a turn before they are read");
// Tiles a CTA takes at least: one each makes as many parts as there are tiles
// to join.  A query over 4,096 rows took 19.1, 16.8, 17.3, 18.8, 21.2 us with
// 1, 2, 3, 4, 6 (13.0 to 13.5 us by now).
constexpr int kMinRun = 2;
template <int D>
struct GqaRing {
  static constexpr int kRow = D / 2;
  static constexpr int k = 0, v = kRows * kRow, ks = 2 * kRows * kRow, vs = ks + 4 * kRows;
  static constexpr int stage = vs + 4 * kRows;
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
__device__ __forceinline__ void copy16(uint32_t dst, const uint8_t* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// Where a lane's parts of the tiles come from: it copies 16 bytes of every
// 32 / kPer-th row of K and of V, and loads the scales of row `lane` of both.
// Pages are looked up a step ahead.
template <int D>
struct GqaSource {
  static constexpr int kPer = D / 32;             // lanes per row
  const GqaArgs& a;
  int32_t seq, head, lane;
  int32_t step = -1, ahead = -1;                  // first row of the step at hand; of the one looked up
  int32_t page[4];
  const uint8_t* at[4];                           // this lane's parts of row 0 of the step
  int32_t have = 0;                               // rows of the step that are there
  __device__ __forceinline__ GqaSource(const GqaArgs& args, int32_t sq, int32_t h, int l)
      : a(args), seq(sq), head(h), lane(l) {}
  __device__ __forceinline__ void look_up(int32_t p) {
    ahead = p;
    page[0] = load_page(a.map[0], a.page_shift[0], seq, p);
    if (!a.one_map)
#pragma unroll
      for (int i = 1; i < 4; ++i) page[i] = load_page(a.map[i], a.page_shift[i], seq, p);
  }
  // Moves to the step at row p, whose rows w sees; `then` (or -1) is the one after it.
  __device__ __forceinline__ void go(int32_t p, const Seen& w, int32_t then) {
    if (ahead != p) look_up(p);
    step = p;
    int64_t r = 0;
    have = kPageStep;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i == 0 || !a.one_map) r = step_rows(a.map[i], a.page_shift[i], seq, p, page[i], have);
      at[i] = a.base[i] + (r + (i & 1 ? lane : lane / kPer)) * a.rb[i] +
              (i & 1 ? head * (D / 32) : head * (D / 2) + (lane % kPer) * 16);
    }
    if (have < kPageStep && lane == 0 && w.some(have, kPageStep - 1)) record_error(a.status, CSA2_ERR_INDEX_RANGE);
    if (then >= 0) look_up(then);
  }
  __device__ __forceinline__ uint32_t scales(int i, uint32_t off) const {
    const uint8_t* p = at[i] + (uint64_t)off * (uint32_t)a.rb[i];
    return D == 128 ? __ldg(reinterpret_cast<const uint32_t*>(p)) : (uint32_t)__ldg(reinterpret_cast<const uint16_t*>(p));
  }
  // Starts the copies of the tile at row `off` of the step, whose rows w
  // sees, into `stage`; ks and vs are the lane's scales.
  __device__ __forceinline__ void copy(uint32_t off, uint32_t stage, const Seen& w, uint32_t& ks, uint32_t& vs) const {
    const int row = lane / kPer, byte = (lane % kPer) * 16;
    const uint8_t* k = at[0] + (uint64_t)off * (uint32_t)a.rb[0];
    const uint8_t* v = at[2] + (uint64_t)off * (uint32_t)a.rb[2];
    const uint32_t kd = stage + GqaRing<D>::k + row * (D / 2) + byte, vd = stage + GqaRing<D>::v + v_at<D>(row, byte);
    constexpr int X = 32 / kPer;                  // 8 or 16 rows on, a tile's image moves by as many rows
    if (w.all(kRows)) {
#pragma unroll
      for (int x = 0; x < kRows; x += X) {
        copy16(kd + x * (D / 2), k + (uint64_t)x * (uint32_t)a.rb[0]);
        copy16(vd + x * (D / 2), v + (uint64_t)x * (uint32_t)a.rb[2]);
      }
      ks = scales(1, off);
      vs = scales(3, off);
      return;
    }
    for (int x = 0; x < kRows; x += X) {
      const bool take = w.row(row + x);
      copy16(kd + x * (D / 2), k + (uint64_t)x * (uint32_t)a.rb[0], take);
      copy16(vd + x * (D / 2), v + (uint64_t)x * (uint32_t)a.rb[2], take);
    }
    ks = vs = 0;
    if (w.row(lane)) {
      ks = scales(1, off);
      vs = scales(3, off);
    }
  }
};

template <int N>
__device__ __forceinline__ void lds_words(const uint8_t* p, uint32_t (&w)[N]) {
  if constexpr (N == 4) {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w;
  } else if constexpr (N == 2) {
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    w[0] = u.x, w[1] = u.y;
  } else {
    w[0] = *reinterpret_cast<const uint32_t*>(p);
  }
}

// Running state of a warp: NT runs of 8 heads.  A lane holds heads 2t and
// 2t + 1 of each run.
template <int D, int NT>
struct GqaState {
  float o[NT][D / 16][4];     // O^T: dims g D/8 + 2j (+ 1), heads 2t and 2t + 1
  float mo[NT][2];            // reference (-inf: no row yet)
  float l[NT][2];             // this lane's part of the sum of weights
};

// One tile: S^T = K Q^T, the weights, O^T += V^T P^T; w: its rows that are seen.
template <int D, int NT>
__device__ __forceinline__ void tile_step(GqaState<D, NT>& st, const uint8_t* stage,
                                          const uint32_t (&qf)[NT][D / 16][2], const float (&qs)[NT][2], const Seen& w,
                                          int g, int t) {
  using R = GqaRing<D>;
  constexpr int H = kRows / 16;                    // MMA heights
  float s[H][NT][4];
#pragma unroll
  for (int h = 0; h < H; ++h) {
#pragma unroll
    for (int n = 0; n < NT; ++n) s[h][n][0] = s[h][n][1] = s[h][n][2] = s[h][n][3] = 0.f;
    const int r0 = 16 * h + g, r1 = r0 + 8;
    uint32_t k0[D / 32], k1[D / 32];
    lds_words(stage + R::k + r0 * R::kRow + t * (D / 8), k0);
    lds_words(stage + R::k + r1 * R::kRow + t * (D / 8), k1);
    const uint32_t sk0 = e4m3x2_to_f16x2(stage[R::ks + r0 * 4 + t * (D / 4) / 32] * 0x101u);
    const uint32_t sk1 = e4m3x2_to_f16x2(stage[R::ks + r1 * 4 + t * (D / 4) / 32] * 0x101u);
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      uint32_t x0[4], x1[4];
      e2m1x8_to_f16(k0[i], x0);
      e2m1x8_to_f16(k1[i], x1);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const uint32_t af[4] = {mul_f16x2(x0[2 * j], sk0), mul_f16x2(x1[2 * j], sk1), mul_f16x2(x0[2 * j + 1], sk0),
                                mul_f16x2(x1[2 * j + 1], sk1)};
#pragma unroll
        for (int n = 0; n < NT; ++n) mma_f16(s[h][n], af, qf[n][2 * i + j][0], qf[n][2 * i + j][1]);
      }
    }
  }
  // x = the logit above the reference
  bool see[2 * H];
#pragma unroll
  for (int i = 0; i < 2 * H; ++i) see[i] = true;
  if (!w.all(kRows)) {
#pragma unroll
    for (int i = 0; i < 2 * H; ++i) see[i] = w.row(g + 8 * i);
  }
  float x[H][NT][4];
  float top = -INFINITY;
#pragma unroll
  for (int h = 0; h < H; ++h)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[h][n][i] = see[2 * h + (i >> 1)] ? fmaf(s[h][n][i], qs[n][i & 1], -st.mo[n][i & 1]) : -INFINITY;
        top = fmaxf(top, x[h][n][i]);
      }
  // past kFine in every tile, whose x are then taken from rounded logits
  bool move = top > kOffset + kLazy;
#pragma unroll
  for (int n = 0; n < NT; ++n) move = move || past_fine(st.mo[n][0]) || past_fine(st.mo[n][1]);
  if (__any_sync(0xffffffffu, move)) {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float f[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float m = -INFINITY;
#pragma unroll
        for (int i = 0; i < 2 * H; ++i) m = see[i] ? fmaxf(m, __fmul_rn(s[i >> 1][n][2 * (i & 1) + e], qs[n][e])) : m;
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        const float mo = fmaxf(st.mo[n][e], reference(m));
        f[e] = st.mo[n][e] == -INFINITY ? 0.f : ex2(st.mo[n][e] - mo);
        st.mo[n][e] = mo;
        st.l[n][e] *= f[e];
#pragma unroll
        for (int i = 0; i < 2 * H; ++i)
          x[i >> 1][n][2 * (i & 1) + e] = see[i] ? exponent(s[i >> 1][n][2 * (i & 1) + e], qs[n][e], mo) : -INFINITY;
      }
#pragma unroll
      for (int j = 0; j < D / 16; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) st.o[n][j][i] *= f[i & 1];
    }
  }
#pragma unroll
  for (int h = 0; h < H; ++h) {
    uint32_t pf[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float p[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) p[i] = ex2(x[h][n][i]);
      st.l[n][0] += p[0] + p[2];
      st.l[n][1] += p[1] + p[3];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const __half2 hp = __floats2half2_rn(p[2 * i], p[2 * i + 1]);
        pf[n][i] = transpose8x8(*reinterpret_cast<const uint32_t*>(&hp));
      }
    }
    uint32_t v[4][D / 64], sv[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = 16 * h + 2 * t + (i & 1) + 8 * (i >> 1);
      lds_words(stage + R::v + v_at<D>(row, g * (D / 16)), v[i]);
      sv[i] = stage[R::vs + row * 4 + g * (D / 8) / 32];
    }
    const uint32_t sv0 = e4m3x2_to_f16x2(sv[0] | sv[1] << 8), sv1 = e4m3x2_to_f16x2(sv[2] | sv[3] << 8);
#pragma unroll
    for (int c = 0; c < D / 64; ++c) {
      constexpr uint32_t kLow = 0x0F0F0F0Fu;
      uint32_t x0[4], x1[4], x2[4], x3[4];
      e2m1x8_to_f16((v[0][c] & kLow) | ((v[1][c] << 4) & ~kLow), x0);
      e2m1x8_to_f16(((v[0][c] >> 4) & kLow) | (v[1][c] & ~kLow), x1);
      e2m1x8_to_f16((v[2][c] & kLow) | ((v[3][c] << 4) & ~kLow), x2);
      e2m1x8_to_f16(((v[2][c] >> 4) & kLow) | (v[3][c] & ~kLow), x3);
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const uint32_t af[4] = {mul_f16x2(x0[b], sv0), mul_f16x2(x1[b], sv0), mul_f16x2(x2[b], sv1),
                                mul_f16x2(x3[b], sv1)};
#pragma unroll
        for (int n = 0; n < NT; ++n) mma_f16(st.o[n][4 * c + b], af, pf[n][0], pf[n][1]);
      }
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
// before this one; whether any thread has the flag.
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t* sh, int64_t* total, bool flag, bool* any) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t s = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t n = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += n;
  }
  if (lane == 31) sh[warp] = s;
  *any = __syncthreads_or(flag);
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
  pdl_wait();      // launched while the grid before it drains: 2.4 us less per call
  pdl_trigger();

  // ---- where this CTA's run of tiles starts
  int64_t total, all, run;
  {
    const int per = (a.nq + kGqaThreads - 1) / kGqaThreads;
    const int i0 = min(tid * per, a.nq), i1 = min(i0 + per, a.nq);
    const bool empty = looks_empty<kGqaThreads>(a);
    int64_t n = 0;
    for (int i = i0; i < i1; ++i) n += tile_range<kRows>(position(a, i), a.window, a.n_sink).count;
    bool empties;
    int64_t start = block_scan(n, scan_s, &total, empty, &empties);
    all = total * a.groups;
    run = max(div_run(all + a.n_cta - 1, a.n_cta), (int64_t)kMinRun);
    const int64_t u = (int64_t)blockIdx.x * run;
    if (start * a.groups <= u && u < (start + n) * a.groups) {
      for (int i = i0; i < i1; ++i) {
        const int64_t c = tile_range<kRows>(position(a, i), a.window, a.n_sink).count;
        if (start * a.groups <= u && u < (start + c) * a.groups) {
          item_s = i;
          item_start_s = start;
        }
        start += c;
      }
    }
    if (empties) write_empties<kGqaThreads>(a, D);
    if (tid == 0) a.joints[blockIdx.x].i0 = -1;
    __syncthreads();
    if (u >= all) return;
  }
  const int64_t u_begin = (int64_t)blockIdx.x * run, u_end = min(u_begin + run, all);
  const int Hq = a.Hkv * a.G;

  int qi = item_s;
  int64_t q_start = item_start_s * a.groups;       // first tile of the query, over its groups
  for (int64_t u = u_begin; u < u_end;) {
    const int32_t pos = position(a, qi);
    const TileRange ur = tile_range<kRows>(pos, a.window, a.n_sink);
    if (u >= q_start + (int64_t)ur.count * a.groups) {     // on to the next query (or past empty ones)
      q_start += (int64_t)ur.count * a.groups;
      ++qi;
      continue;
    }
    const int grp = a.groups == 1 ? 0 : (int)div_run(u - q_start, ur.count);
    const int64_t i_start = q_start + (int64_t)grp * ur.count, i_end = i_start + ur.count;
    const int32_t c0 = (int32_t)(u - i_start), c1 = (int32_t)(min(u_end, i_end) - i_start);
    const int32_t seq = a.seq_of_query ? __ldg(a.seq_of_query + qi) : qi;
    if (tid == 0 && i_start < u_begin && i_start >= u_begin - run)
      a.joints[blockIdx.x] = GqaJoint{i_start, i_end, run, qi, 1, grp};

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
      // tiles c0 + sub, + share, ...: kStages - 1 of them in flight while one is worked on
      uint8_t* ring_s = gqa_s + warp * GqaRing<D>::warp;
      const uint32_t ring = smem_u32(ring_s);
      const Seen seen = seen_rows(pos, a.window, a.n_sink);
      GqaSource<D> src(a, seq, head, lane);
      int32_t load = c0 + sub;
      uint32_t ks = 0, vs = 0, rooms = 0;          // scales on their way; rows that are there, a byte per stage
      int ls = 0, ws = 0;
      auto rows_of = [&](int32_t p0, int32_t room) {   // what is seen of a tile's rows that are there
        Seen w = seen.from(p0);
        w.hi = min(w.hi, room - 1);
        return w;
      };
      auto start = [&]() {                         // starts the next tile's copies; its scales come back
        if (load < c1) {
          const int32_t p0 = ur.row(load, kRows), step = p0 & ~(kPageStep - 1);
          load += share;
          if (step != src.step) {
            // the step after it, by the last tile of this one's reach
            const int32_t ahead = load + (kPageStep / kRows - 1) / share * share;
            src.go(step, seen.from(step), ahead < c1 ? ur.row(ahead, kRows) & ~(kPageStep - 1) : -1);
          }
          const int32_t room = max(0, min(kRows, src.have - (p0 - step)));
          rooms = (rooms & ~(0xFFu << (8 * ls))) | ((uint32_t)room << (8 * ls));
          if (room > 0) src.copy(p0 - step, ring + ls * GqaRing<D>::stage, rows_of(p0, room), ks, vs);
        }
        copies_commit();
      };
      auto put_scales = [&]() {
        uint32_t* to = reinterpret_cast<uint32_t*>(ring_s + ls * GqaRing<D>::stage + GqaRing<D>::ks) + lane;
        to[0] = ks;
        to[kRows] = vs;
        ls = ls + 1 == kStages ? 0 : ls + 1;
      };
      // kStages - 1 rounds that only start tiles, then one per tile
      for (int32_t x = c0 + sub - (kStages - 1) * share; x < c1; x += share) {
        const bool first = x < c0 + sub - (kStages - 2) * share;
        if (x >= c0) {
          copies_wait<kStages - 2>();
          __syncwarp();                            // the tile is there, and its predecessor's stage is free
        }
        if (!first) put_scales();
        start();
        if (x >= c0) {
          if (const int32_t room = (rooms >> (8 * ws)) & 0xFF)
            tile_step<D, NT>(st, ring_s + ws * GqaRing<D>::stage, qf, qs, rows_of(ur.row(x, kRows), room), g, t);
          ws = ws + 1 == kStages ? 0 : ws + 1;
        }
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

// Joins the parts of every item that several CTAs share: block (x, y) some
// rows of the y-th of them, found by the CTA that starts in its middle first,
// and of every gridDim.y-th one on.  W warps work on one row: the parts'
// weights first, then their rows, N of a warp's in flight.  Latency is all
// there is to it (a serial walk over 128 parts took 24 us, and a block per
// output row of a long chunk 105 us): eight warps per row where there are few
// rows, one where there are many, whose parts are few.  Without a number of
// blocks asked for, the compiler keeps to 32 registers and has the rows come
// one by one (a query over 4,096 rows: 14.2 us, with 64 registers 13.3 us).
constexpr int kCombWarps = 8;
template <int D, int W, int N>
__global__ void __launch_bounds__(kCombWarps * 32, N == 8 ? 4 : 8) gqa_combine_kernel(const __grid_constant__ GqaArgs a,
                                                                      int32_t run_heads, bool one) {
  constexpr int R = kCombWarps / W;                    // rows per block
  constexpr int V = D / 32;                            // values per lane
  __shared__ float acc_s[W > 1 ? W : 1][D];
  __shared__ float w_s[R][kMaxCtas];
  __shared__ float m_s[kCombWarps], l_s[kCombWarps];
  __shared__ int16_t joint_s[kMaxCtas];
  __shared__ int32_t count_s[2 * kCombWarps];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, wr = warp % W, rr = warp / W;
  pdl_wait();
  int n_live = 1;                                      // one item: the second CTA starts in it, or it is whole
  if (one) {
    if (__ldcg(&a.joints[1].i0) < 0) return;
  } else {
    // the CTAs whose first item began in the CTA before them
    static_assert(kMaxCtas <= 2 * kCombWarps * 32, "two CTAs per thread");
    uint32_t own[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int c = i * kCombWarps * 32 + tid;
      own[i] = __ballot_sync(0xffffffffu, c > 0 && c < a.n_cta && __ldcg(&a.joints[c].i0) >= 0);
      if (lane == 0) count_s[i * kCombWarps + warp] = __popc(own[i]);
    }
    __syncthreads();
    n_live = 0;
#pragma unroll
    for (int i = 0; i < 2 * kCombWarps; ++i) {
      const int k = i / kCombWarps;
      if (i % kCombWarps == warp && ((own[k] >> lane) & 1u))
        joint_s[n_live + __popc(own[k] & ((1u << lane) - 1u))] = (int16_t)(k * kCombWarps * 32 + tid);
      n_live += count_s[i];
    }
    __syncthreads();
  }
  const int rows = a.q_tile > 0 ? kBlockRows : a.per_cta * run_heads, row = blockIdx.x * R + rr;
  auto block_sync = [&]() {
    if (W > 1) __syncthreads();
    else __syncwarp();
  };
  for (int y = blockIdx.y; y < n_live; y += gridDim.y) {
    const int joint = one ? 1 : joint_s[y];
    const GqaJoint jt = a.joints[joint];
    const int first = joint - 1, parts = (int)div_run(jt.i1 - 1, jt.run) - first + 1;
    // where the row goes
    int64_t at = -1;
    if (a.q_tile > 0) {
      const int r0 = jt.grp % a.subs * run_heads, gs = min(run_heads, a.G - r0), q = row / gs;
      if (q < jt.n_q)
        at = (int64_t)(jt.q0 + q) * (a.Hkv * a.G) + jt.grp / a.subs * a.G + r0 + row % gs;
    } else {
      const int vh = jt.grp * a.per_cta + row / run_heads, h = vh % a.subs * run_heads + row % run_heads;
      if (row < rows && vh < a.vh && h < a.G) at = (int64_t)jt.q0 * (a.Hkv * a.G) + vh / a.subs * a.G + h;
    }
    if (at < 0) continue;                                // W == kCombWarps: the block is one row
    // part p: the first CTA's last part, then each CTA's first
    auto part = [&](int p) { return (int64_t)(2 * (first + p) + (p == 0 ? 1 : 0)) * rows + row; };
    // the first of a warp's parts, and of a lane's weights, on their way together
    float o[N][V];
    auto load_parts = [&](int p0) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int p = p0 + i * W;
        const float* src = a.part_o + part(p) * D + lane * V;
#pragma unroll
        for (int e = 0; e < V; ++e) o[i][e] = 0.f;
        if (p < parts) {
          if constexpr (V == 4) {
            const float4 v = __ldcg(reinterpret_cast<const float4*>(src));
            o[i][0] = v.x, o[i][1] = v.y, o[i][2] = v.z, o[i][3] = v.w;
          } else {
            const float2 v = __ldcg(reinterpret_cast<const float2*>(src));
            o[i][0] = v.x, o[i][1] = v.y;
          }
        }
      }
    };
    const int mine = wr * 32 + lane;
    const float2 ml0 = mine < parts ? __ldcg(&a.part_ml[part(mine)]) : make_float2(-INFINITY, 0.f);
    load_parts(wr);
    float M = ml0.x;
    for (int p = mine + W * 32; p < parts; p += W * 32) M = fmaxf(M, __ldcg(&a.part_ml[part(p)]).x);
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, x));
    if (W > 1) {
      if (lane == 0) m_s[warp] = M;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < W; ++w) M = fmaxf(M, m_s[w]);
    }
    float l = 0.f;
    for (int p = mine; p < parts; p += W * 32) {
      const float2 ml = p == mine ? ml0 : __ldcg(&a.part_ml[part(p)]);
      // a part without a maximum saw only NaN, and its sum says so
      const float f = ml.x == -INFINITY ? (ml.y != ml.y ? ml.y : 0.f) : ex2(ml.x - M);
      w_s[rr][p] = f;
      l += f * ml.y;
    }
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) l += __shfl_xor_sync(0xffffffffu, l, x);
    if (W > 1 && lane == 0) l_s[warp] = l;
    block_sync();
    float acc[V];
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = 0.f;
    for (int p0 = wr; p0 < parts; p0 += N * W) {
      if (p0 != wr) load_parts(p0);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int p = p0 + i * W;
        const float f = p < parts ? w_s[rr][p] : 0.f;
#pragma unroll
        for (int e = 0; e < V; ++e) acc[e] += f * o[i][e];
      }
    }
    if (W > 1) {
#pragma unroll
      for (int i = 0; i < V; ++i) acc_s[wr][lane * V + i] = acc[i];
      __syncthreads();
      l = 0.f;
#pragma unroll
      for (int i = 0; i < V; ++i) acc[i] = 0.f;
#pragma unroll
      for (int w = 0; w < W; ++w) {
        l += l_s[w];
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] += acc_s[w][lane * V + i];
      }
    }
    if (W == 1 || wr == 0) {
      const float inv = l == 0.f ? 0.f : 1.f / l;
      uint32_t* dst = reinterpret_cast<uint32_t*>(a.out + at * D) + lane * (V / 2);
#pragma unroll
      for (int i = 0; i < V / 2; ++i) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(acc[2 * i] * inv, acc[2 * i + 1] * inv);
        dst[i] = *reinterpret_cast<const uint32_t*>(&b);
      }
      if (lane == 0 && a.lse) a.lse[at] = l == 0.f ? -INFINITY : (M + log2f(l)) * 0.69314718055994531f;
    }
    block_sync();                                      // shared memory is free for the next
  }
}

template <int D, int NT>
cudaError_t launch_gqa_t(GqaArgs& a, cudaStream_t st) {
  static SetupMask done{0};
  constexpr size_t rings = (size_t)kGqaWarps * GqaRing<D>::warp, join = (size_t)kGqaWarps * 8 * NT * (D + 2) * 4;
  constexpr size_t smem = rings > join ? rings : join;
  cudaError_t e = ensure_smem(gqa_split_kernel<D, NT>, (int)smem, done);
  if (e != cudaSuccess) return e;
  a.n_cta = sm_count() * (NT == 1 ? 2 : 1);
  if (a.n_cta > kMaxCtas) a.n_cta = kMaxCtas;
  e = launch_k(gqa_split_kernel<D, NT>, dim3(a.n_cta), dim3(kGqaThreads), smem, st, false, true, a);
  if (e != cudaSuccess) return e;
  return launch_gqa_combine(a, D, 8 * NT, (int64_t)a.nq * a.groups, st);
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

void carve_gqa(GqaArgs& a, Carver& c, int32_t D, int nt) {
  const size_t parts = 2 * (size_t)kMaxCtas * a.per_cta * 8 * nt;
  a.joints = c.take<GqaJoint>(kMaxCtas);
  a.part_o = c.take<float>(parts * D);
  a.part_ml = c.take<float2>(parts);
}

// The block kernel's parts: one CTA per SM, kBlockRows rows each.
void carve_block(GqaArgs& a, Carver& c, int32_t D) {
  const size_t parts = (size_t)kMaxCtas * kBlockRows;
  a.joints = c.take<GqaJoint>(kMaxCtas);
  a.part_o = c.take<float>(parts * D);
  a.part_ml = c.take<float2>(parts);
}

}  // namespace

cudaError_t launch_gqa_combine(const GqaArgs& a, int32_t D, int32_t run_heads, int64_t items, cudaStream_t st) {
  if (a.n_cta < 2) return cudaSuccess;
  const int64_t shared = items < a.n_cta - 1 ? items : a.n_cta - 1;    // items that two CTAs can share
  const int64_t rows = a.q_tile > 0 ? kBlockRows : a.per_cta * run_heads;
  const bool few = shared * rows <= 4 * sm_count();
  // Most of a block of queries' rows and most CTAs' joints may be nobody's: blocks for all of them take longer to come
  // and go than the others to join, so one wave of them goes on from item to item, with two parts in flight for eight
  // blocks per SM (five blocks of 77 queries: 25.1 us with all blocks, 23.7 us so; a chunk of 4,096 280 and 276 us).
  const int64_t x = few ? rows : (rows + kCombWarps - 1) / kCombWarps, most = 8 * sm_count() / x;
  const dim3 grid((unsigned)x, (unsigned)(shared < most || few ? shared : most)), block(kCombWarps * 32);
  const bool one = items == 1;
  auto launch = [&](auto kernel) { return launch_k(kernel, grid, block, 0, st, false, true, a, run_heads, one); };
  if (few) return D == 128 ? launch(gqa_combine_kernel<128, kCombWarps, 8>) : launch(gqa_combine_kernel<64, kCombWarps, 8>);
  if (a.q_tile > 0) return D == 128 ? launch(gqa_combine_kernel<128, 1, 2>) : launch(gqa_combine_kernel<64, 1, 2>);
  return D == 128 ? launch(gqa_combine_kernel<128, 1, 8>) : launch(gqa_combine_kernel<64, 1, 8>);
}

size_t gqa_scratch_bytes(int32_t Hq, int32_t Hkv, int32_t D) {
  GqaArgs a{};
  int nt;
  gqa_heads(a, Hkv, Hq / Hkv, &nt);
  Carver c(nullptr), b(nullptr);
  carve_gqa(a, c, D, nt);
  carve_block(a, b, D);
  return (c.used > b.used ? c.used : b.used) + 256;
}

cudaError_t launch_gqa_attn(const uint16_t* q, const csa2_kv_cache& kv, const int32_t* seq_of_query,
                            const int32_t* query_pos, int32_t nq, int32_t Hq, int32_t window, int32_t n_sink,
                            float scale, bool group_queries, uint16_t* out, float* lse, void* ws, int32_t* status,
                            cudaStream_t st) {
  GqaArgs a{};
  int nt;
  const bool blocks = group_queries && nq > 1;
  gqa_heads(a, kv.Hkv, Hq / kv.Hkv, &nt);
  Carver c(ws);
  if (blocks) carve_block(a, c, kv.D);
  else carve_gqa(a, c, kv.D, nt);
  a.q = q, a.out = out, a.lse = lse;
  const csa2_rows* views[4] = {&kv.k_codes, &kv.k_scales, &kv.v_codes, &kv.v_scales};
  a.one_map = 1;
  int64_t limit = kMaxPositions;
  for (int i = 0; i < 4; ++i) {
    const csa2_rows& v = *views[i];
    const int64_t rows = v.page_table ? (int64_t)v.max_pages * v.page_rows
                         : v.seq_rows > 0 ? std::min<int64_t>(v.seq_rows, v.n_rows) : v.n_rows;
    limit = std::min(limit, rows);
    a.base[i] = static_cast<const uint8_t*>(views[i]->base);
    a.rb[i] = views[i]->row_bytes;
    a.map[i] = to_rowmap(*views[i]);
    if (!same_rows(*views[0], *views[i])) a.one_map = 0;
    a.page_shift[i] = -1;
    for (int b = 6; b < 31; ++b)
      if (views[i]->page_table && views[i]->page_rows == 1 << b) a.page_shift[i] = b;
  }
  a.limit = (int32_t)limit;
  a.seq_of_query = seq_of_query;
  a.query_pos = query_pos;
  a.nq = nq;
  a.window = window;
  a.n_sink = window > 0 ? n_sink : 0;
  a.scale_log2 = scale * 1.4426950408889634f;
  a.status = status;
  if (blocks) {
    gqa_block_shape(a);
    return launch_gqa_block(a, kv.D, st);
  }
  if (kv.D == 128) return nt == 1 ? launch_gqa_t<128, 1>(a, st) : launch_gqa_t<128, 2>(a, st);
  return nt == 1 ? launch_gqa_t<64, 1>(a, st) : launch_gqa_t<64, 2>(a, st);
}

}  // namespace csa2
