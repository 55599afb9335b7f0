// Grouped-query attention over the FP4 cache for blocks of queries that share
// the rows they read (a prefill chunk, a speculative block), on the
// 5th-generation tensor cores.
//
// An item is a block of consecutive queries with one KV head: up to 256 rows
// (query, head of the group), two MMA heights.  It walks 128-row cache tiles:
//   S_m [128 rows][128 positions] = Q_m K^T      (tcgen05, f16 -> fp32 in TMEM)
//   P_m = exp2(S_m scale - max + offset)          (f16, over S_m's columns)
//   O_m [128 rows][D] += P_m V                   (A operand from TMEM)
// One persistent CTA per SM, 17 warps:
//   warps 0-7   softmax, four per height, a thread per row: the running maximum
//               (lazy, as in the split kernel) and sum, P to TMEM, O at the end
//   warps 8-15  expand the codes of K and V into f16 tiles in shared memory
//               (code x scale is exact), two stages each
//   warp 16     issues the MMAs, and builds the next item's list of runs
// While one height's softmax works, the tensor cores take the other's products.
// The queries of a block may belong to several sequences: each run of queries
// of one sequence walks its own tiles, and the others' rows are masked there.
//
// Rows a query does not see are masked in S; a value row must also not reach
// it through 0 x NaN, so a NaN scale in V is taken as 0 there and its row's
// logits are made NaN instead, which the queries that see the row inherit.
#include "csa2_device.cuh"
#include "gqa_attn.cuh"

namespace csa2 {

namespace {

constexpr int kT = 128;                          // cache rows per tile
constexpr int kSoftWarps = 8, kFillWarps = 8;
constexpr int kIssueWarp = kSoftWarps + kFillWarps;
constexpr int kBlockThreads = 32 * (kIssueWarp + 1);
constexpr int kMaxRuns = 256;                    // runs of a block, at most one per query
constexpr int kCountWarps = 7;                   // warps that count tiles in the prologue (their scratch is shared memory)
constexpr int kBadRing = 4;

// The runs of a block: consecutive queries of one sequence.
struct Runs {
  int32_t seq[kMaxRuns];
  int32_t hi[kMaxRuns], lo[kMaxRuns];            // last row seen by any of its queries, first row of any window
  int32_t q[kMaxRuns + 1];                       // its first query, relative to the block
};
struct Item {
  Runs runs;
  int32_t cum[kMaxRuns + 1];                     // tiles before each run
  int32_t n_runs;
  int32_t q0, n_q;                               // queries (q0 < 0: no more items)
  int32_t head, r0, gs;                          // KV head, first query head of the run of heads, their number
  int32_t c0, c1;                                // tiles of the item that are this CTA's
  int32_t slot;                                  // where its part goes (-1: the whole item)
};

template <int D>
struct BlockSmem {
  static constexpr int kPlane = kT * D * 2;      // an f16 tile: [D / 64][128 rows][128 bytes], 128B swizzle
  static constexpr int q = 0, k = 2 * kPlane, v = k + 2 * kPlane, items = v + 2 * kPlane;
  static constexpr int bars = items + 2 * (int)sizeof(Item);
  static constexpr int total = bars + 32 * 8 + 64;
};

struct Bars {
  uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2], s_full[2], p_full[2], item_full[2], item_empty[2], q_full,
      o_full, drain;
};

// MN-major operand tile with the 128-byte swizzle: 64 values along MN are 128
// contiguous bytes, 8 steps along K follow at 128 bytes; `mn` bytes lead to the
// next 64 values and 1024 to the next 8 steps.  Fields as smem_desc_kmajor.
__device__ __forceinline__ uint64_t smem_desc_mnmajor(uint32_t addr, uint32_t mn) {
  return (uint64_t)((addr & 0x3FFFFu) >> 4) | ((uint64_t)(mn >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) | (1ull << 46) |
         (2ull << 61);
}
__host__ __device__ constexpr uint32_t idesc_f16(uint32_t M, uint32_t N, uint32_t b_mn) {
  return (1u << 4) | (b_mn << 16) | ((N >> 3) << 17) | ((M >> 4) << 24);   // f16 x f16 -> f32
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool accumulate) {
  mma_bf16(d, a, b, idesc, accumulate);          // kind::f16: the instruction descriptor names the types
}
// A from TMEM: two f16 per 32-bit column.
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate)
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::"r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]),
      "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
      "r"(r[15]), "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Tiles of a run whose queries see rows up to hi, from lo or below n_sink.
__device__ __forceinline__ TileRange run_tiles(int32_t hi, int32_t lo, int32_t n_sink) {
  if (hi < 0) return TileRange{0, 0, 0};
  const int32_t last = hi / kT, first = lo / kT, sink = n_sink > 0 ? (n_sink - 1) / kT + 1 : 0;
  if (first <= sink) return TileRange{0, 0, last + 1};
  return TileRange{sink, (first - sink) * kT, sink + last + 1 - first};
}

// One warp lists the runs of queries [q0, q0 + n) and, in cum (or nullptr), the
// tiles before each; returns their sum.
__device__ int32_t list_runs(const GqaArgs& a, int32_t q0, int32_t n, Runs& r, int32_t* cum, int32_t* n_runs) {
  const int lane = threadIdx.x & 31;
  int32_t runs = 0, carry = 0;
  for (int base = 0; base < n; base += 32) {
    const int i = base + lane;
    const bool in = i < n;
    const int32_t pos = in ? __ldg(a.query_pos + q0 + i) : -1;
    const int32_t seq = in ? (a.seq_of_query ? __ldg(a.seq_of_query + q0 + i) : q0 + i) : 0;
    int32_t prev = __shfl_up_sync(0xffffffffu, seq, 1);
    if (lane == 0) prev = carry;
    const bool starts = in && (i == 0 || seq != prev);
    const uint32_t b = __ballot_sync(0xffffffffu, starts);
    const int32_t at = runs + __popc(b & (0xffffffffu >> (31 - lane))) - 1;
    if (starts) {
      r.seq[at] = seq;
      r.hi[at] = -1;
      r.lo[at] = 0x7fffffff;
      r.q[at] = i;
    }
    __syncwarp();
    if (pos >= 0) {
      atomicMax(&r.hi[at], pos);
      atomicMin(&r.lo[at], seen_rows(pos, a.window, a.n_sink).lo);
    }
    runs += __popc(b);
    carry = __shfl_sync(0xffffffffu, seq, 31);
    __syncwarp();
  }
  if (lane == 0) r.q[runs] = n;
  int32_t total = 0;
  for (int k0 = 0; k0 < runs; k0 += 32) {
    const int k = k0 + lane;
    const int32_t c = k < runs ? run_tiles(r.hi[k], r.lo[k], a.n_sink).count : 0;
    int32_t s = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int32_t x = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += x;
    }
    if (cum && k < runs) cum[k] = total + s - c;
    total += __shfl_sync(0xffffffffu, s, 31);
  }
  if (cum && lane == 0) cum[runs] = total;
  *n_runs = runs;
  __syncwarp();
  return total;
}

// A role's walk over the tiles of an item.
struct Walk {
  const Item& it;
  const GqaArgs& a;
  int32_t run, first, end;                       // run at hand and its tiles
  __device__ __forceinline__ Walk(const Item& i, const GqaArgs& args) : it(i), a(args), run(-1), first(0), end(0) {}
  // Row of tile x (x does not fall from call to call).
  __device__ __forceinline__ int32_t row(int32_t x) {
    while (x >= end) {
      ++run;
      first = it.cum[run];
      end = it.cum[run + 1];
    }
    return run_tiles(it.runs.hi[run], it.runs.lo[run], a.n_sink).row(x - first, kT);
  }
};

// One lane's parts of a tile in the fill: a block of 32 codes of K and of V in
// one or two rows, with all the row's scales.
template <int D>
struct Fill {
  static constexpr int kPass = D / 64;           // passes over the tile: 64 rows each, or all 128
  uint4 k[kPass], v[kPass];
  uint32_t ks[kPass], vs[kPass];
  uint32_t bad;                                  // bit s: step s of the tile is not there
};

template <int D>
__global__ void __launch_bounds__(kBlockThreads, 1) gqa_block_kernel(const __grid_constant__ GqaArgs a) {
  using L = BlockSmem<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Item* items = reinterpret_cast<Item*>(sm + L::items);
  Bars* bar = reinterpret_cast<Bars*>(sm + L::bars);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + L::bars + 32 * 8);
  volatile int32_t* abort_flag = reinterpret_cast<volatile int32_t*>(tmem_slot + 1);
  int32_t* bad_s = reinterpret_cast<int32_t*>(tmem_slot + 4);          // [kBadRing][2]
  __shared__ int64_t scan_s[kIssueWarp + 1];
  __shared__ int32_t first_s;
  __shared__ int64_t first_start_s;
  static_assert(sizeof(Bars) <= 32 * 8, "barriers");
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int n_blocks = (a.nq + a.q_tile - 1) / a.q_tile;
  pdl_trigger();

  // ---- prologue: barriers, TMEM, and where this CTA's run of tiles starts
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar->k_full[i], kFillWarps);
      mbar_init(&bar->k_empty[i], 1);
      mbar_init(&bar->v_full[i], kFillWarps);
      mbar_init(&bar->v_empty[i], 1);
      mbar_init(&bar->s_full[i], 1);
      mbar_init(&bar->p_full[i], 4);
      mbar_init(&bar->item_full[i], 1);
      mbar_init(&bar->item_empty[i], kSoftWarps + kFillWarps);
    }
    mbar_init(&bar->q_full, kSoftWarps);
    mbar_init(&bar->o_full, 1);
    mbar_init(&bar->drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kIssueWarp) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  int32_t* counts = reinterpret_cast<int32_t*>(sm + kCountWarps * sizeof(Runs));
  if (warp < kCountWarps) {
    Runs& scratch = reinterpret_cast<Runs*>(sm)[warp];
    for (int b = warp; b < n_blocks; b += kCountWarps) {
      int32_t n_runs;
      const int32_t c = list_runs(a, b * a.q_tile, min(a.q_tile, a.nq - b * a.q_tile), scratch, nullptr, &n_runs);
      if (lane == 0) counts[b] = c;
      __syncwarp();
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  int64_t all, run;
  {
    const int per = (n_blocks + kBlockThreads - 1) / kBlockThreads;
    const int b0 = min(tid * per, n_blocks), b1 = min(b0 + per, n_blocks);
    int64_t n = 0;
    for (int b = b0; b < b1; ++b) n += counts[b];
    int64_t s = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t x = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += x;
    }
    if (lane == 31) scan_s[warp] = s;
    __syncthreads();
    int64_t total = 0, start = s - n;
    for (int w = 0; w <= kIssueWarp; ++w) {
      if (w < warp) start += scan_s[w];
      total += scan_s[w];
    }
    all = total * a.groups;
    run = div_run(all + a.n_cta - 1, a.n_cta);
    const int64_t u = (int64_t)blockIdx.x * run;
    for (int b = b0; b < b1; ++b) {
      if (blockIdx.x == 0) a.starts[b] = start;
      if (start * a.groups <= u && u < (start + counts[b]) * a.groups) {
        first_s = b;
        first_start_s = start;
      }
      start += counts[b];
    }
    if (blockIdx.x == 0 && tid == 0) {
      a.starts[n_blocks] = total;
      a.starts[n_blocks + 1] = run;
    }
    __syncthreads();
  }
  const int64_t u_begin = min((int64_t)blockIdx.x * run, all), u_end = min(u_begin + run, all);
  const int Hq = a.Hkv * a.G;

  if (warp == kIssueWarp) {
    // ================================================== MMA issue, item lists
    int blk = u_begin < u_end ? first_s : 0;
    int64_t blk_start = u_begin < u_end ? first_start_s * a.groups : 0, u = u_begin;
    // Writes the item at u into slot s (by the whole warp) and moves u past it.
    auto build = [&](int s) {
      Item& it = items[s];
      if (u >= u_end) {
        if (lane == 0) it.q0 = -1;
        __syncwarp();
        return;
      }
      int32_t n_q, count, n_runs;
      while (true) {
        n_q = min(a.q_tile, a.nq - blk * a.q_tile);
        count = list_runs(a, blk * a.q_tile, n_q, it.runs, it.cum, &n_runs);
        if (u < blk_start + (int64_t)count * a.groups) break;
        blk_start += (int64_t)count * a.groups;
        ++blk;
      }
      const int grp = (int)div_run(u - blk_start, count);
      const int64_t i_start = blk_start + (int64_t)grp * count, i_end = i_start + count;
      if (lane == 0) {
        const int sub = grp % a.subs;
        it.n_runs = n_runs;
        it.q0 = blk * a.q_tile;
        it.n_q = n_q;
        it.head = grp / a.subs;
        it.r0 = sub * kBlockRows;
        it.gs = min(kBlockRows, a.G - sub * kBlockRows);
        it.c0 = (int32_t)(u - i_start);
        it.c1 = (int32_t)(min(u_end, i_end) - i_start);
        it.slot = i_start >= u_begin && i_end <= u_end ? -1 : 2 * (int)blockIdx.x + (i_start < u_begin ? 0 : 1);
      }
      u = min(u_end, i_end);
      __syncwarp();
    };
    constexpr uint32_t kIdS = idesc_f16(128, kT, 0), kIdO = idesc_f16(128, D, 1);
    const uint32_t q_s = smem_u32(sm + L::q), k_s = smem_u32(sm + L::k), v_s = smem_u32(sm + L::v);
    auto logits = [&](int m, int st) {           // S_m = Q_m K^T
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        const uint32_t off = (i / 4) * (kT * 128) + (i % 4) * 32;
        mma_ss(tmem + m * kT, smem_desc_kmajor(q_s + m * L::kPlane + off, 128), smem_desc_kmajor(k_s + st * L::kPlane + off, 128),
               kIdS, i > 0);
      }
      mma_commit(&bar->s_full[m]);
    };
    build(0);
    if (lane == 0) mbar_arrive(&bar->item_full[0]);
    uint32_t n = 0, tiles_m[2] = {0, 0};         // tiles so far, of all and of each height
    for (uint32_t i = 0;; ++i) {
      const Item& it = items[i & 1];
      if (it.q0 < 0) break;
      const int heights = it.n_q * it.gs > 128 ? 2 : 1, tiles = it.c1 - it.c0;
      bool ok = true;
      if (lane == 0) {
        ok = mbar_wait(&bar->q_full, i & 1, abort_flag) && mbar_wait(&bar->k_full[n & 1], (n >> 1) & 1, abort_flag);
        if (ok) {
          tc_fence_after();
          for (int m = 0; m < heights; ++m) logits(m, n & 1);
          mma_commit(&bar->k_empty[n & 1]);
        }
      }
      ok = __shfl_sync(0xffffffffu, ok, 0);
      if (!ok) break;
      // the next item, while the first tile's softmax works
      ok = i < 1 || mbar_wait(&bar->item_empty[(i + 1) & 1], ((i - 1) >> 1) & 1, abort_flag);
      if (!__all_sync(0xffffffffu, ok)) break;
      build((i + 1) & 1);
      if (lane == 0) {
        mbar_arrive(&bar->item_full[(i + 1) & 1]);
        for (int j = 0; j < tiles && ok; ++j, ++n) {
          const int st = n & 1;
          ok = mbar_wait(&bar->v_full[st], (n >> 1) & 1, abort_flag);
          for (int m = 0; m < heights && ok; ++m) {
            ok = mbar_wait(&bar->p_full[m], tiles_m[m]++ & 1, abort_flag);
            if (!ok) break;
            tc_fence_after();
            for (int x = 0; x < kT / 16; ++x)
              mma_ts(tmem + 256 + m * D, tmem + m * kT + x * 8, smem_desc_mnmajor(v_s + st * L::kPlane + x * 2048, kT * 128),
                     kIdO, j > 0 || x > 0);
            if (j + 1 < tiles) {
              if (m == 0) ok = mbar_wait(&bar->k_full[st ^ 1], ((n + 1) >> 1) & 1, abort_flag);
              if (!ok) break;
              tc_fence_after();
              logits(m, st ^ 1);
            }
          }
          if (!ok) break;
          mma_commit(&bar->v_empty[st]);
          if (j + 1 < tiles) mma_commit(&bar->k_empty[st ^ 1]);
        }
        if (ok) mma_commit(&bar->o_full);
      }
      ok = __shfl_sync(0xffffffffu, ok, 0);
      if (!ok) break;
    }
    if (lane == 0) {                             // nothing may still read shared memory when the CTA ends
      mma_commit(&bar->drain);
      const uint64_t t0 = global_ns();
      while (!mbar_try_wait(&bar->drain, 0) && global_ns() - t0 < 100000000ull) {
      }
    }
    __syncwarp();
  } else if (warp >= kSoftWarps) {
    // ================================================== fill: codes to f16 tiles
    const int fw = warp - kSoftWarps;
    constexpr int P = Fill<D>::kPass;
    // lanes are laid out so that a quarter of a warp stores to all 32 banks
    const int row = D == 128 ? fw * 8 + ((lane >> 1) & 3) + (lane >> 4) * 4 : fw * 16 + (lane >> 1);
    const int blk32 = D == 128 ? (lane & 1) + ((lane >> 3) & 1) * 2 : lane & 1;
    uint32_t n = 0;
    for (uint32_t i = 0;; ++i) {
      if (!__all_sync(0xffffffffu, mbar_wait(&bar->item_full[i & 1], (i >> 1) & 1, abort_flag))) break;
      const Item& it = items[i & 1];
      if (it.q0 < 0) break;
      Walk walk(it, a);
      const int head = it.head;
      auto load = [&](int32_t x, Fill<D>& f) {
        const int32_t p0 = walk.row(x), seq = it.runs.seq[walk.run], hi = it.runs.hi[walk.run];
        const Seen seen = Seen{hi, it.runs.lo[walk.run], a.n_sink}.from(p0);
        f.bad = 0;
#pragma unroll
        for (int p = 0; p < P; ++p) {
          const int rr = p * 64 + row, step = D == 128 ? p : fw >> 2;    // row of the tile, its step
          const int32_t sp = p0 + step * kPageStep;
          f.k[p] = f.v[p] = make_uint4(0, 0, 0, 0);
          f.ks[p] = f.vs[p] = 0;
          const int32_t s0 = step * kPageStep;
          // a step without a row to see may have no page
          if (!(s0 <= seen.hi && (s0 + kPageStep > seen.lo || s0 < seen.sk))) continue;
          int64_t r[4];
          bool ok = true;
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            r[y] = y > 0 && a.one_map ? r[0]
                                      : step_base(a.map[y], a.page_shift[y], seq, sp, load_page(a.map[y], a.page_shift[y], seq, sp), hi);
            ok = ok && r[y] >= 0;
          }
          if (!ok) {
            f.bad |= 1u << step;
            continue;
          }
          if (!seen.row(rr)) continue;
          const int in = rr - s0;
          f.k[p] = __ldg(reinterpret_cast<const uint4*>(a.base[0] + (r[0] + in) * a.rb[0] + head * (D / 2) + blk32 * 16));
          f.v[p] = __ldg(reinterpret_cast<const uint4*>(a.base[2] + (r[2] + in) * a.rb[2] + head * (D / 2) + blk32 * 16));
          const uint8_t* ks = a.base[1] + (r[1] + in) * a.rb[1] + head * (D / 32);
          const uint8_t* vs = a.base[3] + (r[3] + in) * a.rb[3] + head * (D / 32);
          if (D == 128) {
            f.ks[p] = __ldg(reinterpret_cast<const uint32_t*>(ks));
            f.vs[p] = __ldg(reinterpret_cast<const uint32_t*>(vs));
          } else {
            f.ks[p] = __ldg(reinterpret_cast<const uint16_t*>(ks));
            f.vs[p] = __ldg(reinterpret_cast<const uint16_t*>(vs));
          }
        }
        if (f.bad && lane == 0) record_error(a.status, CSA2_ERR_INDEX_RANGE);
      };
      // 32 codes of row rr times their scale to the f16 tile
      auto expand = [&](uint8_t* plane, int rr, const uint4& c, uint32_t scale) {
        const uint32_t s2 = e4m3x2_to_f16x2(scale * 0x101u);
        const uint32_t w[4] = {c.x, c.y, c.z, c.w};
        uint8_t* base = plane + (blk32 >> 1) * (kT * 128) + rr * 128;
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          uint32_t o[4];
          e2m1x8_to_f16(w[y], o);
          *reinterpret_cast<uint4*>(base + ((((blk32 & 1) * 4 + y) ^ (rr & 7)) << 4)) =
              make_uint4(mul_f16x2(o[0], s2), mul_f16x2(o[1], s2), mul_f16x2(o[2], s2), mul_f16x2(o[3], s2));
        }
      };
      Fill<D> f[2];
      load(it.c0, f[0]);
      bool ok = true;
      for (int32_t x = it.c0; x < it.c1 && ok;) {
#pragma unroll
        for (int b = 0; b < 2; ++b, ++x, ++n) {
          if (x >= it.c1 || !ok) break;
          if (x + 1 < it.c1) load(x + 1, f[b ^ 1]);
          const Fill<D>& c = f[b];
          const int st = n & 1;
          const uint32_t par = ((n >> 1) & 1) ^ 1;
          ok = __all_sync(0xffffffffu, mbar_wait(&bar->k_empty[st], par, abort_flag));
          if (!ok) break;
          if (lane == 0 && (D == 128 ? fw == 0 : (fw & 3) == 0)) {
            if (D == 128) bad_s[(n % kBadRing) * 2] = c.bad & 1, bad_s[(n % kBadRing) * 2 + 1] = c.bad >> 1;
            else bad_s[(n % kBadRing) * 2 + (fw >> 2)] = c.bad != 0;
          }
#pragma unroll
          for (int p = 0; p < P; ++p) {
            // any NaN scale among the row's values: the row's logits are NaN
            uint32_t s = (c.ks[p] >> (8 * blk32)) & 0xFFu;
            bool nan = false;
#pragma unroll
            for (int y = 0; y < D / 32; ++y) nan |= ((c.vs[p] >> (8 * y)) & 0x7Fu) == 0x7Fu;
            if (nan) s = 0x7Fu;
            expand(sm + L::k + st * L::kPlane, p * 64 + row, c.k[p], s);
          }
          fence_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bar->k_full[st]);
          ok = __all_sync(0xffffffffu, mbar_wait(&bar->v_empty[st], par, abort_flag));
          if (!ok) break;
#pragma unroll
          for (int p = 0; p < P; ++p) {
            uint32_t s = (c.vs[p] >> (8 * blk32)) & 0xFFu;
            if ((s & 0x7Fu) == 0x7Fu) s = 0;
            expand(sm + L::v + st * L::kPlane, p * 64 + row, c.v[p], s);
          }
          fence_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bar->v_full[st]);
        }
      }
      if (!ok) break;
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar->item_empty[i & 1]);
    }
  } else {
    // ================================================== softmax: a thread per row
    const int m = warp >> 2, r = tid & 127;      // height, row of it
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;
    const uint32_t s_t = tmem + m * kT + lanes, o_t = tmem + 256 + m * D + lanes;
    uint32_t n_all = 0, n_s = 0;                 // tiles so far, and those of this height
    for (uint32_t i = 0;; ++i) {
      if (!__all_sync(0xffffffffu, mbar_wait(&bar->item_full[i & 1], (i >> 1) & 1, abort_flag))) break;
      const Item& it = items[i & 1];
      if (it.q0 < 0) break;
      const int rows = it.n_q * it.gs, at = m * 128 + r;
      const bool live = at < rows;
      const int qr = live ? at / it.gs : 0;      // query of the block
      const int64_t out_row = (int64_t)(it.q0 + qr) * Hq + it.head * a.G + it.r0 + (at - qr * it.gs);
      // ---- this row of Q, scaled by a power of two into f16
      float qs;
      {
        uint4 w[D / 8];
        uint32_t top = 0;
#pragma unroll
        for (int c = 0; c < D / 8; ++c) {
          w[c] = live ? __ldg(reinterpret_cast<const uint4*>(a.q + out_row * D) + c) : make_uint4(0, 0, 0, 0);
          const uint32_t x[4] = {w[c].x, w[c].y, w[c].z, w[c].w};
#pragma unroll
          for (int e = 0; e < 4; ++e) top = max(top, max(x[e] & 0x7FFFu, (x[e] >> 16) & 0x7FFFu));
        }
        const int e = max((int)(top >> 7), 20);
        const float up = __uint_as_float((uint32_t)(268 - e) << 23);
        qs = __uint_as_float((uint32_t)(e - 14) << 23) * a.scale_log2;
        uint8_t* dst = sm + L::q + m * L::kPlane + r * 128;
#pragma unroll
        for (int c = 0; c < D / 8; ++c) {
          const uint32_t x[4] = {w[c].x, w[c].y, w[c].z, w[c].w};
          uint32_t o[4];
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            const __half2 hh = __floats2half2_rn(__uint_as_float(x[y] << 16) * up, __uint_as_float(x[y] & 0xFFFF0000u) * up);
            o[y] = *reinterpret_cast<const uint32_t*>(&hh);
          }
          *reinterpret_cast<uint4*>(dst + (c / 8) * (kT * 128) + (((c & 7) ^ (r & 7)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
        }
      }
      fence_async_smem();
      tc_fence_before();                         // O of the item before has been read
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar->q_full);
      const int32_t pos = live ? __ldg(a.query_pos + it.q0 + qr) : -1;
      const Seen mine = seen_rows(pos, a.window, a.n_sink);
      float mo = -INFINITY, l = 0.f;
      bool ok = true;
      const bool active = m == 0 || rows > 128;
      Walk walk(it, a);
      for (int32_t x = it.c0; x < it.c1 && active; ++x, ++n_s) {
        const int32_t p0 = walk.row(x);
        // what this row sees of the tile: everything, or by a mask
        const bool in_run = pos >= 0 && qr >= it.runs.q[walk.run] && qr < it.runs.q[walk.run + 1];
        const Seen w = mine.from(p0);
        ok = __all_sync(0xffffffffu, mbar_wait(&bar->s_full[m], n_s & 1, abort_flag));
        if (!ok) break;
        tc_fence_after();
        const uint32_t t = n_all + (uint32_t)(x - it.c0);
        const int32_t bad0 = bad_s[(t % kBadRing) * 2], bad1 = bad_s[(t % kBadRing) * 2 + 1];
        const bool full = __all_sync(0xffffffffu, in_run && w.all(kT) && !(bad0 | bad1));
        uint32_t see[4] = {~0u, ~0u, ~0u, ~0u};
        if (!full) {
          // bits of columns [32 y, 32 y + 32): c <= hi && (c >= lo || c < sk)
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            auto below = [&](int32_t c) {        // columns < c
              const int32_t k = c - 32 * y;
              return k <= 0 ? 0u : (k >= 32 ? ~0u : (1u << k) - 1u);
            };
            see[y] = below(w.hi + 1) & (~below(w.lo) | below(w.sk));
            if (!in_run || (y < 2 ? bad0 : bad1)) see[y] = 0;
          }
        }
        // the largest logit seen
        float top = -INFINITY;
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          uint32_t s[32];
          tmem_ld32(s_t + 32 * y, s);
          tmem_wait_ld();
          if (full) {
#pragma unroll
            for (int c = 0; c < 32; ++c) top = fmaxf(top, __uint_as_float(s[c]));
          } else {
#pragma unroll
            for (int c = 0; c < 32; ++c) top = (see[y] >> c) & 1u ? fmaxf(top, __uint_as_float(s[c])) : top;
          }
        }
        top = top == -INFINITY ? top : top * qs;
        if (__any_sync(0xffffffffu, top > mo + (kOffset + kLazy))) {
          const float m_new = fmaxf(mo, top - kOffset);
          const float f = mo == -INFINITY ? 0.f : ex2(mo - m_new);
          mo = m_new;
          l *= f;
          if (x > it.c0) {
#pragma unroll 1
            for (int y = 0; y < D / 32; ++y) {
              uint32_t o[32];
              tmem_ld32(o_t + 32 * y, o);
              tmem_wait_ld();
              uint32_t half[16];
#pragma unroll
              for (int z = 0; z < 2; ++z) {
#pragma unroll
                for (int c = 0; c < 16; ++c) half[c] = __float_as_uint(__uint_as_float(o[16 * z + c]) * f);
                tmem_st16(o_t + 32 * y + 16 * z, half);
              }
            }
            tmem_wait_st();
          }
        }
        // the weights, over the logits' columns
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          uint32_t s[32], p[16];
          tmem_ld32(s_t + 32 * y, s);
          tmem_wait_ld();
          if (full) {
#pragma unroll
            for (int c = 0; c < 32; ++c) s[c] = __float_as_uint(ex2(fmaf(__uint_as_float(s[c]), qs, -mo)));
          } else {
#pragma unroll
            for (int c = 0; c < 32; ++c)
              s[c] = (see[y] >> c) & 1u ? __float_as_uint(ex2(fmaf(__uint_as_float(s[c]), qs, -mo))) : 0u;
          }
#pragma unroll
          for (int c = 0; c < 16; ++c) {
            const float p0f = __uint_as_float(s[2 * c]), p1f = __uint_as_float(s[2 * c + 1]);
            l += p0f + p1f;
            const __half2 hh = __floats2half2_rn(p0f, p1f);
            p[c] = *reinterpret_cast<const uint32_t*>(&hh);
          }
          tmem_st16(s_t + 16 * y, p);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar->p_full[m]);
      }
      if (!ok) break;
      n_all += (uint32_t)(it.c1 - it.c0);
      // ---- the output, or this CTA's part of it
      ok = __all_sync(0xffffffffu, mbar_wait(&bar->o_full, i & 1, abort_flag));
      if (!ok) break;
      tc_fence_after();
      if (active) {
        const int slot = it.slot;
        const float inv = l == 0.f ? 0.f : 1.f / l;
        const int64_t part = (int64_t)slot * kBlockRows + at;
#pragma unroll 1
        for (int y = 0; y < D / 32; ++y) {
          uint32_t o[32];
          tmem_ld32(o_t + 32 * y, o);
          tmem_wait_ld();
          if (live && slot < 0) {
            uint4* dst = reinterpret_cast<uint4*>(a.out + out_row * D + 32 * y);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              uint32_t b[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const __nv_bfloat162 bb = __floats2bfloat162_rn(__uint_as_float(o[8 * c + 2 * e]) * inv,
                                                                __uint_as_float(o[8 * c + 2 * e + 1]) * inv);
                b[e] = *reinterpret_cast<const uint32_t*>(&bb);
              }
              dst[c] = make_uint4(b[0], b[1], b[2], b[3]);
            }
          } else if (live) {
            uint4* dst = reinterpret_cast<uint4*>(a.part_o + part * D + 32 * y);
#pragma unroll
            for (int c = 0; c < 8; ++c) dst[c] = make_uint4(o[4 * c], o[4 * c + 1], o[4 * c + 2], o[4 * c + 3]);
          }
        }
        if (live && slot < 0 && a.lse)
          a.lse[out_row] = l == 0.f ? -INFINITY : (mo + log2f(l)) * 0.69314718055994531f;
        if (live && slot >= 0) a.part_ml[part] = make_float2(mo, l);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar->item_empty[i & 1]);
    }
    tc_fence_before();
  }
  __syncthreads();
  if (warp == kIssueWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  if (tid == 0 && *abort_flag) record_error(a.status, CSA2_ERR_TIMEOUT);
}

template <int D>
cudaError_t launch_block_t(GqaArgs& a, cudaStream_t st) {
  static SetupMask done{0};
  constexpr int smem = BlockSmem<D>::total + 1024 + 64;
  static_assert(smem <= 227 * 1024, "shared memory");
  static_assert(kCountWarps * (int)sizeof(Runs) + 16384 * 4 <= BlockSmem<D>::items, "the prologue's counts fit the tiles");
  cudaError_t e = ensure_smem(gqa_block_kernel<D>, smem, done);
  if (e != cudaSuccess) return e;
  gqa_block_kernel<D><<<a.n_cta, kBlockThreads, smem, st>>>(a);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch_gqa_combine(a, D, kBlockRows, st);
}

}  // namespace

void gqa_block_shape(GqaArgs& a) {
  a.q_tile = a.G <= kBlockRows ? kBlockRows / a.G : 1;
  a.subs = (a.G + kBlockRows - 1) / kBlockRows;
  a.vh = a.groups = a.Hkv * a.subs;
  a.per_cta = 1;
}

cudaError_t launch_gqa_block(GqaArgs& a, int32_t D, cudaStream_t st) {
  a.n_cta = sm_count() < 160 ? sm_count() : 160;
  return D == 128 ? launch_block_t<128>(a, st) : launch_block_t<64>(a, st);
}

}  // namespace csa2
