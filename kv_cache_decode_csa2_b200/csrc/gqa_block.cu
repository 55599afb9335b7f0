// Grouped-query attention over the FP4 cache for blocks of queries that share
// the rows they read (a prefill chunk, a speculative block), on the
// 5th-generation tensor cores.
//
// An item is a run of consecutive queries of one sequence with one KV head: up
// to 256 rows (query, head of the group), two MMA heights.  It walks 128-row
// cache tiles:
//   S_m [128 rows][128 positions] = Q_m K^T      (tcgen05, f16 -> fp32 in TMEM)
//   P_m = exp2(S_m scale - max + offset)          (f16, over S_m's columns)
//   O_m [128 rows][D] += P_m V                   (A operand from TMEM)
// One persistent CTA per SM, 16 warps (17 would cost every thread 32 of its
// 128 registers):
//   warps 0-7   softmax, four per height, a thread per row: the running maximum
//               (lazy, as in the split kernel) and sum, P to TMEM, O at the end
//   warps 8-14  expand the codes of K and V into f16 tiles in shared memory
//               (code x scale is exact), two stages each
//   warp 15     issues the MMAs, and works out ahead where the others' tiles are
// The issuer takes the heights in turn (P V of a tile, then Q K^T of the next),
// so that the tensor cores work for one while the other is at its softmax;
// issued by the softmax warps themselves the heights fell into step, and an
// issuing warp was late for its own tile.  An item of at most 128 rows has its
// tiles dealt out to the two heights in turn, whose results join at the end.
// Queries are taken in blocks of as many as fit 256 rows, and a block falls
// into the runs of its queries' sequences, one item each per KV head.
//
// Measured on 64 query and 8 KV heads, D = 128: 2,048 queries over 16,384 rows
// 1.10 to 1.14 ms (903 to 940 TFLOP/s, 0.55 to 0.57 of the dense f16 rate), a
// windowed chunk of 4,096 (1,024 rows and 4 sinks) 266 to 269 us, 8 blocks of 5
// queries over 158,000 rows 161 to 165 us; the chunk of 2,048 at D = 64 0.95 ms.
// A 128-row tile takes 4,700 clocks: 3,000 of softmax, the rest products and
// hand-over, the other height's between them.
//
// Rows a query does not see are masked in S; a value row must also not reach
// it through 0 x NaN, so a NaN scale in V is taken as 0 there and its row's
// logits are made NaN instead, which the queries that see the row inherit.
#include "csa2_device.cuh"
#include "gqa_attn.cuh"

namespace csa2 {

namespace {

constexpr int kT = 128;                          // cache rows per tile
constexpr int kSoftWarps = 8, kFillWarps = 7;
constexpr int kIssueWarp = kSoftWarps + kFillWarps;
constexpr int kWarps = kIssueWarp + 1;
constexpr int kBlockThreads = 32 * kWarps;
constexpr int kMaxRuns = 256;                    // runs of a block, at most one per query
// Warps that count tiles in the prologue; their scratch is the tiles' space, which at D = 64 has room for seven.
template <int D>
constexpr int kCountWarps = D == 128 ? kWarps : 7;
constexpr int kBatch = 16;                       // tiles whose places are worked out together

// Where a tile is: worked out kBatch tiles at a time, a lane per step of 64
// rows (done by every filling warp for itself, it took longer than the softmax).
struct alignas(16) Place {
  int32_t end[2], lo, sk;                        // its rows that are there and may be seen: of step s those below end[s], from lo or below sk
  uint32_t r[2][4];                              // first physical row of each step in each plane
  int32_t row, pad[3];                           // its first row
};

// The runs of a block: consecutive queries of one sequence.
struct Runs {
  int32_t seq[kMaxRuns];
  int32_t hi[kMaxRuns], lo[kMaxRuns];            // last row seen by any of its queries, first row of any window
  int32_t q[kMaxRuns + 1];                       // its first query, relative to the block
};
struct Item {
  int32_t q0, n_q;                               // its queries (q0 < 0: no more items)
  int32_t seq, hi, lo;                           // their sequence and rows
  int32_t head, r0, gs;                          // KV head, first query head of the run of heads, their number
  int32_t c0, c1;                                // tiles of the item that are this CTA's
  int32_t slot;                                  // where its part goes (-1: the whole item)
};

template <int D>
struct BlockSmem {
  static constexpr int kPlane = kT * D * 2;      // an f16 tile: [D / 64][128 rows][128 bytes], 128B swizzle
  static constexpr int q = 0, k = 2 * kPlane, v = k + 2 * kPlane, items = v + 2 * kPlane;
  static constexpr int runs = items + 2 * (int)sizeof(Item), cum = runs + (int)sizeof(Runs);
  static constexpr int places = (cum + (kMaxRuns + 1) * 4 + 15) / 16 * 16;
  static constexpr int bars = places + 2 * kBatch * (int)sizeof(Place);
  static constexpr int total = bars + 32 * 8 + 64;
};

struct Bars {
  uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2], s_full[2], p_full[2], o_full[2], item_full[2], item_empty[2],
      place_full[2], q_full, both_done, stored, taken, drain;
};

// Waits as mbar_wait does, but asleep for up to a few microseconds at a time:
// sixteen warps that poll take the issue slots of those that work.
__device__ __forceinline__ bool sleepy_try(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity), "r"(4000u)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ bool block_wait(uint64_t* bar, uint32_t parity, volatile int32_t* abort_flag) {
  if (sleepy_try(bar, parity)) return true;
  const uint64_t t0 = global_ns();
  while (true) {
    if (sleepy_try(bar, parity)) return true;
    if (*abort_flag) return false;
    if (global_ns() - t0 > kWaitLimitNs) {
      *abort_flag = 1;
      return false;
    }
  }
}
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
// A tcgen05.ld delivers its registers only at the wait: the values go through
// it, so that nothing that uses them can be placed before.
__device__ __forceinline__ void tmem_wait_ld16(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]),
                 "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :
               : "memory");
}
__device__ __forceinline__ void tmem_wait_ld32(uint32_t (&r)[32]) {
  uint32_t (&lo)[16] = *reinterpret_cast<uint32_t (*)[16]>(&r[0]);
  uint32_t (&hi)[16] = *reinterpret_cast<uint32_t (*)[16]>(&r[16]);
  tmem_wait_ld16(lo);
  tmem_wait_ld16(hi);
}
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n\ttcgen05.wait::ld.sync.aligned;"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr)
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
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%8], {%0,%1,%2,%3,%4,%5,%6,%7};" ::"r"(r[0]), "r"(r[1]), "r"(r[2]),
               "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(taddr)
               : "memory");
}
// Two fp32 operations per instruction.
__device__ __forceinline__ float2 fma2(uint32_t x0, uint32_t x1, float m, float c) {
  float2 r;
  asm("{\n\t.reg .b64 x, y, z;\n\t"
      "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %4};\n\tmov.b64 z, {%5, %5};\n\t"
      "fma.rn.f32x2 x, x, y, z;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "r"(x0), "r"(x1), "f"(m), "f"(c));
  return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ void add2(float2& acc, float x0, float x1) {
  asm("{\n\t.reg .b64 x, y;\n\t"
      "mov.b64 x, {%0, %1};\n\tmov.b64 y, {%2, %3};\n\t"
      "add.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "+f"(acc.x), "+f"(acc.y)
      : "f"(x0), "f"(x1));
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
    const int32_t pos = in ? position(a, q0 + i) : -1;
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

template <int D>
__global__ void __launch_bounds__(kBlockThreads, 1) gqa_block_kernel(const __grid_constant__ GqaArgs a) {
  using L = BlockSmem<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Item* items = reinterpret_cast<Item*>(sm + L::items);
  Bars* bar = reinterpret_cast<Bars*>(sm + L::bars);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + L::bars + 32 * 8);
  volatile int32_t* abort_flag = reinterpret_cast<volatile int32_t*>(tmem_slot + 1);
  Place* places = reinterpret_cast<Place*>(sm + L::places);            // [2][kBatch]
  __shared__ int64_t scan_s[kWarps];
  __shared__ float2 join_s[128];
  __shared__ int32_t first_s;
  __shared__ int64_t first_start_s;
  static_assert(sizeof(Bars) <= 32 * 8, "barriers");
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int n_blocks = (a.nq + a.q_tile - 1) / a.q_tile;
  pdl_wait();      // launched while the grid before it drains
  pdl_trigger();

  const bool empty = looks_empty<kBlockThreads>(a);

  // ---- prologue: barriers, TMEM, and where this CTA's run of tiles starts
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar->k_full[i], kFillWarps);
      mbar_init(&bar->k_empty[i], 1);
      mbar_init(&bar->v_full[i], kFillWarps);
      mbar_init(&bar->v_empty[i], 1);
      mbar_init(&bar->s_full[i], 1);
      mbar_init(&bar->p_full[i], 4);             // the four warps of a height
      mbar_init(&bar->o_full[i], 1);
      mbar_init(&bar->item_full[i], 1);
      mbar_init(&bar->place_full[i], 1);
      mbar_init(&bar->item_empty[i], kSoftWarps + kFillWarps);
    }
    mbar_init(&bar->both_done, kSoftWarps);      // both heights of an item that they share
    mbar_init(&bar->stored, 4);
    mbar_init(&bar->taken, 4);
    mbar_init(&bar->q_full, kSoftWarps);
    mbar_init(&bar->drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  int32_t* counts = reinterpret_cast<int32_t*>(sm + kCountWarps<D> * sizeof(Runs));
  if (warp >= kWarps - kCountWarps<D>) {
    const int cw = warp - (kWarps - kCountWarps<D>);
    Runs& scratch = reinterpret_cast<Runs*>(sm)[cw];
    for (int b = cw; b < n_blocks; b += kCountWarps<D>) {
      int32_t n_runs;
      const int32_t c = list_runs(a, b * a.q_tile, min(a.q_tile, a.nq - b * a.q_tile), scratch, nullptr, &n_runs);
      if (lane == 0) counts[b] = c;
      __syncwarp();
    }
  }
  tc_fence_before();
  const bool empties = __syncthreads_or(empty);
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
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) start += scan_s[w];
      total += scan_s[w];
    }
    all = total * a.groups;
    run = div_run(all + a.n_cta - 1, a.n_cta);
    const int64_t u = (int64_t)blockIdx.x * run;
    for (int b = b0; b < b1; ++b) {
      if (start * a.groups <= u && u < (start + counts[b]) * a.groups) {
        first_s = b;
        first_start_s = start;
      }
      start += counts[b];
    }
    if (empties) write_empties<kBlockThreads>(a, D);
    if (tid == 0) a.joints[blockIdx.x].i0 = -1;
    __syncthreads();
  }
  const int64_t u_begin = min((int64_t)blockIdx.x * run, all), u_end = min(u_begin + run, all);
  const int Hq = a.Hkv * a.G;

  if (warp == kIssueWarp) {
    // ================================================== MMA issue, item lists
    int blk = u_begin < u_end ? first_s : 0, listed = -1, n_runs = 0;
    int32_t count = 0;                           // tiles of the block listed, for one head
    int64_t blk_start = u_begin < u_end ? first_start_s * a.groups : 0, u = u_begin;
    Runs& runs = *reinterpret_cast<Runs*>(sm + L::runs);
    int32_t* cum = reinterpret_cast<int32_t*>(sm + L::cum);        // tiles before each run
    // Writes the item at u into slot s (by the whole warp) and moves u past it.
    // A block's items go run by run, head by head.
    auto build = [&](int s) {
      Item& it = items[s];
      if (u >= u_end) {
        if (lane == 0) it.q0 = -1;
        __syncwarp();
        return;
      }
      while (true) {
        if (listed != blk) {
          count = list_runs(a, blk * a.q_tile, min(a.q_tile, a.nq - blk * a.q_tile), runs, cum, &n_runs);
          listed = blk;
        }
        if (u < blk_start + (int64_t)count * a.groups) break;
        blk_start += (int64_t)count * a.groups;
        ++blk;
      }
      int k = 0, last = n_runs - 1;              // the run: cum <= tile < cum of the next
      const int64_t in_block = u - blk_start;
      while (k < last) {
        const int mid = (k + last + 1) >> 1;
        if ((int64_t)cum[mid] * a.groups <= in_block) k = mid;
        else last = mid - 1;
      }
      const int32_t n = cum[k + 1] - cum[k];
      const int grp = (int)div_run(in_block - (int64_t)cum[k] * a.groups, n);
      const int64_t i_start = blk_start + (int64_t)cum[k] * a.groups + (int64_t)grp * n, i_end = i_start + n;
      if (lane == 0) {
        const int sub = grp % a.subs;
        it.q0 = blk * a.q_tile + runs.q[k];
        it.n_q = runs.q[k + 1] - runs.q[k];
        it.seq = runs.seq[k];
        it.hi = runs.hi[k];
        it.lo = runs.lo[k];
        it.head = grp / a.subs;
        it.r0 = sub * kBlockRows;
        it.gs = min(kBlockRows, a.G - sub * kBlockRows);
        it.c0 = (int32_t)(u - i_start);
        it.c1 = (int32_t)(min(u_end, i_end) - i_start);
        it.slot = i_start >= u_begin && i_end <= u_end ? -1 : 2 * (int)blockIdx.x + (i_start < u_begin ? 0 : 1);
        if (i_start < u_begin && i_start >= u_begin - run)
          a.joints[blockIdx.x] = GqaJoint{i_start, i_end, run, it.q0, it.n_q, grp};
      }
      u = min(u_end, i_end);
      __syncwarp();
    };
    constexpr uint32_t kIdS = idesc_f16(128, kT, 0), kIdO = idesc_f16(128, D, 1);
    const uint64_t q_d = smem_desc_kmajor(smem_u32(sm + L::q), 128), k_d = smem_desc_kmajor(smem_u32(sm + L::k), 128),
                   v_d = smem_desc_mnmajor(smem_u32(sm + L::v), kT * 128);
    auto wait = [&](uint64_t* b, uint32_t parity) {
      return (bool)__all_sync(0xffffffffu, block_wait(b, parity, abort_flag));
    };
    // Issued by one elected lane; descriptors come from uniform registers.
    auto logits = [&](int m, uint32_t n) {       // S_m = Q_m K^T of the CTA's tile n
      const uint64_t qd = q_d + (uint32_t)(m * (L::kPlane >> 4)), kd = k_d + (uint32_t)((n & 1) * (L::kPlane >> 4));
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        const uint32_t off = ((i / 4) * (kT * 128) + (i % 4) * 32) >> 4;
        mma_ss(tmem + m * kT, qd + off, kd + off, kIdS, i > 0);
      }
      mma_commit(&bar->s_full[m]);
    };
    auto values = [&](int m, uint32_t n, bool first) {   // O_m += P_m V of tile n
      const uint64_t vd = v_d + (uint32_t)((n & 1) * (L::kPlane >> 4));
#pragma unroll
      for (int i = 0; i < kT / 16; ++i)
        mma_ts(tmem + 256 + m * D, tmem + m * kT + i * 8, vd + (uint32_t)(i * (2048 >> 4)), kIdO, !first || i > 0);
    };
    // Works out the places of kBatch tiles of an item from tile x on, into half
    // `h` of the ring: lane 2 k + s has step s of tile x + k.
    auto locate = [&](const Item& it, int32_t x, uint32_t h) {
      const int32_t t = x + (lane >> 1);
      const int s = lane & 1;
      const bool in = t < it.c1;
      Place* pl = places + h * kBatch + (lane >> 1);
      bool bad = false;
      int32_t p0 = 0, have = 0;
      Seen w{-1, 0, 0};
      if (in) {
        const int32_t seq = it.seq;
        p0 = run_tiles(it.hi, it.lo, a.n_sink).row(t, kT);
        w = Seen{it.hi, it.lo, a.n_sink}.from(p0);
        // a step without a row to see may have no page
        const int32_t at = p0 + s * kPageStep;
        const Seen ws = w.from(s * kPageStep);
        if (ws.some(0, kPageStep - 1)) {
          uint32_t r0 = 0;
          have = kPageStep;
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            if (y == 0 || !a.one_map)            // rows of a plane fit 31 bits
              r0 = (uint32_t)step_rows(a.map[y], a.page_shift[y], seq, at, load_page(a.map[y], a.page_shift[y], seq, at), have);
            pl->r[s][y] = r0;
          }
          // an error only if a query sees them: between the windows of far queries pages may have been given back
          if (have < kPageStep && ws.some(have, kPageStep - 1))
            for (int i = 0; i < it.n_q && !bad; ++i)
              bad = seen_rows(position(a, it.q0 + i), a.window, a.n_sink).from(at).some(have, kPageStep - 1);
        }
        pl->end[s] = s * kPageStep + min(have, w.hi + 1 - s * kPageStep);
        if (s == 0) {
          pl->lo = w.lo;
          pl->sk = w.sk;
          pl->row = p0;
        }
      }
      if (__any_sync(0xffffffffu, bad) && lane == 0) record_error(a.status, CSA2_ERR_INDEX_RANGE);
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar->place_full[h]);
    };
    build(0);
    if (lane == 0) mbar_arrive(&bar->item_full[0]);
    uint32_t batch = 0;                          // batches of places so far
    if (items[0].q0 >= 0) locate(items[0], items[0].c0, 0);
    uint32_t n0 = 0, n_p[2] = {0, 0};            // tiles before the item; batches of each height
    for (uint32_t i = 0;; ++i) {
      const Item& it = items[i & 1];
      if (it.q0 < 0) break;
      const bool pair = it.n_q * it.gs <= 128;   // both heights hold the same rows and take every other tile
      const uint32_t tiles = it.c1 - it.c0;
      bool ok = wait(&bar->q_full, i & 1) && wait(&bar->k_full[n0 & 1], (n0 >> 1) & 1);
      if (ok && pair && tiles > 1) ok = wait(&bar->k_full[(n0 + 1) & 1], ((n0 + 1) >> 1) & 1);
      if (!ok) break;
      tc_fence_after();
      if (elect_one()) {
        logits(0, n0);
        if (!pair) logits(1, n0);
        mma_commit(&bar->k_empty[n0 & 1]);
        if (pair && tiles > 1) {
          logits(1, n0 + 1);
          mma_commit(&bar->k_empty[(n0 + 1) & 1]);
        }
      }
      __syncwarp();
      // the next item, while the first tile's softmax works
      if (i > 0 && !wait(&bar->item_empty[(i + 1) & 1], ((i - 1) >> 1) & 1)) break;
      build((i + 1) & 1);
      if (lane == 0) mbar_arrive(&bar->item_full[(i + 1) & 1]);
      // batches: P V of a tile, then Q K^T of the height's next.  The operands
      // are waited for before P: while an S product reads shared memory at its
      // full rate, a barrier there takes hundreds of clocks.  Heights that take
      // every other tile wait for K last (201 -> 169 us for 8 blocks of 5
      // queries: V of the tile after next was filled later for it).
      const uint32_t step = pair ? 2 : 1, batches = pair ? tiles : 2 * tiles;
      for (uint32_t b = 0; b < batches && ok; ++b) {
        const int m = b & 1;
        const uint32_t j = pair ? b : b >> 1, n = n0 + j, nn = n + step;
        const bool more = j + step < tiles, last_use = pair || m == 1;
        ok = wait(&bar->v_full[n & 1], (n >> 1) & 1) && (pair || !more || wait(&bar->k_full[nn & 1], (nn >> 1) & 1)) &&
             wait(&bar->p_full[m], n_p[m] & 1);
        if (!ok) break;
        ++n_p[m];
        tc_fence_after();
        if (elect_one()) {
          values(m, n, j < step);
          if (last_use) mma_commit(&bar->v_empty[n & 1]);
          if (!more) {
            mma_commit(&bar->o_full[m]);
          } else {
            if (pair) {
              ok = block_wait(&bar->k_full[nn & 1], (nn >> 1) & 1, abort_flag);
              tc_fence_after();
            }
            if (ok) {
              logits(m, nn);
              if (last_use) mma_commit(&bar->k_empty[nn & 1]);
            }
          }
        }
        ok = __all_sync(0xffffffffu, ok);
        // The first tile of a batch is through: the batch before is done with
        // (its tiles' P have all been taken), and its half of the ring is free.
        if (j % kBatch == 0 && (pair || m == 1)) {
          ++batch;
          const Item& then = items[(i + 1) & 1];
          if (j + kBatch < tiles) locate(it, it.c0 + j + kBatch, batch & 1);
          else if (then.q0 >= 0) locate(then, then.c0, batch & 1);
        }
      }
      if (!ok) break;
      n0 += tiles;
    }
    if (elect_one()) {                           // nothing may still read shared memory when the CTA ends
      mma_commit(&bar->drain);
      const uint64_t t0 = global_ns();
      while (!mbar_try_wait(&bar->drain, 0) && global_ns() - t0 < 100000000ull) {
      }
    }
    __syncwarp();
  } else if (warp >= kSoftWarps) {
    // ================================================== fill: codes to f16 tiles
    // A group is 8 (D = 64: 16) rows of a tile, a lane a block of 32 codes of one of
    // them; lanes are laid out so that a quarter of a warp stores to all 32
    // banks.  Warp f expands groups f, f + 7, ... of K and of V; of the groups
    // left over, the first warps take K's and the last ones V's.
    const int fw = warp - kSoftWarps;
    constexpr int NG = D == 128 ? 16 : 8, EACH = NG / kFillWarps, PER = EACH + 1, LEFT = NG - EACH * kFillWarps, GR = kT / NG;
    const int in_g = D == 128 ? ((lane >> 1) & 3) + (lane >> 4) * 4 : lane >> 1;
    const int blk32 = D == 128 ? (lane & 1) + ((lane >> 3) & 1) * 2 : lane & 1;
    const int left = kFillWarps - 1 - fw;        // of V's left over, this one's (K's: fw)
    auto k_group = [&](int j) { return fw + j * kFillWarps; };
    auto v_group = [&](int j) { return j < EACH ? fw + j * kFillWarps : EACH * kFillWarps + left; };
    static_assert(LEFT > 0 && 2 * LEFT <= kFillWarps && PER * GR <= 32 && EACH >= 1, "one warp has at most one group left over");
    // The scales of all its rows are loaded at once, a row per lane, and handed
    // round (loaded with each block of codes they kept the load pipe waiting).
    const int s_group = lane / GR < EACH ? k_group(lane / GR)
                        : lane / GR == EACH && fw < LEFT ? k_group(EACH)
                        : lane / GR == EACH && left < LEFT ? v_group(EACH) : NG;
    const int s_row = s_group * GR + lane % GR;
    const uint32_t s_in = s_row & (kPageStep - 1);
    // Everything that does not change from tile to tile is worked out here: a
    // filling warp gets an instruction in every eight clocks or so, and with
    // the addresses made for each load the fill took longer than the softmax.
    uint32_t in_k[PER], in_v[PER];               // this lane's row of each group, within its step
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      in_k[j] = (k_group(j) * GR + in_g) & (kPageStep - 1);
      in_v[j] = (v_group(j) * GR + in_g) & (kPageStep - 1);
    }
    constexpr int kNext = kFillWarps * GR * 128; // bytes from one of its groups to the next in a tile
    uint8_t* to[4];                              // where the four chunks of its block go in K's first group
#pragma unroll
    for (int y = 0; y < 4; ++y)
      to[y] = sm + L::k + (blk32 >> 1) * (kT * 128) + (fw * GR + in_g) * 128 + ((((blk32 & 1) * 4 + y) ^ (in_g & 7)) << 4);
    const int to_v_left = (v_group(EACH) - fw) * GR * 128;         // of V's group left over, from the first
    const uint32_t my_scale = blk32 * 0x11;      // byte_perm selector: this block's scale, twice
    uint32_t n = 0, batch = 0;                   // tiles and batches of places so far
    for (uint32_t i = 0;; ++i) {
      if (!__all_sync(0xffffffffu, block_wait(&bar->item_full[i & 1], (i >> 1) & 1, abort_flag))) break;
      const Item& it = items[i & 1];
      if (it.q0 < 0) break;
      const uint8_t* const bk = a.base[0] + it.head * (D / 2) + blk32 * 16;
      const uint8_t* const bks = a.base[1] + it.head * (D / 32);
      const uint8_t* const bv = a.base[2] + it.head * (D / 2) + blk32 * 16;
      const uint8_t* const bvs = a.base[3] + it.head * (D / 32);
      int4 seen = {};                            // the place of the tile whose loads are next
      uint4 pr[2] = {};
      bool ok = true;
      auto rows_of = [&](int32_t x) {            // moves to tile x
        const int32_t j = x - it.c0;
        if (j % kBatch == 0) {
          ok = __all_sync(0xffffffffu, block_wait(&bar->place_full[batch & 1], (batch >> 1) & 1, abort_flag));
          ++batch;
        }
        const Place& pl = places[((batch - 1) & 1) * kBatch + j % kBatch];
        seen = *reinterpret_cast<const int4*>(pl.end);
        pr[0] = *reinterpret_cast<const uint4*>(pl.r[0]);
        pr[1] = *reinterpret_cast<const uint4*>(pl.r[1]);
      };
      uint4 kc[PER], vc[PER];
      uint32_t ks = 0, vs = 0;                   // scales of row s_row in K and V
      uint32_t vf[PER];                          // the V blocks' scales, twice
      // (volatile: a plain load may be moved past the barriers to where it is used)
      auto load_scales = [&](const uint8_t* p) {
        uint32_t r;
        if (D == 128)
          asm volatile("ld.global.nc.b32 %0, [%1];" : "=r"(r) : "l"(p));
        else
          asm volatile("{\n\t.reg .b16 t;\n\tld.global.nc.b16 t, [%1];\n\tcvt.u32.u16 %0, t;\n\t}" : "=r"(r) : "l"(p));
        return r;
      };
      auto load_codes = [&](const uint8_t* base, uint32_t r, int64_t rb) {
        uint4 u;
        asm volatile("ld.global.nc.v4.b32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w)
                     : "l"(base + (uint64_t)r * (uint32_t)rb));
        return u;
      };
      auto has_k = [&](int j) { return j < EACH || fw < LEFT; };
      auto has_v = [&](int j) { return j < EACH || left < LEFT; };
      auto seen_row = [&](int rr) {              // whether row rr of the tile is to be read
        return rr < (rr >= kPageStep ? seen.y : seen.x) && (rr >= seen.z || rr < seen.w);
      };
      auto load_k = [&]() {
        ks = vs = 0;
        if (s_group < NG && seen_row(s_row)) {
          const bool hi = s_row >= kPageStep;
          ks = load_scales(bks + (uint64_t)((hi ? pr[1].y : pr[0].y) + s_in) * (uint32_t)a.rb[1]);
          vs = load_scales(bvs + (uint64_t)((hi ? pr[1].w : pr[0].w) + s_in) * (uint32_t)a.rb[3]);
        }
#pragma unroll
        for (int j = 0; j < PER; ++j) {
          const int rr = k_group(j) * GR + in_g;
          kc[j] = make_uint4(0, 0, 0, 0);
          if (has_k(j) && seen_row(rr)) kc[j] = load_codes(bk, (rr >= kPageStep ? pr[1].x : pr[0].x) + in_k[j], a.rb[0]);
        }
      };
      auto load_v = [&]() {
#pragma unroll
        for (int j = 0; j < PER; ++j) {
          const int rr = v_group(j) * GR + in_g;
          vc[j] = make_uint4(0, 0, 0, 0);
          if (has_v(j) && seen_row(rr)) vc[j] = load_codes(bv, (rr >= kPageStep ? pr[1].z : pr[0].z) + in_v[j], a.rb[2]);
        }
      };
      // Nothing of these loads is to be used before this point: scales taken
      // apart where they are loaded make the warp wait there.
      auto arrived = [&](uint4& c) { asm volatile("" : "+r"(c.x), "+r"(c.y), "+r"(c.z), "+r"(c.w)); };
      // 32 codes times their scale (twice in s2's bytes) to the f16 tile, `off`
      // bytes from K's first group
      auto expand = [&](int off, const uint4& c, uint32_t s2) {
        const uint32_t w[4] = {c.x, c.y, c.z, c.w};
        const uint32_t f = e4m3x2_to_f16x2(s2);
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          uint32_t o[4];
          e2m1x8_to_f16(w[y], o);
          *reinterpret_cast<uint4*>(to[y] + off) =
              make_uint4(mul_f16x2(o[0], f), mul_f16x2(o[1], f), mul_f16x2(o[2], f), mul_f16x2(o[3], f));
        }
      };
      rows_of(it.c0);
      if (!ok) break;
      load_k();
      load_v();
      for (int32_t x = it.c0; x < it.c1; ++x, ++n) {
        const int st = n & 1;
        const uint32_t par = ((n >> 1) & 1) ^ 1;
        // (read now: while products read shared memory, a trip there is long)
        if (x + 1 < it.c1) rows_of(x + 1);
        ok = ok && __all_sync(0xffffffffu, block_wait(&bar->k_empty[st], par, abort_flag));
        if (!ok) break;
#pragma unroll
        for (int j = 0; j < PER; ++j) arrived(kc[j]);
        asm volatile("" : "+r"(ks), "+r"(vs));
#pragma unroll
        for (int j = 0; j < PER; ++j) {
          const uint32_t k4 = __shfl_sync(0xffffffffu, ks, (j * GR + in_g) & 31), v4 = __shfl_sync(0xffffffffu, vs, (j * GR + in_g) & 31);
          const uint32_t v2 = __byte_perm(v4, 0, my_scale);
          vf[j] = (v2 & 0x7Fu) == 0x7Fu ? 0u : v2;
          if (!has_k(j)) break;
          // any NaN scale (0x7F without its sign) among the row's values: its logits are NaN
          const bool nan = ((v4 & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
          expand(st * L::kPlane + j * kNext, kc[j], nan ? 0x7F7Fu : __byte_perm(k4, 0, my_scale));
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar->k_full[st]);
        if (x + 1 < it.c1) load_k();
        ok = __all_sync(0xffffffffu, block_wait(&bar->v_empty[st], par, abort_flag));
        if (!ok) break;
#pragma unroll
        for (int j = 0; j < PER; ++j) arrived(vc[j]);
#pragma unroll
        for (int j = 0; j < PER; ++j)
          if (has_v(j)) expand(L::v - L::k + st * L::kPlane + (j < EACH ? j * kNext : to_v_left), vc[j], vf[j]);
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar->v_full[st]);
        if (x + 1 < it.c1) load_v();
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
    uint32_t n_batch = 0, n_s = 0, n_o = 0, n_pair = 0;   // batches of places so far; this height's tiles, outputs, shared items
    for (uint32_t i = 0;; ++i) {
      if (!__all_sync(0xffffffffu, block_wait(&bar->item_full[i & 1], (i >> 1) & 1, abort_flag))) break;
      const Item& it = items[i & 1];
      if (it.q0 < 0) break;
      const int rows = it.n_q * it.gs;
      const bool pair = rows <= 128;             // both heights hold the same rows and take every other tile
      const int at = (pair ? 0 : m * 128) + r, step = pair ? 2 : 1;
      const bool live = at < rows;
      const int qr = live ? at / it.gs : 0;      // query of the run
      const int64_t out_row = (int64_t)(it.q0 + qr) * Hq + it.head * a.G + it.r0 + (at - qr * it.gs);
      const int32_t x0 = it.c0 + (pair ? m : 0), c1 = it.c1;
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
        // (not 0, which would make the -inf of a row that is not seen a NaN)
        qs = fmaxf(__uint_as_float((uint32_t)(e - 14) << 23) * a.scale_log2, 1e-38f);
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
      bool ok = true;
      const int32_t pos = live ? position(a, it.q0 + qr) : -1;
      const Seen mine = seen_rows(pos, a.window, a.n_sink);
      float mo = -INFINITY;                      // the row's reference
      float mul = qs, sub = 0.f;                 // a weight's exponent is x mul - sub of what stands in a column
      float2 l = make_float2(0.f, 0.f);
      const bool idle = !__any_sync(0xffffffffu, live);      // no row of this warp is anyone's
      for (int32_t x = x0; x < c1; x += step, ++n_s) {
        ok = __all_sync(0xffffffffu, ok && block_wait(&bar->s_full[m], n_s & 1, abort_flag));
        if (!ok) break;
        tc_fence_after();
        // what this row sees of the tile: everything, or by a mask
        const int32_t j = x - it.c0;
        const Place& pl = places[((n_batch + j / kBatch) & 1) * kBatch + j % kBatch];
        const Seen w = live ? mine.from(pl.row) : Seen{kT, 0, 0};   // a row behind the last counts as seeing all
        const int2 end = *reinterpret_cast<const int2*>(pl.end);
        const bool full = __all_sync(0xffffffffu, w.all(kT) && end.x == kPageStep && end.y == kT);
        // bits of columns [32 y, 32 y + 32) seen: c <= hi && (c >= lo || c < sk), of rows that are there
        auto below = [](int32_t k) { return k <= 0 ? 0u : (k >= 32 ? ~0u : (1u << k) - 1u); };
        auto see = [&](int y) {
          return below(min(w.hi + 1, y < 2 ? end.x : end.y) - 32 * y) & (~below(w.lo - 32 * y) | below(w.sk - 32 * y));
        };
        // The weights, 32 columns at a time, over the logits' columns.  The
        // reference moves only when a logit exceeds it by kLazy (past kFine in
        // every tile, to the largest of the columns left): O, the sum and the
        // weights of the tile already stored are then scaled, and these
        // columns, taken on trust, are taken again, once.  (One rolled loop:
        // the code of the roles has to stay in the instruction caches together.)
        mul = qs;
        float limit = fabsf(mo) <= kFine ? kOffset + kLazy : -INFINITY;
#pragma unroll 1
        for (int y = idle ? 4 : 0; y < 4;) {
          uint32_t s[32];
          tmem_ld32(s_t + 32 * y, s);
          tmem_wait_ld32(s);
          if (!full) {
            const uint32_t bits = see(y);        // unseen: a logit of -inf, whatever it was
#pragma unroll
            for (int c = 0; c < 32; ++c)
              if (!((bits >> c) & 1u)) s[c] = 0xFF800000u;
          }
          float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
          for (int c = 0; c < 16; ++c) {
            const float2 v = fma2(s[2 * c], s[2 * c + 1], mul, -sub);
            s[2 * c] = __float_as_uint(v.x), s[2 * c + 1] = __float_as_uint(v.y);
            top[c & 1] = max3(top[c & 1], v.x, v.y);
          }
          float2 add = make_float2(0.f, 0.f);
          uint32_t p[16];
#pragma unroll
          for (int c = 0; c < 16; ++c) {
            const float p0f = ex2(__uint_as_float(s[2 * c])), p1f = ex2(__uint_as_float(s[2 * c + 1]));
            add2(add, p0f, p1f);
            const __half2 hh = __floats2half2_rn(p0f, p1f);
            p[c] = *reinterpret_cast<const uint32_t*>(&hh);
          }
          const float most = fmaxf(top[0], top[1]);
          if (!__any_sync(0xffffffffu, most > limit)) {
            l.x += add.x, l.y += add.y;
            tmem_st16(s_t + 16 * y, p);
            if (limit == INFINITY) limit = mo == -INFINITY ? -INFINITY : kOffset + kLazy;
            ++y;
            continue;
          }
          // a whole number: weights already rounded are scaled exactly
          const bool done = past_fine(mo) && limit > -INFINITY;      // an earlier turn of this tile did what follows
          float m_new = done ? mo : fmaxf(mo, reference(floorf(most + sub)));
          const bool far = !done && (past_fine(mo) || past_fine(m_new));
          if (__any_sync(0xffffffffu, far)) {
            // these rows' logits, each rounded once, in the products' place, and the largest
            float high = -INFINITY;
#pragma unroll 1
            for (int z = 2 * y; z < 8; ++z) {
              const uint32_t bits = full ? ~0u : see(z >> 1) >> (16 * (z & 1));
              uint32_t b[16];
              tmem_ld16(s_t + 16 * z, b);
              tmem_wait_ld16(b);
#pragma unroll
              for (int c = 0; c < 16; ++c) {
                const float v = __fmul_rn(__uint_as_float(b[c]), qs);
                if ((bits >> c) & 1u) high = fmaxf(high, v);
                if (far) b[c] = __float_as_uint(v);
              }
              tmem_st16(s_t + 16 * z, b);
            }
            if (far) m_new = fmaxf(mo, reference(floorf(high)));
          }
          const float f = mo == -INFINITY ? 0.f : ex2(mo - m_new);
          mo = m_new;
          if (far) mul = 1.f;
          sub = mo == -INFINITY ? 0.f : mo;
          limit = INFINITY;                      // taken now, whatever comes
          l.x *= f, l.y *= f;
          tmem_wait_st();                        // the weights before are in place
#pragma unroll 1
          for (int z = 0; z < 2 * y; ++z) {
            uint32_t b[8];
            tmem_ld8(s_t + 8 * z, b);
#pragma unroll
            for (int c = 0; c < 8; ++c) {        // in fp32: f may be below f16's smallest step
              const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&b[c]));
              const __half2 hh = __floats2half2_rn(v.x * f, v.y * f);
              b[c] = *reinterpret_cast<const uint32_t*>(&hh);
            }
            tmem_st8(s_t + 8 * z, b);
          }
          if (x > x0) {
#pragma unroll 1
            for (int z = 0; z < D / 8; ++z) {
              uint32_t o[8];
              tmem_ld8(o_t + 8 * z, o);
#pragma unroll
              for (int c = 0; c < 8; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * f);
              tmem_st8(o_t + 8 * z, o);
            }
          }
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar->p_full[m]);
      }
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      const bool some = x0 < c1;
      if (some) {
        ok = __all_sync(0xffffffffu, block_wait(&bar->o_full[m], n_o++ & 1, abort_flag));
        if (!ok) break;
        tc_fence_after();
      }
      n_batch += (uint32_t)(c1 - it.c0 + kBatch - 1) / kBatch;
      float sum = l.x + l.y, scale = 1.f;
      if (pair) {
        // the second height's maximum, sum and O join the first's, in the space of Q
        float* o_s = reinterpret_cast<float*>(sm + L::q);      // [D / 4][128 rows] of four values
        if (lane == 0) mbar_arrive(&bar->both_done);           // and its products are done with it
        ok = __all_sync(0xffffffffu, block_wait(&bar->both_done, n_pair & 1, abort_flag));
        if (!ok) break;
        if (m == 1) {
#pragma unroll 1
          for (int y = 0; y < D / 16; ++y) {
            uint32_t o[16];
            if (some) {
              tmem_ld16(o_t + 16 * y, o);
              tmem_wait_ld16(o);
            }
#pragma unroll
            for (int c = 0; c < 4; ++c)
              reinterpret_cast<uint4*>(o_s)[(4 * y + c) * 128 + r] =
                  some ? make_uint4(o[4 * c], o[4 * c + 1], o[4 * c + 2], o[4 * c + 3]) : make_uint4(0, 0, 0, 0);
          }
          join_s[r] = make_float2(mo, sum);
          __syncwarp();
          if (lane == 0) mbar_arrive(&bar->stored);
        } else {
          ok = __all_sync(0xffffffffu, block_wait(&bar->stored, n_pair & 1, abort_flag));
          if (!ok) break;
          const float2 ml = join_s[r];
          const float top = fmaxf(mo, ml.x);
          // a side without a maximum saw nothing, or only NaN: its sum is 0 or NaN
          const float f0 = mo == -INFINITY ? (sum != sum ? sum : 0.f) : ex2(mo - top);
          scale = ml.x == -INFINITY ? (ml.y != ml.y ? ml.y : 0.f) : ex2(ml.x - top);
          sum = sum * f0 + ml.y * scale;
          mo = top;
          l.x = f0;                              // O of the first height is scaled by it below
        }
      }
      // ---- the output, or this CTA's part of it
      if (!pair || m == 0) {
        const int slot = it.slot;
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        const int64_t part = (int64_t)slot * kBlockRows + at;
#pragma unroll 1
        for (int y = 0; y < D / 16; ++y) {
          uint32_t o[16];
          tmem_ld16(o_t + 16 * y, o);
          tmem_wait_ld16(o);
          if (pair) {
            const uint4* other = reinterpret_cast<const uint4*>(sm + L::q);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const uint4 b = other[(4 * y + c) * 128 + r];
              const uint32_t bw[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
              for (int e = 0; e < 4; ++e)
                o[4 * c + e] = __float_as_uint(__uint_as_float(o[4 * c + e]) * l.x + __uint_as_float(bw[e]) * scale);
            }
          }
          if (live && slot < 0) {
            uint4* dst = reinterpret_cast<uint4*>(a.out + out_row * D + 16 * y);
#pragma unroll
            for (int c = 0; c < 2; ++c) {
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
            uint4* dst = reinterpret_cast<uint4*>(a.part_o + part * D + 16 * y);
#pragma unroll
            for (int c = 0; c < 4; ++c) dst[c] = make_uint4(o[4 * c], o[4 * c + 1], o[4 * c + 2], o[4 * c + 3]);
          }
        }
        if (live && slot < 0 && a.lse)
          a.lse[out_row] = sum == 0.f ? -INFINITY : (mo + log2f(sum)) * 0.69314718055994531f;
        if (live && slot >= 0) a.part_ml[part] = make_float2(mo, sum);
      }
      __syncwarp();
      if (pair) {                                // the space of Q is free when the first height has read it
        if (m == 0 && lane == 0) mbar_arrive(&bar->taken);
        ok = __all_sync(0xffffffffu, block_wait(&bar->taken, n_pair & 1, abort_flag));
        if (!ok) break;
        ++n_pair;
      }
      if (lane == 0) mbar_arrive(&bar->item_empty[i & 1]);
    }
    tc_fence_before();
  }
  __syncthreads();
  if (warp == 0) {
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
  static_assert(kCountWarps<D> * (int)sizeof(Runs) + 16384 * 4 <= BlockSmem<D>::items, "the prologue's counts fit the tiles");
  cudaError_t e = ensure_smem(gqa_block_kernel<D>, smem, done);
  if (e != cudaSuccess) return e;
  e = launch_k(gqa_block_kernel<D>, dim3(a.n_cta), dim3(kBlockThreads), smem, st, false, true, a);
  if (e != cudaSuccess) return e;
  return launch_gqa_combine(a, D, kBlockRows, (int64_t)a.nq * a.groups, st);   // a run per query at most
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
