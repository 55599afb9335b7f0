// Append of keys and values to the grouped-query FP4 cache, with the position
// rotation applied on the way.
//
// Row i is token row_pos[i] of its sequence.  Its query and key heads are
// turned by the position's angles, pair by pair (a, b):
//   a' = a cos - b sin,  b' = b cos + a sin
// in fp32 with each product and each sum rounded once (no contraction), so
// the stored codes do not depend on how the compiler fuses the expression.
// Keys and values are then quantised in blocks of 32 (fp4_device.cuh: E4M3
// scale nearest to amax / 6, E2M1 codes nearest to x / scale) straight from
// fp32 and written where the page table puts the position; queries leave as
// bf16.  A block that holds a NaN gets the NaN scale, so attention over that
// row shows it; infinities saturate to the largest stored value.
//
// Bound by HBM: every value is read once and written once, and the table row
// of a position is read once per slot.  A slot of lanes owns one head at a
// time.  For keys and values a lane has eight values (16 bytes of bf16): loads
// and stores are coalesced, a block's maximum is two shuffles, and the rotation
// partner of the half-split layout is one shuffle away; for queries, which are
// most of the work, it has both sides of eight pairs.  A slot walks `per` heads of
// its token with the angles in registers, kBatch heads' loads in flight (queries:
// two heads' of bf16, one of fp32).
//
// Measured on 64 query and 8 KV heads, D = 128, bf16: 32,768 tokens 271 to 275 us
// (1.38 GB, 5.05 TB/s, 0.77 of the copy rate), 2,048 tokens 23.9 us (3.65
// TB/s), 32 tokens 6.5 to 7.1 us, which is the launch; 32,768 tokens of fp32 402
// us (5.10 TB/s), of D = 64 145 us (4.75 TB/s).  What is left waits for loads.
#include "csa2_device.cuh"
#include "fp4_device.cuh"
#include "internal.h"

namespace csa2 {

namespace {

constexpr int kAppendThreads = 256;
constexpr int kBatch = 4;     // heads whose loads are in flight at once

struct AppendArgs {
  const void* x[3];           // q, k, v rows
  int64_t ld[3];              // row strides in values
  int32_t heads[3];           // Hq (0: no queries), Hkv, Hkv
  int32_t first[3];           // first chunk of each kind within a token
  int32_t chunks;             // chunks of a token
  int32_t per;                // heads per chunk
  int64_t n;
  const int32_t* seq_of_row;
  const int32_t* row_pos;
  const float* cos_sin;       // [n_pos][rot]: cosines, then sines
  int64_t n_pos;
  int32_t rot;
  uint8_t* codes[2];          // K, V
  uint8_t* scales[2];
  int64_t codes_rb[2], scales_rb[2];
  RowMap cmap[2], smap[2];
  int32_t cshift[2], sshift[2];   // log2 of the rows per page (-1: not a power of two)
  int32_t one_map;            // all four planes place rows alike
  uint16_t* q_out;            // [n][Hq][D]
  uint16_t* kv_out[2];        // [n][Hkv][D] or nullptr
  int32_t* status;
};

// The row of (seq, pos), refusing a position outside the sequence's own
// share of a contiguous plane.
__device__ __forceinline__ int64_t write_row(const RowMap& m, int32_t shift, int32_t seq, int32_t pos) {
  if (seq < 0) return -1;
  int64_t r;
  if (m.page_table) {
    const int32_t pg = shift >= 0 ? pos >> shift : pos / m.page_rows;
    const int32_t phys = pg < m.max_pages ? __ldg(m.page_table + (int64_t)seq * m.max_pages + pg) : -1;
    r = phys < 0 ? -1 : (int64_t)phys * m.page_rows + (pos - pg * m.page_rows);
  } else {
    r = m.seq_rows > 0 && pos >= m.seq_rows ? -1 : (int64_t)seq * m.seq_rows + pos;
  }
  return r < m.n_rows ? r : -1;
}

template <bool F32>
struct Raw {                  // eight values as loaded
  uint4 u[F32 ? 2 : 1];
};
template <bool F32>
__device__ __forceinline__ Raw<F32> load8(const void* base, int64_t at) {
  Raw<F32> r;
  const uint4* p = reinterpret_cast<const uint4*>(static_cast<const char*>(base) + at * (F32 ? 4 : 2));
#pragma unroll
  for (int i = 0; i < (F32 ? 2 : 1); ++i) r.u[i] = p[i];
  return r;
}
template <bool F32>
__device__ __forceinline__ void widen(const Raw<F32>& r, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < (F32 ? 2 : 1); ++i) {
    const uint32_t w[4] = {r.u[i].x, r.u[i].y, r.u[i].z, r.u[i].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (F32) {
        v[4 * i + j] = __uint_as_float(w[j]);
      } else {
        v[2 * j] = __uint_as_float(w[j] << 16);
        v[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
      }
    }
  }
}
template <bool F32>
__device__ __forceinline__ Raw<F32> from_lane(uint32_t mask, const Raw<F32>& r, int lane, int width) {
  Raw<F32> o;
#pragma unroll
  for (int i = 0; i < (F32 ? 2 : 1); ++i) {
    o.u[i].x = __shfl_sync(mask, r.u[i].x, lane, width);
    o.u[i].y = __shfl_sync(mask, r.u[i].y, lane, width);
    o.u[i].z = __shfl_sync(mask, r.u[i].z, lane, width);
    o.u[i].w = __shfl_sync(mask, r.u[i].w, lane, width);
  }
  return o;
}

__device__ __forceinline__ float turn_a(float a, float b, float c, float s) {
  return __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
}
__device__ __forceinline__ float turn_b(float a, float b, float c, float s) {
  return __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
}

// Where a token goes: its rows in [K, V][codes, scales].  False for a padding
// row, and, with the error recorded, for a token out of range: a token is
// stored whole or not at all.
__device__ __forceinline__ bool place_token(const AppendArgs& a, int64_t row, bool report, int32_t& pos,
                                            int64_t (&rows)[2][2]) {
  pos = __ldg(a.row_pos + row);
  if (pos < 0) return false;
  const int32_t seq = a.seq_of_row ? __ldg(a.seq_of_row + row) : (int32_t)row;
  rows[0][0] = write_row(a.cmap[0], a.cshift[0], seq, pos);
  rows[0][1] = a.one_map ? rows[0][0] : write_row(a.smap[0], a.sshift[0], seq, pos);
  rows[1][0] = a.one_map ? rows[0][0] : write_row(a.cmap[1], a.cshift[1], seq, pos);
  rows[1][1] = a.one_map ? rows[0][0] : write_row(a.smap[1], a.sshift[1], seq, pos);
  const bool ok = !(a.rot > 0 && pos >= a.n_pos) && rows[0][0] >= 0 && rows[0][1] >= 0 && rows[1][0] >= 0 &&
                  rows[1][1] >= 0;
  if (!ok && report) record_error(a.status, CSA2_ERR_INDEX_RANGE);
  return ok;
}

__device__ __forceinline__ void load_angles(const float* t, int half, float (&co)[8], float (&si)[8]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float4 c4 = __ldg(reinterpret_cast<const float4*>(t) + i);
    const float4 s4 = __ldg(reinterpret_cast<const float4*>(t + half) + i);
    co[4 * i] = c4.x, co[4 * i + 1] = c4.y, co[4 * i + 2] = c4.z, co[4 * i + 3] = c4.w;
    si[4 * i] = s4.x, si[4 * i + 1] = s4.y, si[4 * i + 2] = s4.z, si[4 * i + 3] = s4.w;
  }
}

// Queries: a lane has sixteen values of a head, of the half-split layout both
// sides of eight pairs, so that the rotation asks nothing of other lanes.
template <int D, bool F32, bool PAIRS>
__device__ __forceinline__ void append_queries(const AppendArgs& a, uint32_t tokens, int chunk) {
  constexpr int LPH = D / 16, QB = F32 ? 1 : 2;   // lanes per head; heads whose loads are in flight
  const int64_t row = ((int64_t)tokens * kAppendThreads + threadIdx.x) / LPH;
  const int l = threadIdx.x % LPH;
  if (row >= a.n) return;
  int32_t pos;
  int64_t rows[2][2];
  if (!place_token(a, row, l == 0, pos, rows)) return;
  const int half = a.rot / 2;
  const bool turned = l * 16 < a.rot;
  const int first = PAIRS || !turned ? l * 16 : l * 8, second = PAIRS || !turned ? first + 8 : first + half;
  float co[8], si[8];
  if (turned) load_angles(a.cos_sin + (int64_t)pos * a.rot + l * 8, half, co, si);
  const int h0 = chunk * a.per, h1 = min(h0 + a.per, a.heads[0]);
  const int64_t in = row * a.ld[0], out = row * a.heads[0] * D;
  for (int hb = h0; hb < h1; hb += QB) {
    Raw<F32> raw[QB][2];
#pragma unroll
    for (int j = 0; j < QB; ++j)
      if (hb + j < h1) {
        raw[j][0] = load8<F32>(a.x[0], in + (hb + j) * D + first);
        raw[j][1] = load8<F32>(a.x[0], in + (hb + j) * D + second);
      }
#pragma unroll
    for (int j = 0; j < QB; ++j) {
      if (hb + j >= h1) break;
      float v[2][8];
      widen<F32>(raw[j][0], v[0]);
      widen<F32>(raw[j][1], v[1]);
      if (turned) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          float& x = PAIRS ? v[e / 4][2 * (e % 4)] : v[0][e];
          float& y = PAIRS ? v[e / 4][2 * (e % 4) + 1] : v[1][e];
          const float nx = turn_a(x, y, co[e], si[e]);
          y = turn_b(x, y, co[e], si[e]);
          x = nx;
        }
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const __nv_bfloat162 b = __floats2bfloat162_rn(v[i][2 * e], v[i][2 * e + 1]);
          w[e] = *reinterpret_cast<const uint32_t*>(&b);
        }
        *reinterpret_cast<uint4*>(a.q_out + out + (hb + j) * D + (i ? second : first)) = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
  }
}

// Keys (KV = 0) or values (KV = 1): a lane has eight values of a head.
template <int D, bool F32, bool PAIRS, int KV>
__device__ __forceinline__ void append_rows(const AppendArgs& a, uint32_t tokens, int chunk) {
  constexpr int LPH = D / 8;
  const int64_t row = ((int64_t)tokens * kAppendThreads + threadIdx.x) / LPH;
  const int l = threadIdx.x % LPH, lane = threadIdx.x & 31;
  const uint32_t mask = ((1u << LPH) - 1u) << (lane / LPH * LPH);
  if (row >= a.n) return;
  const int h0 = (chunk - a.first[1 + KV]) * a.per, h1 = min(h0 + a.per, a.heads[1 + KV]);
  int32_t pos;
  int64_t rows[2][2];
  if (!place_token(a, row, l == 0, pos, rows)) return;
  // this lane's angles: eight of the half-split layout (values l*8..l*8+7 are
  // one side of eight pairs), four of the interleaved one
  const int half = a.rot / 2;
  const bool turned = KV == 0 && l * 8 < a.rot;
  const bool low = l * 8 < half;
  const int partner = !turned || PAIRS ? l : (low ? l + half / 8 : l - half / 8);
  constexpr int NA = PAIRS ? 4 : 8;
  float co[NA], si[NA];
  if (turned) {
    const float* t = a.cos_sin + (int64_t)pos * a.rot + (PAIRS ? l * 4 : (low ? l * 8 : l * 8 - half));
#pragma unroll
    for (int i = 0; i < NA / 4; ++i) {
      const float4 c4 = __ldg(reinterpret_cast<const float4*>(t) + i);
      const float4 s4 = __ldg(reinterpret_cast<const float4*>(t + half) + i);
      co[4 * i] = c4.x, co[4 * i + 1] = c4.y, co[4 * i + 2] = c4.z, co[4 * i + 3] = c4.w;
      si[4 * i] = s4.x, si[4 * i + 1] = s4.y, si[4 * i + 2] = s4.z, si[4 * i + 3] = s4.w;
    }
  }

  for (int hb = h0; hb < h1; hb += kBatch) {
    Raw<F32> raw[kBatch];
#pragma unroll
    for (int j = 0; j < kBatch; ++j)
      if (hb + j < h1) raw[j] = load8<F32>(a.x[1 + KV], row * a.ld[1 + KV] + (hb + j) * D + l * 8);
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int h = hb + j;
      if (h >= h1) break;                         // uniform in the slot
      float v[8];
      widen<F32>(raw[j], v);
      if (!PAIRS && KV == 0 && a.rot > 0) {
        float o[8];
        widen<F32>(from_lane<F32>(mask, raw[j], partner, LPH), o);
        if (turned) {
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] = low ? turn_a(v[e], o[e], co[e % NA], si[e % NA])
                                                 : turn_b(o[e], v[e], co[e % NA], si[e % NA]);
        }
      }
      if (PAIRS && turned) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float x = v[2 * e], y = v[2 * e + 1];
          v[2 * e] = turn_a(x, y, co[e], si[e]);
          v[2 * e + 1] = turn_b(x, y, co[e], si[e]);
        }
      }
      // magnitudes compare as their bits, with a NaN above everything
      uint32_t top = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(v[e]) & 0x7FFFFFFFu);
      top = max(top, __shfl_xor_sync(mask, top, 1));
      top = max(top, __shfl_xor_sync(mask, top, 2));
      uint32_t sb = 0x7Fu, w = 0;                 // the block holds a NaN
      if (top <= 0x7F800000u) {
        sb = e4m3_scale_for(__uint_as_float(top));
        const float s = e4m3_pos(sb);
        if (s > 0.f) {
          const float r = 1.0f / s;
          const bool wide = F32 || (KV == 0 && a.rot > 0);   // more than bf16's 8 significant bits
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            if (top == 0x7F800000u) v[e] = fminf(fmaxf(v[e], -2688.f), 2688.f);
            const float q = quot(v[e], s, r);
            v[e] = wide ? off_midpoint(q, v[e], s) : q;
          }
          w = e2m1x8(v);
        }
      }
      *reinterpret_cast<uint32_t*>(a.codes[KV] + rows[KV][0] * a.codes_rb[KV] + h * (D / 2) + l * 4) = w;
      if ((l & 3) == 0) a.scales[KV][rows[KV][1] * a.scales_rb[KV] + h * (D / 32) + l / 4] = (uint8_t)sb;
      if (a.kv_out[KV]) {
        uint32_t o[4];
        dequant8(w, sb, o);
        *reinterpret_cast<uint4*>(a.kv_out[KV] + (row * a.heads[1 + KV] + h) * D + l * 8) =
            make_uint4(o[0], o[1], o[2], o[3]);
      }
    }
  }
}

template <int D, bool F32, bool PAIRS>
__global__ void __launch_bounds__(kAppendThreads, 4) kv_append_kernel(const __grid_constant__ AppendArgs a) {
  pdl_wait();      // launched while the grid before it drains
  // The chunks of a group of blocks are neighbours.  A query lane holds twice as
  // many values, so a query block covers twice as many tokens as one of keys or
  // values, and the query blocks of the grid's second half find no token left.
  const uint32_t tokens = blockIdx.x / (uint32_t)a.chunks;
  const int chunk = (int)(blockIdx.x - tokens * (uint32_t)a.chunks);
  if (chunk < a.first[1]) append_queries<D, F32, PAIRS>(a, tokens, chunk);
  else if (chunk < a.first[2]) append_rows<D, F32, PAIRS, 0>(a, tokens, chunk);
  else append_rows<D, F32, PAIRS, 1>(a, tokens, chunk);
}

template <int D, bool F32>
cudaError_t launch_append_t(const AppendArgs& a, bool pairs, unsigned grid, cudaStream_t st) {
  if (pairs) return launch_k(kv_append_kernel<D, F32, true>, dim3(grid), dim3(kAppendThreads), 0, st, false, true, a);
  return launch_k(kv_append_kernel<D, F32, false>, dim3(grid), dim3(kAppendThreads), 0, st, false, true, a);
}

int32_t page_shift(const csa2_rows& v) {
  for (int b = 6; b < 31; ++b)
    if (v.page_table && v.page_rows == 1 << b) return b;
  return -1;
}

}  // namespace

bool same_rows(const csa2_rows& x, const csa2_rows& y) {
  return x.page_table == y.page_table && x.n_rows == y.n_rows &&
         (x.page_table ? x.page_rows == y.page_rows && x.max_pages == y.max_pages : x.seq_rows == y.seq_rows);
}

cudaError_t launch_kv_append(const void* q, const void* k, const void* v, bool f32, int32_t n, int32_t Hq,
                             int64_t ld_q, int64_t ld_k, int64_t ld_v, const int32_t* seq_of_row,
                             const int32_t* row_pos, const float* cos_sin, int64_t n_pos, int32_t rot,
                             bool interleaved, const csa2_kv_cache& c, uint16_t* q_out, uint16_t* k_out,
                             uint16_t* v_out, int32_t* status, cudaStream_t st) {
  AppendArgs a{};
  a.x[0] = q, a.x[1] = k, a.x[2] = v;
  a.ld[0] = ld_q, a.ld[1] = ld_k, a.ld[2] = ld_v;
  a.heads[0] = Hq, a.heads[1] = a.heads[2] = c.Hkv;
  a.n = n;
  a.seq_of_row = seq_of_row;
  a.row_pos = row_pos;
  a.cos_sin = cos_sin;
  a.n_pos = n_pos;
  a.rot = rot;
  const csa2_rows* cd[2] = {&c.k_codes, &c.v_codes};
  const csa2_rows* sc[2] = {&c.k_scales, &c.v_scales};
  for (int i = 0; i < 2; ++i) {
    a.codes[i] = static_cast<uint8_t*>(const_cast<void*>(cd[i]->base));
    a.scales[i] = static_cast<uint8_t*>(const_cast<void*>(sc[i]->base));
    a.codes_rb[i] = cd[i]->row_bytes;
    a.scales_rb[i] = sc[i]->row_bytes;
    a.cmap[i] = to_rowmap(*cd[i]);
    a.smap[i] = to_rowmap(*sc[i]);
    a.cshift[i] = page_shift(*cd[i]);
    a.sshift[i] = page_shift(*sc[i]);
  }
  a.one_map = same_rows(c.k_codes, c.k_scales) && same_rows(c.k_codes, c.v_codes) && same_rows(c.k_codes, c.v_scales);
  a.q_out = q_out;
  a.kv_out[0] = k_out;
  a.kv_out[1] = v_out;
  a.status = status;
  // One head per slot while the launch cannot fill the device; when it can,
  // enough heads that a slot's own reading (row, page, angles) is the smaller
  // part of what it reads (2,048 tokens of 64 + 2 x 8 heads: 27.4 us with four
  // heads per slot, 26.0 us with sixteen).  Lanes are counted as for keys and
  // values, a query head's twice.
  const int lph = c.D / 8;
  const int64_t lanes = (int64_t)n * (Hq + 2 * c.Hkv) * lph, full = (int64_t)sm_count() * 2048;
  a.per = lanes <= full ? 1 : lanes <= 8 * full ? kBatch : 4 * kBatch;
  a.first[0] = 0;
  a.first[1] = (Hq + a.per - 1) / a.per;
  a.first[2] = a.first[1] + (c.Hkv + a.per - 1) / a.per;
  a.chunks = a.first[2] + (c.Hkv + a.per - 1) / a.per;
  const int64_t blocks = ((int64_t)n * lph + kAppendThreads - 1) / kAppendThreads * a.chunks;
  if (blocks > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
  const unsigned grid = (unsigned)blocks;
  if (c.D == 128)
    return f32 ? launch_append_t<128, true>(a, interleaved, grid, st) : launch_append_t<128, false>(a, interleaved, grid, st);
  return f32 ? launch_append_t<64, true>(a, interleaved, grid, st) : launch_append_t<64, false>(a, interleaved, grid, st);
}

}  // namespace csa2
