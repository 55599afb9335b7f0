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
// of a position is read once per slot.  A slot of D / 8 lanes owns one head
// at a time, eight values (16 bytes of bf16) per lane: loads and stores are
// coalesced, a block's maximum is two shuffles, and the rotation partner of
// the half-split layout is one shuffle away.  A slot walks up to `per` heads
// of its token with the angles in registers, kBatch heads' loads in flight.
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
  int32_t chunks;             // chunks of one token
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
  int32_t one_map;            // all four planes place rows alike
  uint16_t* q_out;            // [n][Hq][D]
  uint16_t* kv_out[2];        // [n][Hkv][D] or nullptr
  int32_t* status;
};

// The row of (seq, pos), refusing a position outside the sequence's own
// share of a contiguous plane.
__device__ __forceinline__ int64_t write_row(const RowMap& m, int32_t seq, int32_t pos) {
  if (seq < 0 || (!m.page_table && m.seq_rows > 0 && pos >= m.seq_rows)) return -1;
  return map_row(m, seq, pos);
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

template <int D, bool F32, bool PAIRS>
__global__ void __launch_bounds__(kAppendThreads) kv_append_kernel(const __grid_constant__ AppendArgs a) {
  constexpr int LPH = D / 8;                      // lanes per head
  const int64_t slot = ((int64_t)blockIdx.x * kAppendThreads + threadIdx.x) / LPH;
  const int l = threadIdx.x % LPH, lane = threadIdx.x & 31;
  const uint32_t mask = (LPH == 32 ? 0xffffffffu : ((1u << LPH) - 1u)) << (lane / LPH * LPH);
  const int64_t row = slot / a.chunks;
  if (row >= a.n) return;
  const int ch = (int)(slot % a.chunks);
  const int kind = ch >= a.first[2] ? 2 : (ch >= a.first[1] ? 1 : 0);   // query, key, value
  const int h0 = (ch - a.first[kind]) * a.per;
  const int h1 = min(h0 + a.per, a.heads[kind]);

  const int32_t pos = __ldg(a.row_pos + row);
  if (pos < 0) return;                            // a padding row
  const int32_t seq = a.seq_of_row ? __ldg(a.seq_of_row + row) : (int32_t)row;
  // a token is stored whole or not at all
  int64_t rows[2][2];                             // [K, V][codes, scales]
  bool ok = !(a.rot > 0 && pos >= a.n_pos);
  rows[0][0] = write_row(a.cmap[0], seq, pos);
  rows[0][1] = a.one_map ? rows[0][0] : write_row(a.smap[0], seq, pos);
  rows[1][0] = a.one_map ? rows[0][0] : write_row(a.cmap[1], seq, pos);
  rows[1][1] = a.one_map ? rows[0][0] : write_row(a.smap[1], seq, pos);
  ok = ok && rows[0][0] >= 0 && rows[0][1] >= 0 && rows[1][0] >= 0 && rows[1][1] >= 0;
  if (!ok) {
    if (l == 0) record_error(a.status, CSA2_ERR_INDEX_RANGE);
    return;
  }

  // this lane's angles: eight of the half-split layout (values l*8..l*8+7 are
  // one side of eight pairs), four of the interleaved one
  const int half = a.rot / 2;
  const bool turned = kind < 2 && l * 8 < a.rot;
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
      if (hb + j < h1) raw[j] = load8<F32>(a.x[kind], row * a.ld[kind] + (int64_t)(hb + j) * D + l * 8);
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int h = hb + j;
      if (h >= h1) break;                         // uniform in the slot
      float v[8];
      widen<F32>(raw[j], v);
      if (!PAIRS && kind < 2 && a.rot > 0) {
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
      if (kind == 0) {
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * e], v[2 * e + 1]);
          w[e] = *reinterpret_cast<const uint32_t*>(&b);
        }
        *reinterpret_cast<uint4*>(a.q_out + (row * a.heads[0] + h) * D + l * 8) = make_uint4(w[0], w[1], w[2], w[3]);
        continue;
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
          const bool wide = F32 || (kind == 1 && a.rot > 0);   // more than bf16's 8 significant bits
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            if (top == 0x7F800000u) v[e] = fminf(fmaxf(v[e], -2688.f), 2688.f);
            const float q = quot(v[e], s, r);
            v[e] = wide ? off_midpoint(q, v[e], s) : q;
          }
          w = e2m1x8(v);
        }
      }
      const int kv = kind - 1;
      *reinterpret_cast<uint32_t*>(a.codes[kv] + rows[kv][0] * a.codes_rb[kv] + h * (D / 2) + l * 4) = w;
      if ((l & 3) == 0) a.scales[kv][rows[kv][1] * a.scales_rb[kv] + h * (D / 32) + l / 4] = (uint8_t)sb;
      if (a.kv_out[kv]) {
        uint32_t o[4];
        dequant8(w, sb, o);
        *reinterpret_cast<uint4*>(a.kv_out[kv] + (row * a.heads[kind] + h) * D + l * 8) =
            make_uint4(o[0], o[1], o[2], o[3]);
      }
    }
  }
}

template <int D, bool F32>
void launch_append_t(const AppendArgs& a, bool pairs, unsigned grid, cudaStream_t st) {
  if (pairs) kv_append_kernel<D, F32, true><<<grid, kAppendThreads, 0, st>>>(a);
  else kv_append_kernel<D, F32, false><<<grid, kAppendThreads, 0, st>>>(a);
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
  }
  a.one_map = same_rows(c.k_codes, c.k_scales) && same_rows(c.k_codes, c.v_codes) && same_rows(c.k_codes, c.v_scales);
  a.q_out = q_out;
  a.kv_out[0] = k_out;
  a.kv_out[1] = v_out;
  a.status = status;
  // One head per slot while the launch cannot fill the device, four when it can.
  const int lph = c.D / 8;
  const int64_t heads = (int64_t)n * (Hq + 2 * c.Hkv);
  a.per = heads * lph <= (int64_t)sm_count() * 2048 ? 1 : kBatch;
  a.first[0] = 0;
  a.first[1] = (Hq + a.per - 1) / a.per;
  a.first[2] = a.first[1] + (c.Hkv + a.per - 1) / a.per;
  a.chunks = a.first[2] + (c.Hkv + a.per - 1) / a.per;
  const int64_t grid = ((int64_t)n * a.chunks * lph + kAppendThreads - 1) / kAppendThreads;
  if (grid > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
  if (c.D == 128) {
    if (f32) launch_append_t<128, true>(a, interleaved, (unsigned)grid, st);
    else launch_append_t<128, false>(a, interleaved, (unsigned)grid, st);
  } else {
    if (f32) launch_append_t<64, true>(a, interleaved, (unsigned)grid, st);
    else launch_append_t<64, false>(a, interleaved, (unsigned)grid, st);
  }
  return cudaGetLastError();
}

}  // namespace csa2
