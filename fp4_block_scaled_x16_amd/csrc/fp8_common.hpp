// Device helpers of the FP8 block-128 kernels: block scales, element
// conversions, and the 128 x 128 tile in which the quantizers and the
// activation kernels encode a matrix along its rows and its columns.
//
// Formats (include/fp4.h): element = RNE(x * 2^-e) in E4M3 (E5 false, largest
// value 1.75 * 2^8) or E5M2 (E5 true, 1.75 * 2^15); block scale byte e + 127,
// e the smallest integer with largest * 2^e >= amax, at least -127.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fp4_device.hpp"
#include "fp4_internal.hpp"
#include "quant_common.hpp"

namespace fp8dev {

using fp4dev::bf16_to_f32;

__host__ __device__ __forceinline__ int64_t up16(int64_t v) { return (v + 15) & ~int64_t(15); }
__host__ __device__ __forceinline__ int64_t up128(int64_t v) { return (v + 127) & ~int64_t(127); }

// Block amaxes are carried as bits: those of a nonnegative float that is no
// NaN, which order as integers do (an integer maximum needs no
// canonicalization, and takes its DPP operand directly).
//
// amax = m * 2^k, 1 <= m < 2: e = k - 8 (E5M2: k - 15) if m <= 1.75, one
// more otherwise.  Adding 2^21 - 1 to the bits carries into the exponent
// field exactly when the mantissa exceeds 0x600000 (m > 1.75).  Subnormal
// amaxes and zero land below 0 and are clamped, which is e = -127; an
// infinite amax gives the code of the largest finite one.
template <bool E5>
__device__ __forceinline__ uint32_t scale_code(uint32_t amax) {
  const int e = static_cast<int>((amax + 0x1FFFFFu) >> 23) - (E5 ? 15 : 8);
  return static_cast<uint32_t>(e > 0 ? e : 0);
}

// The scale 2^e of a code as the converts below take it: in the exponent
// field (0 being 2^-127).
__device__ __forceinline__ float code_scale(uint32_t code) { return __uint_as_float(code << 23); }

// Four element codes in one word, byte k from y_k * 2^-e, which lies within the
// format (block scales are rounded up): gfx950's packed converts divide by
// their scale exactly.
template <bool E5>
__device__ __forceinline__ uint32_t pack4(float y0, float y1, float y2, float y3, float scale) {
  fp4dev::s16x2 w;
  w = __builtin_nondeterministic_value(w);       // both halves are written
  if constexpr (E5) {
    w = __builtin_amdgcn_cvt_scalef32_pk_bf8_f32(w, y0, y1, scale, false);
    w = __builtin_amdgcn_cvt_scalef32_pk_bf8_f32(w, y2, y3, scale, true);
  } else {
    w = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(w, y0, y1, scale, false);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(w, y2, y3, scale, true);
  }
  return __builtin_bit_cast(uint32_t, w);
}

typedef float float2v __attribute__((ext_vector_type(2)));

// The values of a word's four codes times the scale (exact).
template <bool E5>
__device__ __forceinline__ void unpack4(uint32_t w, float* v, float scale) {
  float2v lo, hi;
  if constexpr (E5) {
    lo = __builtin_amdgcn_cvt_scalef32_pk_f32_bf8(w, scale, false);
    hi = __builtin_amdgcn_cvt_scalef32_pk_f32_bf8(w, scale, true);
  } else {
    lo = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w, scale, false);
    hi = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w, scale, true);
  }
  v[0] = lo.x;
  v[1] = lo.y;
  v[2] = hi.x;
  v[3] = hi.y;
}

// fp32 -> bf16, nearest even (gfx950's packed convert); NaN stays a NaN.
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  return __builtin_bit_cast(uint32_t, bf16x2{static_cast<__bf16>(lo), static_cast<__bf16>(hi)});
}
__device__ __forceinline__ uint16_t to_bf16(float v) {
  return __builtin_bit_cast(uint16_t, static_cast<__bf16>(v));
}

// ------------------------------------------------------------ the tile ---
// A workgroup of 512 threads holds a 128 x 128 tile: thread t has rows
// 4 (t / 16) .. + 3 and columns 8 (t % 16) .. + 7, so 16 lanes cover a row's
// block (a 256-byte run of bf16, a 128-byte run of codes), a wave 16 rows,
// and the four rows of a thread are one word of a transposed code row and
// one word of KMAJOR scales.
constexpr int kTile = 128;
constexpr int kTileThreads = 512;

struct TilePos {
  int64_t r0, c0;        // first row and column of the tile
  int l, tr;             // column group (of 8) and row group (of 4) of the thread
  __device__ __forceinline__ int64_t row(int p) const { return r0 + 4 * tr + p; }
  __device__ __forceinline__ int64_t col() const { return c0 + 8 * l; }
};

// (Tiles are fewer than 2^31: each holds a 128-byte run at least, and only a
// matrix of one tile row or column as little.)
__device__ __forceinline__ TilePos tile_pos(int64_t id, int64_t tiles_c) {
  TilePos t;
  const uint32_t i = static_cast<uint32_t>(id), n = static_cast<uint32_t>(tiles_c), tr = i / n;
  t.r0 = static_cast<int64_t>(tr) * kTile;
  t.c0 = static_cast<int64_t>(i - tr * n) * kTile;
  t.l = threadIdx.x & 15;
  t.tr = threadIdx.x >> 4;
  return t;
}

// 8 bf16 of row r from column c on; zeros outside [rows, cols].  The row
// pitch is a multiple of 8 and the base 16-byte aligned, so a group with one
// valid element is an aligned 16 bytes of one allocation: it is read whole and
// what lies behind column `cols` is masked.
__device__ __forceinline__ uint4 load_bf16x8(const uint16_t* __restrict__ x, int64_t r, int64_t rows,
                                             int64_t c, int64_t cols, int64_t ld) {
  uint4 q = make_uint4(0u, 0u, 0u, 0u);
  if (r < rows && c < cols) {
    q = *reinterpret_cast<const uint4*>(x + r * ld + c);
    if (c + 8 > cols) {
      const int n = static_cast<int>(cols - c);          // 1 .. 7
      auto keep = [n](uint32_t w, int k) {
        return n >= 2 * k + 2 ? w : n == 2 * k + 1 ? w & 0xFFFFu : 0u;
      };
      q = make_uint4(keep(q.x, 0), keep(q.y, 1), keep(q.z, 2), keep(q.w, 3));
    }
  }
  return q;
}

// The thread's part of a bf16 tile; a tile inside the matrix without tests.
__device__ __forceinline__ void load_tile(uint4 (&q)[4], const uint16_t* __restrict__ x, const TilePos& t,
                                          int64_t rows, int64_t cols, int64_t ld) {
  if (t.r0 + kTile <= rows && t.c0 + kTile <= cols) {
#pragma unroll
    for (int p = 0; p < 4; ++p) q[p] = *reinterpret_cast<const uint4*>(x + t.row(p) * ld + t.col());
  } else {
#pragma unroll
    for (int p = 0; p < 4; ++p) q[p] = load_bf16x8(x, t.row(p), rows, t.col(), cols, ld);
  }
}

// 8 values as bf16 into row r, columns c ..; a partial group element by
// element.
__device__ __forceinline__ void store_bf16x8(uint16_t* __restrict__ x, int64_t r, int64_t rows,
                                             int64_t c, int64_t cols, int64_t ld,
                                             const float (&v)[8]) {
  if (r >= rows || c >= cols) return;
  uint16_t* p = x + r * ld + c;
  if (c + 8 <= cols) {
    *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]),
                                              pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
  } else {
#pragma unroll
    for (int i = 0; i < 7; ++i)
      if (c + i < cols) p[i] = to_bf16(v[i]);
  }
}

// Largest over the 16 lanes of a row's block, in every one of them: the
// rotations within a DPP row.
template <int CTRL>
__device__ __forceinline__ uint32_t dpp_max(uint32_t v) {
  const uint32_t o = __builtin_amdgcn_update_dpp(0, static_cast<int>(v), CTRL, 0xF, 0xF, true);
  return v > o ? v : o;
}
__device__ __forceinline__ uint32_t max16(uint32_t v) {
  v = dpp_max<0x128>(v);   // row_ror:8
  v = dpp_max<0x124>(v);
  v = dpp_max<0x122>(v);
  return dpp_max<0x121>(v);
}

// |v| of 8 values: starting from 0, fmaxf passes a NaN over.
__device__ __forceinline__ uint32_t absmax8(const float (&v)[8]) {
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(v[i]));
  return __float_as_uint(m);
}

__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }

// Lanes' a and b in rows of 16: [max(a0, a1), max(b0, b1), max(a2, a3), max(b2, b3)].
__device__ __forceinline__ uint32_t join_rows16(uint32_t a, uint32_t b) {
  const auto r = __builtin_amdgcn_permlane16_swap(a, b, false, false);
  return umax(r[0], r[1]);
}
// In halves of 32: [max(a0, a1), max(b0, b1)].
__device__ __forceinline__ uint32_t join_rows32(uint32_t a, uint32_t b) {
  const auto r = __builtin_amdgcn_permlane32_swap(a, b, false, false);
  return umax(r[0], r[1]);
}

// The tile's codes from code column `col` (block kb) on, as they lie in memory:
// 8 of each of the thread's rows, and the rows' scales.
struct RawCodes {
  uint2 q[4];
  uint32_t scales;
};
__device__ __forceinline__ RawCodes load_raw(const TilePos& t, const uint8_t* __restrict__ codes,
                                             const uint8_t* __restrict__ scales, int64_t rows,
                                             int64_t pitch, int64_t col, int64_t kb) {
  const int64_t rp = up16(rows);
  const uint8_t *c = codes + t.row(0) * pitch + col, *s = scales + kb * rp + t.row(0);
  RawCodes r;
  if (t.r0 + kTile <= rows) {
#pragma unroll
    for (int p = 0; p < 4; ++p) r.q[p] = *reinterpret_cast<const uint2*>(c + p * pitch);
    r.scales = *reinterpret_cast<const uint32_t*>(s);
  } else {
    // rows outside: zero codes and, their own being of any value, zero scales
    const int64_t n = rows - t.row(0);
    r = {};
#pragma unroll
    for (int p = 0; p < 4; ++p)
      if (p < n) r.q[p] = *reinterpret_cast<const uint2*>(c + p * pitch);
    if (n > 0) r.scales = *reinterpret_cast<const uint32_t*>(s) & (n < 4 ? (1u << (8 * n)) - 1u : ~0u);
  }
  return r;
}

// Row p's values.
template <bool E5>
__device__ __forceinline__ void raw_values(const RawCodes& r, int p, float (&v)[8]) {
  const float s = code_scale((r.scales >> (8 * p)) & 0xFFu);
  unpack4<E5>(r.q[p].x, v, s);
  unpack4<E5>(r.q[p].y, v + 4, s);
}

// Nonzero values that a word of four codes holds as zero.
template <typename V>
__device__ __forceinline__ uint32_t lost4(uint32_t w, const V& v) {
  uint32_t n = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) n += (v(i) != 0.0f && ((w >> (8 * i)) & 0x7Fu) == 0u) ? 1u : 0u;
  return n;
}

// Encode the thread's rows with their scale codes and store them: codes is
// the row-major code matrix of pitch cp, `col` the code column; scales the
// KMAJOR scales of block kb.
template <bool E5, bool CNT>
__device__ __forceinline__ void store_rows(const TilePos& t, const float (&v)[4][8],
                                           const uint32_t (&sc)[4], int64_t rows, int64_t cp,
                                           int64_t col, int64_t kb, uint8_t* __restrict__ codes,
                                           uint8_t* __restrict__ scales, uint32_t& lost) {
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const float s = code_scale(sc[p]);
    uint2 w;
    w.x = pack4<E5>(v[p][0], v[p][1], v[p][2], v[p][3], s);
    w.y = pack4<E5>(v[p][4], v[p][5], v[p][6], v[p][7], s);
    if constexpr (CNT) {
      lost += lost4(w.x, [&](int i) { return v[p][i]; });
      lost += lost4(w.y, [&](int i) { return v[p][4 + i]; });
    }
    if (t.row(p) < rows) *reinterpret_cast<uint2*>(codes + t.row(p) * cp + col) = w;
  }
  const int64_t rp = up16(rows);
  if (t.l == 0 && t.row(0) < rp)
    *reinterpret_cast<uint32_t*>(scales + kb * rp + t.row(0)) =
        sc[0] | (sc[1] << 8) | (sc[2] << 16) | (sc[3] << 24);
}

// Scale codes of the thread's rows in 1x128 blocks.
template <bool E5>
__device__ __forceinline__ void row_scales(const float (&v)[4][8], uint32_t (&sc)[4]) {
#pragma unroll
  for (int p = 0; p < 4; ++p) sc[p] = scale_code<E5>(max16(absmax8(v[p])));
}

// Column amaxes over the wave's 16 rows into one row of cmax[8][128] per wave:
// the exchanges between its four row groups leave two columns' maxima in a
// lane (8 l + q and 8 l + 4 + q, q = lane / 16).
typedef uint32_t ColMax[kTileThreads / 64][kTile];
__device__ __forceinline__ void col_partial(const TilePos& t, const float (&v)[4][8], ColMax& cmax) {
  uint32_t m[8];
#pragma unroll
  for (int c = 0; c < 8; ++c)
    m[c] = __float_as_uint(fmaxf(fmaxf(fmaxf(fmaxf(0.0f, fabsf(v[0][c])), fabsf(v[1][c])),
                                       fabsf(v[2][c])), fabsf(v[3][c])));
  const int q = (threadIdx.x >> 4) & 3, w = threadIdx.x >> 6;
  cmax[w][8 * t.l + q] = join_rows32(join_rows16(m[0], m[1]), join_rows16(m[2], m[3]));
  cmax[w][8 * t.l + 4 + q] = join_rows32(join_rows16(m[4], m[5]), join_rows16(m[6], m[7]));
}

// After a barrier: threads c0 .. c0 + 127 each make the scale code of one
// column; after another, a thread takes those of its 8 columns.
template <bool E5>
__device__ __forceinline__ void col_codes(const ColMax& cmax, uint8_t (&code)[kTile], int c0) {
  const int c = static_cast<int>(threadIdx.x) - c0;
  if (c >= 0 && c < kTile) {
    uint32_t m = cmax[0][c];
#pragma unroll
    for (int w = 1; w < kTileThreads / 64; ++w) m = umax(m, cmax[w][c]);
    code[c] = static_cast<uint8_t>(scale_code<E5>(m));
  }
}

// Transposed code tile in LDS: 128 columns of 128 bytes.  Column c's word of
// rows 4q .. 4q + 3 lies in row c ^ (c / 64), 16-byte chunk (q / 4) ^ (c / 8 % 8):
// the words that a wave writes at once (16 columns 8 apart, 4 row groups of one
// chunk) are spread over all 64 words of a row pair, and a thread reads 16
// bytes.  Half a wave still meets two to a bank of 32; a layout without that
// measured the same times, the memory traffic being the bound.
constexpr int kTileWords = kTile * kTile / 4;
__device__ __forceinline__ int tile_chunk(int c, int ch) {
  return (c ^ (c >> 6)) * 8 + (ch ^ ((c >> 3) & 7));
}

// Encode the thread's columns with their scale codes (byte c of sc: column c)
// into the LDS tile.
template <bool E5, bool CNT>
__device__ __forceinline__ void encode_cols(const TilePos& t, const float (&v)[4][8], const uint2& sc,
                                            uint32_t* tile, uint32_t& lost) {
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    const float s = code_scale(((c < 4 ? sc.x : sc.y) >> (8 * (c & 3))) & 0xFFu);
    const uint32_t w = pack4<E5>(v[0][c], v[1][c], v[2][c], v[3][c], s);
    if constexpr (CNT) lost += lost4(w, [&](int i) { return v[i][c]; });
    tile[tile_chunk(8 * t.l + c, t.tr >> 2) * 4 + (t.tr & 3)] = w;
  }
}

// The LDS tile to rows col0 .. of the transpose's code matrix (pitch rp, a
// multiple of 128): 8 lanes write a row's 128 bytes.  `n`: columns of the
// tile inside the matrix.
__device__ __forceinline__ void store_cols(const TilePos& t, const uint32_t* tile, int64_t n,
                                           int64_t col0, int64_t rp, uint8_t* __restrict__ codes_t) {
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int q = threadIdx.x + k * kTileThreads;
    const int c = q >> 3, ch = q & 7;
    if (c < n)
      *reinterpret_cast<uint4*>(codes_t + (col0 + c) * rp + t.r0 + 16 * ch) =
          reinterpret_cast<const uint4*>(tile)[tile_chunk(c, ch)];
  }
}

// Workgroups for `tiles` tiles, at most per_cu per CU.
inline int tile_grid(int64_t tiles, int per_cu) {
  const int64_t cap = fp4lib::grid_cap(per_cu);
  return static_cast<int>(tiles < cap ? tiles : cap);
}

}  // namespace fp8dev
