// FP8 block-128 quantization: bf16 -> E4M3 / E5M2 codes with one power-of-two
// scale per 1x128 or 128x128 block, along the rows, along the columns (the
// transpose's code matrix) or both from one read; their values; and the
// re-encoding of row codes along the columns.
//
// All are bound by HBM: a quantizer reads 2 bytes per element and writes 1
// (+ 1/128) per orientation, a re-encoding reads 1 and writes 1.  One
// 128 x 128 tile per workgroup step: a block of either orientation lies in
// one tile, so every scale is known after one read, and the tile is the unit
// of the transposition through LDS (fp8_common.hpp).
//
// Measured: 8192 x 4096 along rows or columns 16.4 us (6.2 TB/s, part of it in
// the last-level cache), both 24.2 (5.5), 12288 x 4608 in 2D both ways 40.4
// (5.6), codes along the columns 8192 x 4096 12.3 (5.5); a large copy reaches 5.16.
#include "fp8_common.hpp"

using namespace fp8dev;
using fp4quant::flush_counters;
using fp4quant::unpack8;

namespace {

constexpr int kWgPerCu = 4;

// Two workgroups per CU (128 registers a thread), so that one's loads are
// under way while the other waits at a barrier.
template <bool E5, bool ROW, bool COL, bool TWO_D, bool CNT>
__global__ __launch_bounds__(kTileThreads, 4) void k_quant_fp8(fp4lib::Fp8QuantArgs a) {
  __shared__ ColMax cmax;
  __shared__ __attribute__((aligned(16))) uint8_t code[kTile];
  __shared__ __attribute__((aligned(16))) uint32_t tile[COL ? kTileWords : 4];
  const int64_t tiles_c = (a.cols + kTile - 1) / kTile;
  const int64_t n = (a.rows + kTile - 1) / kTile * tiles_c;
  uint32_t lost = 0;
  for (int64_t id = blockIdx.x; id < n; id += gridDim.x) {
    const TilePos t = tile_pos(id, tiles_c);
    float v[4][8];
    {
      uint4 q[4];
      load_tile(q, a.x, t, a.rows, a.cols, a.ld);
#pragma unroll
      for (int p = 0; p < 4; ++p) unpack8(q[p], v[p]);
    }
    uint32_t sr[4];
    uint2 sc;
    if constexpr (TWO_D) {
      // one amax per tile: each wave's into LDS, the largest of the 8 in every thread
      uint32_t m = max16(umax(umax(absmax8(v[0]), absmax8(v[1])), umax(absmax8(v[2]), absmax8(v[3]))));
      m = join_rows16(m, m);
      m = join_rows32(m, m);
      uint32_t* part = cmax[0] + 8 * ((id / gridDim.x) & 1);   // two sets: the next tile's is another
      part[threadIdx.x >> 6] = m;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < kTileThreads / 64; ++w) m = umax(m, part[w]);
      const uint32_t s = scale_code<E5>(m);
#pragma unroll
      for (int p = 0; p < 4; ++p) sr[p] = s;
      sc.x = sc.y = s * 0x01010101u;
    } else if constexpr (COL) {
      col_partial(t, v, cmax);
      __syncthreads();
      col_codes<E5>(cmax, code, 0);
      __syncthreads();
      sc = *reinterpret_cast<const uint2*>(code + 8 * t.l);
    }
    if constexpr (ROW) {
      if constexpr (!TWO_D) row_scales<E5>(v, sr);
      store_rows<E5, CNT>(t, v, sr, a.rows, up128(a.cols), t.col(), t.c0 / kTile, a.codes, a.scales,
                          lost);
    }
    if constexpr (COL) {
      const int64_t sp = up16(a.cols);
      if (t.tr == 0 && t.col() < sp)
        *reinterpret_cast<uint2*>(a.scales_t + t.r0 / kTile * sp + t.col()) = sc;
      encode_cols<E5, CNT>(t, v, sc, tile, lost);
      __syncthreads();
      // the next tile's first barrier separates these reads from its writes
      store_cols(t, tile, a.cols - t.c0, t.c0, up128(a.rows), a.codes_t);
    }
  }
  if constexpr (CNT) {
    uint32_t cnt[5] = {0, 0, 0, 0, lost};
    flush_counters<kTileThreads>(cnt, a.counters);
  }
}

// The columns of row codes: values code * 2^e (exact in fp32), encoded anew
// in blocks along the rows.
template <bool E5>
__global__ __launch_bounds__(kTileThreads, 4) void k_requant_t_fp8(
    const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales, int64_t rows,
    int64_t cols, uint8_t* __restrict__ codes_t, uint8_t* __restrict__ scales_t) {
  __shared__ ColMax cmax;
  __shared__ __attribute__((aligned(16))) uint8_t code[kTile];
  __shared__ __attribute__((aligned(16))) uint32_t tile[kTileWords];
  const int64_t tiles_c = (cols + kTile - 1) / kTile;
  const int64_t n = (rows + kTile - 1) / kTile * tiles_c;
  uint32_t unused = 0;
  for (int64_t id = blockIdx.x; id < n; id += gridDim.x) {
    const TilePos t = tile_pos(id, tiles_c);
    float v[4][8];
    const RawCodes raw = load_raw(t, codes, scales, rows, up128(cols), t.col(), t.c0 / kTile);
#pragma unroll
    for (int p = 0; p < 4; ++p) raw_values<E5>(raw, p, v[p]);
    col_partial(t, v, cmax);
    __syncthreads();
    col_codes<E5>(cmax, code, 0);
    __syncthreads();
    const uint2 sc = *reinterpret_cast<const uint2*>(code + 8 * t.l);
    const int64_t sp = up16(cols);
    if (t.tr == 0 && t.col() < sp)
      *reinterpret_cast<uint2*>(scales_t + t.r0 / kTile * sp + t.col()) = sc;
    encode_cols<E5, false>(t, v, sc, tile, unused);
    __syncthreads();
    store_cols(t, tile, cols - t.c0, t.c0, up128(rows), codes_t);
  }
}

// One thread per 8 codes of a row.
template <bool E5, bool F32>
__global__ __launch_bounds__(256) void k_dequant_fp8(const uint8_t* __restrict__ codes,
                                                     const uint8_t* __restrict__ scales,
                                                     int64_t rows, int64_t cols,
                                                     void* __restrict__ out) {
  const uint64_t per_row = static_cast<uint64_t>((cols + 7) >> 3);
  const uint64_t n = static_cast<uint64_t>(rows) * per_row;
  const int64_t cp = up128(cols), rp = up16(rows);
  const bool whole = (cols & 7) == 0;
  for (uint64_t i = static_cast<uint64_t>(blockIdx.x) * 256 + threadIdx.x; i < n;
       i += static_cast<uint64_t>(gridDim.x) * 256) {
    const int64_t r = static_cast<int64_t>(i / per_row);
    const int64_t c = static_cast<int64_t>(i - r * per_row) * 8;
    const uint2 q = *reinterpret_cast<const uint2*>(codes + r * cp + c);
    const float s = code_scale(scales[(c >> 7) * rp + r]);
    float v[8];
    unpack4<E5>(q.x, v, s);
    unpack4<E5>(q.y, v + 4, s);
    if constexpr (F32) {
      float* d = static_cast<float*>(out) + r * cols + c;
      if (whole) {
        reinterpret_cast<float4*>(d)[0] = make_float4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<float4*>(d)[1] = make_float4(v[4], v[5], v[6], v[7]);
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (c + k < cols) d[k] = v[k];
      }
    } else if (whole) {
      store_bf16x8(static_cast<uint16_t*>(out), r, rows, c, cols, cols, v);
    } else {
      uint16_t* d = static_cast<uint16_t*>(out) + r * cols + c;
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (c + k < cols) d[k] = to_bf16(v[k]);
    }
  }
}

template <bool E5, bool CNT>
void launch_quant(const fp4lib::Fp8QuantArgs& a, hipStream_t s) {
  const int64_t tiles = (a.rows + kTile - 1) / kTile * ((a.cols + kTile - 1) / kTile);
  const dim3 grid(tile_grid(tiles, kWgPerCu)), block(kTileThreads);
  const bool row = a.codes, col = a.codes_t;
  if (a.block2d) {
    if (row && col) hipLaunchKernelGGL((k_quant_fp8<E5, true, true, true, CNT>), grid, block, 0, s, a);
    else if (row) hipLaunchKernelGGL((k_quant_fp8<E5, true, false, true, CNT>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((k_quant_fp8<E5, false, true, true, CNT>), grid, block, 0, s, a);
  } else {
    if (row && col) hipLaunchKernelGGL((k_quant_fp8<E5, true, true, false, CNT>), grid, block, 0, s, a);
    else if (row) hipLaunchKernelGGL((k_quant_fp8<E5, true, false, false, CNT>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((k_quant_fp8<E5, false, true, false, CNT>), grid, block, 0, s, a);
  }
}

}  // namespace

namespace fp4lib {

hipError_t launch_quant_fp8(const Fp8QuantArgs& a, hipStream_t s) {
  if (a.e5m2) {
    if (a.counters) launch_quant<true, true>(a, s);
    else launch_quant<true, false>(a, s);
  } else {
    if (a.counters) launch_quant<false, true>(a, s);
    else launch_quant<false, false>(a, s);
  }
  return hipGetLastError();
}

hipError_t launch_requant_t_fp8(int e5m2, const uint8_t* codes, const uint8_t* scales, int64_t rows,
                                int64_t cols, uint8_t* codes_t, uint8_t* scales_t, hipStream_t s) {
  const int64_t tiles = (rows + kTile - 1) / kTile * ((cols + kTile - 1) / kTile);
  const dim3 grid(tile_grid(tiles, kWgPerCu)), block(kTileThreads);
  if (e5m2)
    hipLaunchKernelGGL(k_requant_t_fp8<true>, grid, block, 0, s, codes, scales, rows, cols, codes_t,
                       scales_t);
  else
    hipLaunchKernelGGL(k_requant_t_fp8<false>, grid, block, 0, s, codes, scales, rows, cols, codes_t,
                       scales_t);
  return hipGetLastError();
}

hipError_t launch_dequant_fp8(int e5m2, const uint8_t* codes, const uint8_t* scales, int64_t rows,
                              int64_t cols, void* out, int out_fp32, hipStream_t s) {
  const uint64_t n = static_cast<uint64_t>(rows) * static_cast<uint64_t>((cols + 7) >> 3);
  const dim3 grid(fp4quant::grid_for(n, 8, 256)), block(256);
  auto* k = e5m2 ? (out_fp32 ? k_dequant_fp8<true, true> : k_dequant_fp8<true, false>)
                 : (out_fp32 ? k_dequant_fp8<false, true> : k_dequant_fp8<false, false>);
  hipLaunchKernelGGL(k, grid, block, 0, s, codes, scales, rows, cols, out);
  return hipGetLastError();
}

}  // namespace fp4lib
