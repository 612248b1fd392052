// The activation of a feed-forward layer between its two 8-bit linears, and
// its backward pass from an 8-bit checkpoint of its input (include/fp4.h):
//
//   k_act_fp8       h (bf16) -> codes of a = act(h) and of h, along the rows
//   k_act_grad_fp8  codes of h, da (bf16) -> codes of dh along rows and
//                   columns, codes of a along the columns (or bf16 values)
//
// Both are bound by HBM: per element of a, SwiGLU forward reads 4 bytes and
// writes 3, backward reads 4 and writes 5; in values instead of codes the two
// linears' quantizers would read and write another 16.  The 128 x 128 tile of
// fp8_common.hpp, on the halves of h at once.
//
// sigmoid is 1 / (1 + 2^(-g log2 e)) on the hardware exp2 and reciprocal (1 ulp
// each; the argument's rounding makes |g| 2^-24 of relative error in the
// exponential, which counts where the exponential dominates): far below half
// a step of the 8-bit and bf16 results.
#include "fp8_common.hpp"

using namespace fp8dev;
using fp4quant::unpack8;

namespace {

constexpr int kWgPerCu = 4;

__device__ __forceinline__ float sigmoid(float g) {
  const float t = __builtin_amdgcn_exp2f(-1.44269504088896341f * g);
  return __builtin_amdgcn_rcpf(1.0f + t);      // t = inf: 0
}

template <bool GLU>
__global__ __launch_bounds__(kTileThreads) void k_act_fp8(fp4lib::Fp8ActArgs a) {
  const int64_t tiles_c = (a.cols + kTile - 1) / kTile;
  const int64_t n = (a.rows + kTile - 1) / kTile * tiles_c;
  const int64_t fp = up128(a.cols);
  uint32_t unused = 0;
  for (int64_t id = blockIdx.x; id < n; id += gridDim.x) {
    const TilePos t = tile_pos(id, tiles_c);
    float g[4][8], u[4][8], v[4][8];
    {
      uint4 q[4], w[4];
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        q[p] = load_bf16x8(a.h, t.row(p), a.rows, t.col(), a.cols, a.ld);
        if constexpr (GLU)
          w[p] = load_bf16x8(a.h + a.cols, t.row(p), a.rows, t.col(), a.cols, a.ld);
      }
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        unpack8(q[p], g[p]);
        if constexpr (GLU) unpack8(w[p], u[p]);
      }
    }
#pragma unroll
    for (int p = 0; p < 4; ++p)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if constexpr (GLU) {
          v[p][i] = g[p][i] * sigmoid(g[p][i]) * u[p][i];
        } else {
          const float r = g[p][i] < 0.0f ? 0.0f : g[p][i];     // keeps a NaN
          v[p][i] = r * r;
        }
      }
    uint32_t sc[4];
    const int64_t kb = t.c0 / kTile;
    if (a.a_codes) {
      row_scales<false>(v, sc);
      store_rows<false, false>(t, v, sc, a.rows, fp, t.col(), kb, a.a_codes, a.a_scales, unused);
    }
    if (a.a) {
#pragma unroll
      for (int p = 0; p < 4; ++p) store_bf16x8(a.a, t.row(p), a.rows, t.col(), a.cols, a.ld_a, v[p]);
    }
    if (a.h_codes) {
      const int64_t hp = GLU ? 2 * fp : fp;
      row_scales<false>(g, sc);
      store_rows<false, false>(t, g, sc, a.rows, hp, t.col(), kb, a.h_codes, a.h_scales, unused);
      if constexpr (GLU) {
        row_scales<false>(u, sc);
        store_rows<false, false>(t, u, sc, a.rows, hp, fp + t.col(), fp / kTile + kb, a.h_codes,
                                 a.h_scales, unused);
      }
    }
  }
}

// The values of the tile's codes from code column `col` (block kb) on.
__device__ __forceinline__ void load_codes(const TilePos& t, const uint8_t* __restrict__ codes,
                                           const uint8_t* __restrict__ scales, int64_t rows,
                                           int64_t hp, int64_t col, int64_t kb, float (&v)[4][8]) {
  const int64_t rp = up16(rows);
  uint2 q[4] = {};
  uint32_t se = 0;
#pragma unroll
  for (int p = 0; p < 4; ++p)
    if (t.row(p) < rows) q[p] = *reinterpret_cast<const uint2*>(codes + t.row(p) * hp + col);
  if (t.row(0) < rp) se = *reinterpret_cast<const uint32_t*>(scales + kb * rp + t.row(0));
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const float s = t.row(p) < rows ? fp4dev::ue8m0_decode((se >> (8 * p)) & 0xFFu) : 0.0f;
    unpack4<false>(q[p].x, v[p]);
    unpack4<false>(q[p].y, v[p] + 4);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[p][i] *= s;
  }
}

template <bool GLU, bool E5>
__global__ __launch_bounds__(kTileThreads) void k_act_grad_fp8(fp4lib::Fp8ActGradArgs a) {
  constexpr int H = GLU ? 2 : 1;          // halves of h
  __shared__ __attribute__((aligned(16))) float cmax[H + 1][kTileThreads / 64][kTile];
  __shared__ __attribute__((aligned(16))) uint32_t tile[H + 1][kTileWords];
  const int64_t tiles_c = (a.cols + kTile - 1) / kTile;
  const int64_t n = (a.rows + kTile - 1) / kTile * tiles_c;
  const int64_t fp = up128(a.cols), hp = H * fp, rp = up128(a.rows);
  uint32_t unused = 0;
  for (int64_t id = blockIdx.x; id < n; id += gridDim.x) {
    const TilePos t = tile_pos(id, tiles_c);
    const int64_t kb = t.c0 / kTile, cols_in = a.cols - t.c0;
    float d[H][4][8], v[4][8];            // dh, a
    {
      uint4 q[4];
#pragma unroll
      for (int p = 0; p < 4; ++p) q[p] = load_bf16x8(a.da, t.row(p), a.rows, t.col(), a.cols, a.ld);
      load_codes(t, a.h_codes, a.h_scales, a.rows, hp, t.col(), kb, d[0]);
      if constexpr (GLU)
        load_codes(t, a.h_codes, a.h_scales, a.rows, hp, fp + t.col(), fp / kTile + kb, d[1]);
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        float da[8];
        unpack8(q[p], da);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float g = d[0][p][i];
          if constexpr (GLU) {
            const float u = d[1][p][i], s = sigmoid(g), silu = g * s;
            v[p][i] = silu * u;
            d[0][p][i] = da[i] * u * (s * (1.0f + g * (1.0f - s)));
            d[1][p][i] = da[i] * silu;
          } else {
            const float r = g < 0.0f ? 0.0f : g;
            v[p][i] = r * r;
            d[0][p][i] = da[i] * (2.0f * r);
          }
        }
      }
    }
#pragma unroll
    for (int h = 0; h < H; ++h) {
      if (a.dh_codes) {
        uint32_t sc[4];
        row_scales<E5>(d[h], sc);
        store_rows<E5, false>(t, d[h], sc, a.rows, hp, h * fp + t.col(), h * (fp / kTile) + kb,
                              a.dh_codes, a.dh_scales, unused);
      }
      if (a.dh) {
#pragma unroll
        for (int p = 0; p < 4; ++p)
          store_bf16x8(a.dh + h * a.cols, t.row(p), a.rows, t.col(), a.cols, a.ld_dh, d[h][p]);
      }
    }
    if (a.a) {
#pragma unroll
      for (int p = 0; p < 4; ++p) store_bf16x8(a.a, t.row(p), a.rows, t.col(), a.cols, a.ld_a, v[p]);
    }
    if (a.dh_t_codes || a.a_t_codes) {
#pragma unroll
      for (int h = 0; h < H; ++h) col_partial(t, d[h], cmax[h]);
      col_partial(t, v, cmax[H]);
      __syncthreads();
      if (a.dh_t_codes) {
#pragma unroll
        for (int h = 0; h < H; ++h) {
          float m[8];
          uint32_t sc[8];
          col_max(t, cmax[h], m);
#pragma unroll
          for (int c = 0; c < 8; ++c) sc[c] = scale_code<E5>(m[c]);
          // row h * cols + column of the transpose (SwiGLU: cols is a multiple
          // of 8 and 2 cols one of 16, so there is no padding)
          if (t.tr == 0 && t.col() < (GLU ? a.cols : up16(a.cols)))
            store_scales8(sc, a.dh_t_scales + t.r0 / kTile * up16(H * a.cols) + h * a.cols + t.col());
          encode_cols<E5, false>(t, d[h], sc, tile[h], unused);
        }
      }
      if (a.a_t_codes) {
        float m[8];
        uint32_t sc[8];
        col_max(t, cmax[H], m);
#pragma unroll
        for (int c = 0; c < 8; ++c) sc[c] = scale_code<false>(m[c]);
        if (t.tr == 0 && t.col() < up16(a.cols))
          store_scales8(sc, a.a_t_scales + t.r0 / kTile * up16(a.cols) + t.col());
        encode_cols<false, false>(t, v, sc, tile[H], unused);
      }
      __syncthreads();
      if (a.dh_t_codes) {
#pragma unroll
        for (int h = 0; h < H; ++h)
          store_cols(t, tile[h], cols_in, h * a.cols + t.c0, rp, a.dh_t_codes);
      }
      if (a.a_t_codes) store_cols(t, tile[H], cols_in, t.c0, rp, a.a_t_codes);
    }
  }
}

}  // namespace

namespace fp4lib {

hipError_t launch_act_quant_fp8(const Fp8ActArgs& a, hipStream_t s) {
  const int64_t tiles = (a.rows + kTile - 1) / kTile * ((a.cols + kTile - 1) / kTile);
  const dim3 grid(tile_grid(tiles, kWgPerCu)), block(kTileThreads);
  if (a.act == FP4_ACT_SWIGLU) hipLaunchKernelGGL(k_act_fp8<true>, grid, block, 0, s, a);
  else hipLaunchKernelGGL(k_act_fp8<false>, grid, block, 0, s, a);
  return hipGetLastError();
}

hipError_t launch_act_grad_fp8(const Fp8ActGradArgs& a, hipStream_t s) {
  const int64_t tiles = (a.rows + kTile - 1) / kTile * ((a.cols + kTile - 1) / kTile);
  const dim3 grid(tile_grid(tiles, kWgPerCu)), block(kTileThreads);
  const bool glu = a.act == FP4_ACT_SWIGLU;
  if (glu && a.e5m2) hipLaunchKernelGGL((k_act_grad_fp8<true, true>), grid, block, 0, s, a);
  else if (glu) hipLaunchKernelGGL((k_act_grad_fp8<true, false>), grid, block, 0, s, a);
  else if (a.e5m2) hipLaunchKernelGGL((k_act_grad_fp8<false, true>), grid, block, 0, s, a);
  else hipLaunchKernelGGL((k_act_grad_fp8<false, false>), grid, block, 0, s, a);
  return hipGetLastError();
}

}  // namespace fp4lib
