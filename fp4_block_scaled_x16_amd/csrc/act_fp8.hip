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
// fp8_common.hpp, on the halves of h at once.  SwiGLU at 8192 x 6144: 71 us (5.0
// TB/s) forward, 95 (4.8) backward.
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

// The same bits, of which the compiler knows nothing (it would keep what it
// has unpacked from them).
__device__ __forceinline__ uint4 reread(uint4 q) {
  asm volatile("" : "+v"(q.x), "+v"(q.y), "+v"(q.z), "+v"(q.w));
  return q;
}

template <bool GLU>
__global__ __launch_bounds__(kTileThreads, 4) void k_act_fp8(fp4lib::Fp8ActArgs a) {
  const int64_t tiles_c = (a.cols + kTile - 1) / kTile;
  const int64_t n = (a.rows + kTile - 1) / kTile * tiles_c;
  const int64_t fp = up128(a.cols);
  uint32_t unused = 0;
  for (int64_t id = blockIdx.x; id < n; id += gridDim.x) {
    const TilePos t = tile_pos(id, tiles_c);
    // h stays as it was read, and is unpacked again for its own codes: with three
    // fp32 tiles in 128 registers it spills (8192 x 6144: 71.3 us, 72; three
    // workgroups per CU in 80 registers: 101)
    uint4 q[4], w[4];
    load_tile(q, a.h, t, a.rows, a.cols, a.ld);
    if constexpr (GLU) load_tile(w, a.h + a.cols, t, a.rows, a.cols, a.ld);
    float v[4][8];
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      float g[8], u[8];
      unpack8(q[p], g);
      if constexpr (GLU) unpack8(w[p], u);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if constexpr (GLU) {
          v[p][i] = g[i] * sigmoid(g[i]) * u[i];
        } else {
          const float r = g[i] < 0.0f ? 0.0f : g[i];     // keeps a NaN
          v[p][i] = r * r;
        }
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
#pragma unroll
      for (int p = 0; p < 4; ++p) unpack8(reread(q[p]), v[p]);
      row_scales<false>(v, sc);
      store_rows<false, false>(t, v, sc, a.rows, hp, t.col(), kb, a.h_codes, a.h_scales, unused);
      if constexpr (GLU) {
#pragma unroll
        for (int p = 0; p < 4; ++p) unpack8(reread(w[p]), v[p]);
        row_scales<false>(v, sc);
        store_rows<false, false>(t, v, sc, a.rows, hp, fp + t.col(), fp / kTile + kb, a.h_codes,
                                 a.h_scales, unused);
      }
    }
  }
}

// What a tile of the backward pass reads.
template <bool GLU>
struct GradInput {
  RawCodes h[GLU ? 2 : 1];
  uint4 da[4];
};
template <bool GLU>
__device__ __forceinline__ GradInput<GLU> load_grad(const fp4lib::Fp8ActGradArgs& a, const TilePos& t) {
  const int64_t fp = up128(a.cols), hp = (GLU ? 2 : 1) * fp, kb = t.c0 / kTile;
  GradInput<GLU> in;
  load_tile(in.da, a.da, t, a.rows, a.cols, a.ld);
  in.h[0] = load_raw(t, a.h_codes, a.h_scales, a.rows, hp, t.col(), kb);
  if constexpr (GLU) in.h[1] = load_raw(t, a.h_codes, a.h_scales, a.rows, hp, fp + t.col(), fp / kTile + kb);
  return in;
}

// VALUES: bf16 dh and a; else codes.
//
// SwiGLU to codes holds three fp32 tiles, 96 registers a thread and as many
// again around them: one workgroup fits on a CU, so it loops over tiles and
// loads the next one's input before it computes (8192 x 6144: 95 us, 4.8 TB/s;
// two workgroups of 128 registers spill: 217 us).  The others fit twice, and
// overlap each other better than a loop does (squared ReLU, 8192 x 21504: 216
// us, 4.9 TB/s; the loop took a tenth more).
template <bool GLU, bool VALUES>
constexpr bool kGradLoop = GLU && !VALUES;

template <bool GLU, bool E5, bool VALUES>
__global__ __launch_bounds__(kTileThreads, (kGradLoop<GLU, VALUES> ? 2 : 4)) void k_act_grad_fp8(fp4lib::Fp8ActGradArgs a) {
  constexpr int H = GLU ? 2 : 1;          // halves of h
  __shared__ ColMax cmax[VALUES ? 1 : H + 1];
  __shared__ __attribute__((aligned(16))) uint8_t code[H + 1][kTile];
  __shared__ __attribute__((aligned(16))) uint32_t tile[VALUES ? 1 : H + 1][VALUES ? 4 : kTileWords];
  const int64_t tiles_c = (a.cols + kTile - 1) / kTile;
  const int64_t n = (a.rows + kTile - 1) / kTile * tiles_c;
  const int64_t fp = up128(a.cols), hp = H * fp, rp = up128(a.rows);
  uint32_t unused = 0;
  constexpr bool LOOP = kGradLoop<GLU, VALUES>;
  GradInput<GLU> next;
  if (LOOP && blockIdx.x < n) next = load_grad<GLU>(a, tile_pos(blockIdx.x, tiles_c));
  for (int64_t id = blockIdx.x; id < n; id += gridDim.x) {
    const TilePos t = tile_pos(id, tiles_c);
    const int64_t kb = t.c0 / kTile, cols_in = a.cols - t.c0;
    float d[H][4][8], v[4][8];            // dh, a
    {
      const GradInput<GLU> in = LOOP ? next : load_grad<GLU>(a, t);
      if (LOOP && id + gridDim.x < n) next = load_grad<GLU>(a, tile_pos(id + gridDim.x, tiles_c));
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        float da[8];
        unpack8(in.da[p], da);
#pragma unroll
        for (int h = 0; h < H; ++h) raw_values<false>(in.h[h], p, d[h][p]);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float g = d[0][p][i];
          if constexpr (GLU) {
            const float u = d[1][p][i], s = sigmoid(g), silu = g * s;
            v[p][i] = silu * u;
            d[0][p][i] = da[i] * u * __builtin_fmaf(silu, 1.0f - s, s);
            d[1][p][i] = da[i] * silu;
          } else {
            const float r = g < 0.0f ? 0.0f : g;
            v[p][i] = r * r;
            d[0][p][i] = da[i] * (2.0f * r);
          }
        }
      }
    }
    if constexpr (VALUES) {
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        if (a.a) store_bf16x8(a.a, t.row(p), a.rows, t.col(), a.cols, a.ld_a, v[p]);
#pragma unroll
        for (int h = 0; h < H; ++h)
          if (a.dh) store_bf16x8(a.dh + h * a.cols, t.row(p), a.rows, t.col(), a.cols, a.ld_dh, d[h][p]);
      }
    } else {
#pragma unroll
      for (int h = 0; h < H; ++h) col_partial(t, d[h], cmax[h]);
      col_partial(t, v, cmax[H]);
      __syncthreads();
#pragma unroll
      for (int h = 0; h < H; ++h) col_codes<E5>(cmax[h], code[h], h * kTile);
      col_codes<false>(cmax[H], code[H], H * kTile);
      __syncthreads();
#pragma unroll
      for (int h = 0; h < H; ++h) {
        if (a.dh_codes) {
          uint32_t sc[4];
          row_scales<E5>(d[h], sc);
          store_rows<E5, false>(t, d[h], sc, a.rows, hp, h * fp + t.col(), h * (fp / kTile) + kb,
                                a.dh_codes, a.dh_scales, unused);
        }
        if (a.dh_t_codes) {
          const uint2 sc = *reinterpret_cast<const uint2*>(code[h] + 8 * t.l);
          // row h * cols + column of the transpose (SwiGLU: cols is a multiple
          // of 8 and 2 cols one of 16, so there is no padding)
          if (t.tr == 0 && t.col() < (GLU ? a.cols : up16(a.cols)))
            *reinterpret_cast<uint2*>(a.dh_t_scales + t.r0 / kTile * up16(H * a.cols) + h * a.cols +
                                      t.col()) = sc;
          encode_cols<E5, false>(t, d[h], sc, tile[h], unused);
        }
      }
      if (a.a_t_codes) {
        const uint2 sc = *reinterpret_cast<const uint2*>(code[H] + 8 * t.l);
        if (t.tr == 0 && t.col() < up16(a.cols))
          *reinterpret_cast<uint2*>(a.a_t_scales + t.r0 / kTile * up16(a.cols) + t.col()) = sc;
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

template <bool GLU>
void launch_grad(const fp4lib::Fp8ActGradArgs& a, hipStream_t s) {
  const int64_t tiles = (a.rows + kTile - 1) / kTile * ((a.cols + kTile - 1) / kTile);
  const dim3 block(kTileThreads);
  if (a.dh || a.a)
    hipLaunchKernelGGL((k_act_grad_fp8<GLU, false, true>), dim3(tile_grid(tiles, kWgPerCu)), block, 0, s, a);
  if (!a.dh_codes && !a.dh_t_codes && !a.a_t_codes) return;
  const dim3 grid(tile_grid(tiles, kGradLoop<GLU, false> ? 1 : kWgPerCu));
  if (a.e5m2) hipLaunchKernelGGL((k_act_grad_fp8<GLU, true, false>), grid, block, 0, s, a);
  else hipLaunchKernelGGL((k_act_grad_fp8<GLU, false, false>), grid, block, 0, s, a);
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
  if (a.act == FP4_ACT_SWIGLU) launch_grad<true>(a, s);
  else launch_grad<false>(a, s);
  return hipGetLastError();
}

}  // namespace fp4lib
