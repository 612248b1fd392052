// FP8 block-128 GEMM: D[M, N] (+)= sum_j 2^(eA[m, j] + eB[n, j]) sum_{k in block j}
// a[m, k] b[n, k] on E4M3 / E5M2 codes (include/fp4.h, fp4_gemm).
//
// Two arithmetics, chosen by the output's type:
//
// * bf16 D: gfx950's scaled MFMA multiplies 8-bit operands at the full 8-bit
//   rate with a UE8M0 scale per lane and 32 values of K, so a block-128 scale
//   is applied by handing the instruction the same byte for every part of the
//   block: no vector work at all beside the matrix instructions.  The
//   instruction sums 8 products at a time on the grid of the largest one's
//   exponent - 13, cutting the others off there (measured with single
//   products beside large ones; 1.5e-5 of a random product's norm), before the
//   groups are added in fp32.  A bf16 result has half a step of 2^-9.
// * fp32 D: operands go to bf16 with their block scale applied, both exact
//   (bf16 has fp32's exponents; one packed convert for two elements), and
//   the bf16 MFMA adds their products in fp32, at half the rate.
//
// Code rows are zero-padded to whole blocks, so no kernel masks K.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fp4_internal.hpp"
#include "fp8_common.hpp"
#include "gemm_common.hpp"

namespace fp8gemm {
namespace {

using fp4gemm::floatx16;
using fp4gemm::int8v;
using fp4gemm::ring_barrier;
using fp4gemm::wait_vmcnt;

constexpr int kThreads = 256;
constexpr int kStepBytes = 128;            // one K block per step
constexpr int kChunks = kStepBytes / 16;

struct Params {
  fp4lib::Fp8GemmArgs g;
  int tiles_m, tiles_n;
};

// Chunk q of LDS row r lies at position q ^ swizzle(r): 8 consecutive rows
// reading the same chunk, and the 8 rows of each parity among 16, are on
// different banks.
__device__ __forceinline__ int swizzle(int row) { return (row & 7) ^ ((row >> 3) & 1); }

// Tile order: a contiguous range of tiles per XCD (consecutive workgroups go
// round-robin over the 8), walked in groups of 8 tile rows.
__device__ __forceinline__ void tile_coords(const Params& p, int& tm, int& tn) {
  const int T = p.tiles_m * p.tiles_n;
  int id = blockIdx.x;
  if ((T & 7) == 0) id = (id & 7) * (T >> 3) + (id >> 3);
  constexpr int G = 8;
  const int per_group = G * p.tiles_n;
  const int g = id / per_group;
  const int first = g * G;
  const int gm = min(p.tiles_m - first, G);
  const int r = id - g * per_group;
  tm = first + r % gm;
  tn = r / gm;
}

// The scale bytes of R consecutive operand rows (R = 1, 2, 4) in one word.
template <int R>
__device__ __forceinline__ uint32_t load_scales(const uint8_t* p) {
  if constexpr (R == 4) return *reinterpret_cast<const uint32_t*>(p);
  else if constexpr (R == 2) return *reinterpret_cast<const uint16_t*>(p);
  else return *p;
}

// A workgroup's tile is 64 MI x 64 NI: four waves 2 x 2, each 32 MI x 32 NI
// in MFMAs of 32 x 32 x 64.  MFMA tile mi of a wave takes rows MI i + mi (i =
// 0..31): a lane's MI scales are then consecutive bytes, loaded as one word
// whose byte the instruction selects, and NI consecutive columns of D meet in
// one lane.  LDS rows are in MFMA order (slot mi * 32 + i).
template <int MI, int NI>
struct Stage {
  uint4 a[64 * MI * kChunks], b[64 * NI * kChunks];
};

template <int MI, int NI>
struct Src {
  const uint8_t* a[2 * MI];    // this lane's 16 bytes of slot wave * 16 MI + 8 j + lane / 8
  const uint8_t* b[2 * NI];
  const uint8_t* sa;           // scales of this lane's rows at block 0
  const uint8_t* sb;
  int64_t ska, skb;
};

// Operand row of LDS slot `slot` of a tile (R = MI or NI).
template <int R>
__device__ __forceinline__ int slot_row(int slot) {
  const int part = slot / (32 * R), in = slot % (32 * R);
  return part * 32 * R + (in & 31) * R + (in >> 5);
}

// 16 bytes per lane from global memory to LDS `dst` + 16 * lane.
__device__ __forceinline__ void dma16(const uint8_t* src, uint4* dst) {
  __builtin_amdgcn_global_load_lds(src, dst, 16, 0, 0);
}

template <int MI, int NI>
__device__ __forceinline__ void dma(Stage<MI, NI>& S, const Src<MI, NI>& s, int64_t kb, int wave) {
  const int64_t o = kb * kStepBytes;
#pragma unroll
  for (int j = 0; j < 2 * MI; ++j)
    dma16(s.a[j] + o, &S.a[wave * 128 * MI + j * 64]);
#pragma unroll
  for (int j = 0; j < 2 * NI; ++j)
    dma16(s.b[j] + o, &S.b[wave * 128 * NI + j * 64]);
}

template <int KS>
__device__ __forceinline__ int8v frag(const uint4* base, int slot, int h) {
  const int q = 4 * KS + 2 * h, z = swizzle(slot);
  const uint4 x = base[slot * kChunks + (q ^ z)], y = base[slot * kChunks + ((q + 1) ^ z)];
  return int8v{(int)x.x, (int)x.y, (int)x.z, (int)x.w, (int)y.x, (int)y.y, (int)y.z, (int)y.w};
}

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

// 8 codes (two words) with their block's scale as bf16, exact.
template <bool E5>
__device__ __forceinline__ bf16x8 widen8(uint32_t w0, uint32_t w1, float s) {
  bf16x2 a, b, c, d;
  if constexpr (E5) {
    a = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(w0, s, false);
    b = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(w0, s, true);
    c = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(w1, s, false);
    d = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(w1, s, true);
  } else {
    a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w0, s, false);
    b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w0, s, true);
    c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w1, s, false);
    d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w1, s, true);
  }
  return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// 2^e of scale byte `k` of a word.
__device__ __forceinline__ float scale_of(uint32_t word, int k) {
  return __uint_as_float(((word >> (8 * k)) & 0xFFu) << 23);
}

template <int FA, int MI, int NI, int mi, int ni>
__device__ __forceinline__ void mfma_one(floatx16 (&acc)[MI][NI], const int8v (&a)[MI],
                                         const int8v (&b)[NI], uint32_t sa, uint32_t sb) {
  acc[mi][ni] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
      b[ni], a[mi], acc[mi][ni], 0, FA, ni, static_cast<int>(sb), mi, static_cast<int>(sa));
}

template <int FA, int MI, int NI, int X = 0>
__device__ __forceinline__ void mfma_slice(floatx16 (&acc)[MI][NI], const int8v (&a)[MI],
                                           const int8v (&b)[NI], uint32_t sa, uint32_t sb) {
  if constexpr (X < MI * NI) {
    mfma_one<FA, MI, NI, X / NI, X % NI>(acc, a, b, sa, sb);
    mfma_slice<FA, MI, NI, X + 1>(acc, a, b, sa, sb);
  }
}

// D through LDS: each wave's 32 rows of one mi (rows MI i + mi) x 32 NI
// columns go through its own buffer, in which a lane writes NI consecutive
// columns, and leave as whole row segments of 128 NI bytes.  Every value is
// the fp32 sum, plus the old D if accumulating, rounded once for bf16.
template <int MI, int NI>
__device__ __forceinline__ void epilogue(const fp4lib::Fp8GemmArgs& g, floatx16 (&acc)[MI][NI],
                                         int64_t row0, int64_t col0, int lane, float* buf) {
  constexpr int W = 32 * NI, P = W + 4;
  const int i = lane & 31, h = lane >> 5;
  const int64_t left = g.N - col0;           // columns of D from col0 on
  const int es = g.d_bf16 ? 2 : 4;
  // whole groups of 4 columns, aligned
  const bool vec = left >= W && (g.ldd & 3) == 0 &&
                   (reinterpret_cast<uintptr_t>(g.D) & (4 * es - 1)) == 0;
#pragma unroll
  for (int mi = 0; mi < MI; ++mi) {
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      float* d = buf + i * P + (8 * (k >> 2) + 4 * h + (k & 3)) * NI;
#pragma unroll
      for (int ni = 0; ni < NI; ++ni) d[ni] = acc[mi][ni][k];
    }
    __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
    if (vec) {
      constexpr int L = W / 4;               // lanes of a row
#pragma unroll 4
      for (int k = 0; k < 32 * L / 64; ++k) {
        const int r = k * (64 / L) + lane / L, c = (lane % L) * 4;
        const int64_t row = row0 + r * MI + mi;
        if (row >= g.M) continue;
        float4 v = *reinterpret_cast<const float4*>(buf + r * P + c);
        if (g.d_bf16) {
          uint2* d = reinterpret_cast<uint2*>(static_cast<uint16_t*>(g.D) + row * g.ldd + col0 + c);
          if (g.accumulate) {
            const uint2 o = *d;
            v.x += __uint_as_float(o.x << 16);
            v.y += __uint_as_float(o.x & 0xFFFF0000u);
            v.z += __uint_as_float(o.y << 16);
            v.w += __uint_as_float(o.y & 0xFFFF0000u);
          }
          *d = make_uint2(fp8dev::to_bf16(v.x) | (fp8dev::to_bf16(v.y) << 16),
                          fp8dev::to_bf16(v.z) | (fp8dev::to_bf16(v.w) << 16));
        } else {
          float4* d = reinterpret_cast<float4*>(static_cast<float*>(g.D) + row * g.ldd + col0 + c);
          if (g.accumulate) {
            const float4 o = *d;
            v = make_float4(v.x + o.x, v.y + o.y, v.z + o.z, v.w + o.w);
          }
          *d = v;
        }
      }
    } else {
      for (int k = 0; k < 32 * W / 64; ++k) {
        const int r = (k * 64 + lane) / W, c = (k * 64 + lane) % W;
        const int64_t row = row0 + r * MI + mi;
        if (row >= g.M || c >= left) continue;
        float v = buf[r * P + c];
        if (g.d_bf16) {
          uint16_t* d = static_cast<uint16_t*>(g.D) + row * g.ldd + col0 + c;
          if (g.accumulate) v += __uint_as_float(static_cast<uint32_t>(*d) << 16);
          *d = static_cast<uint16_t>(fp8dev::to_bf16(v));
        } else {
          float* d = static_cast<float*>(g.D) + row * g.ldd + col0 + c;
          *d = g.accumulate ? *d + v : v;
        }
      }
    }
    // these reads precede the next rows' writes
    __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
  }
}

// PREC: bf16 MFMA (fp32 D); else the scaled 8-bit one (bf16 D).
template <int FA, bool PREC, int MI, int NI>
__global__ __launch_bounds__(kThreads) void k_gemm_fp8(Params p) {
  __shared__ Stage<MI, NI> s0, s1;
  const fp4lib::Fp8GemmArgs& g = p.g;
  int tm, tn;
  tile_coords(p, tm, tn);
  const int64_t m0 = static_cast<int64_t>(tm) * (64 * MI), n0 = static_cast<int64_t>(tn) * (64 * NI);
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave >> 1, wn = wave & 1;
  const int i = lane & 31, h = lane >> 5;

  // Rows outside the operands read their last row; their outputs are not stored.
  Src<MI, NI> src;
#pragma unroll
  for (int j = 0; j < 2 * MI; ++j) {
    const int slot = wave * 16 * MI + 8 * j + (lane >> 3);
    const int64_t r = min(m0 + slot_row<MI>(slot), g.M - 1);
    src.a[j] = g.codes[0] + r * g.ld[0] + 16 * ((lane & 7) ^ swizzle(slot));
  }
#pragma unroll
  for (int j = 0; j < 2 * NI; ++j) {
    const int slot = wave * 16 * NI + 8 * j + (lane >> 3);
    const int64_t r = min(n0 + slot_row<NI>(slot), g.N - 1);
    src.b[j] = g.codes[1] + r * g.ld[1] + 16 * ((lane & 7) ^ swizzle(slot));
  }
  // the scales' pitch is a multiple of 16 and at least the rows
  src.sa = g.scales[0] + min(m0 + wm * 32 * MI + i * MI, g.s_kblk[0] - MI);
  src.sb = g.scales[1] + min(n0 + wn * 32 * NI + i * NI, g.s_kblk[1] - NI);
  src.ska = g.s_kblk[0];
  src.skb = g.s_kblk[1];

  floatx16 acc[MI][NI];
#pragma unroll
  for (int mi = 0; mi < MI; ++mi)
#pragma unroll
    for (int ni = 0; ni < NI; ++ni) acc[mi][ni] = floatx16{};

  const int nkb = static_cast<int>(g.nkb);
  // One step on stage C: its DMA has landed for every wave, the other stage
  // N (read in the previous step) takes block kb + 1 (the last one again at
  // the end, unread).
  auto step = [&](Stage<MI, NI>& C, Stage<MI, NI>& N, int kb) {
    wait_vmcnt<0>();
    ring_barrier();
    dma(N, src, min(kb + 1, nkb - 1), wave);
    const uint32_t sa = load_scales<MI>(src.sa + kb * src.ska);
    const uint32_t sb = load_scales<NI>(src.sb + kb * src.skb);
    if constexpr (PREC) {
      // a lane's 16 bytes of a row feed two products of 16 K values
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        uint4 ca[MI], cb[NI];
#pragma unroll
        for (int mi = 0; mi < MI; ++mi) {
          const int slot = wm * 32 * MI + mi * 32 + i;
          ca[mi] = C.a[slot * kChunks + ((2 * q + h) ^ swizzle(slot))];
        }
#pragma unroll
        for (int ni = 0; ni < NI; ++ni) {
          const int slot = wn * 32 * NI + ni * 32 + i;
          cb[ni] = C.b[slot * kChunks + ((2 * q + h) ^ swizzle(slot))];
        }
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          bf16x8 a[MI], b[NI];
#pragma unroll
          for (int mi = 0; mi < MI; ++mi)
            a[mi] = widen8<FA == 1>(half ? ca[mi].z : ca[mi].x, half ? ca[mi].w : ca[mi].y, scale_of(sa, mi));
#pragma unroll
          for (int ni = 0; ni < NI; ++ni)
            b[ni] = widen8<false>(half ? cb[ni].z : cb[ni].x, half ? cb[ni].w : cb[ni].y, scale_of(sb, ni));
#pragma unroll
          for (int mi = 0; mi < MI; ++mi)
#pragma unroll
            for (int ni = 0; ni < NI; ++ni)
              acc[mi][ni] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(b[ni], a[mi], acc[mi][ni], 0, 0, 0);
        }
      }
    } else {
      int8v a[MI], b[NI];
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
#pragma unroll
        for (int mi = 0; mi < MI; ++mi) {
          const int slot = wm * 32 * MI + mi * 32 + i;
          a[mi] = ks ? frag<1>(C.a, slot, h) : frag<0>(C.a, slot, h);
        }
#pragma unroll
        for (int ni = 0; ni < NI; ++ni) {
          const int slot = wn * 32 * NI + ni * 32 + i;
          b[ni] = ks ? frag<1>(C.b, slot, h) : frag<0>(C.b, slot, h);
        }
        mfma_slice<FA, MI, NI>(acc, a, b, sa, sb);
      }
    }
  };
  if (nkb > 0) {
    dma(s0, src, 0, wave);
    int kb = 0;
    for (; kb + 1 < nkb; kb += 2) {
      step(s0, s1, kb);
      step(s1, s0, kb + 1);
    }
    if (kb < nkb) step(s0, s1, kb);
  }
  wait_vmcnt<0>();
  ring_barrier();
  // both stages are done with: stage 0 and 1 hold the waves' buffers
  constexpr int kBuf = 32 * (32 * NI + 4);
  static_assert(2 * kBuf * sizeof(float) <= sizeof(Stage<MI, NI>), "two epilogue buffers per stage");
  float* buf = reinterpret_cast<float*>(wave < 2 ? &s0 : &s1) + (wave & 1) * kBuf;
  epilogue<MI, NI>(g, acc, m0 + wm * 32 * MI, n0 + wn * 32 * NI, lane, buf);
}

template <int FA, bool PREC, int MI, int NI>
hipError_t launch(const fp4lib::Fp8GemmArgs& g, hipStream_t s) {
  Params p{g, static_cast<int>((g.M + 64 * MI - 1) / (64 * MI)),
           static_cast<int>((g.N + 64 * NI - 1) / (64 * NI))};
  hipLaunchKernelGGL((k_gemm_fp8<FA, PREC, MI, NI>), dim3(p.tiles_m * p.tiles_n), dim3(kThreads), 0,
                     s, p);
  return hipGetLastError();
}

}  // namespace
}  // namespace fp8gemm

namespace fp4lib {

hipError_t launch_gemm_fp8(const Fp8GemmArgs& g, hipStream_t s) {
  using fp8gemm::launch;
  if (g.a_e5m2) return g.d_bf16 ? launch<1, false, 2, 2>(g, s) : launch<1, true, 2, 2>(g, s);
  return g.d_bf16 ? launch<0, false, 2, 2>(g, s) : launch<0, true, 2, 2>(g, s);
}

}  // namespace fp4lib
