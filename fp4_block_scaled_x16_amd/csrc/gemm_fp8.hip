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
//   groups are added in fp32.  Half a step of a bf16 result is 2^-9 to 2^-8 of it.
//   What is cut off makes sums of one sign smaller, by 1e-5 of themselves (K = 4096,
//   squares of normal values against magnitudes of others), 1/200 of that.
// * fp32 D: operands go to bf16 with their block scale applied, exact from 2^-126
//   to below 2^128 (bf16 has fp32's exponents; one packed convert for two
//   elements), and the bf16 MFMA adds their products in fp32, at half the rate.
//
// Code rows are zero-padded to whole blocks, so no kernel masks K.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <atomic>
#include <cmath>

#include "fp4_internal.hpp"
#include "fp8_common.hpp"
#include "gemm_common.hpp"
#include "gemm_fp8_common.hpp"

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
__device__ __forceinline__ void tile_coords(const Params& p, int id, int& tm, int& tn) {
  const int T = p.tiles_m * p.tiles_n;
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

// 16 and 8 bytes at an element's alignment (gfx950 takes them as one access).
typedef float float4_any __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t uint32_any __attribute__((aligned(1)));
typedef uint32_t uint2_any __attribute__((ext_vector_type(2), aligned(2)));
typedef uint32_t uint4_any __attribute__((ext_vector_type(4), aligned(2)));

// D through LDS: each wave's 32 rows of one mi (rows MI i + mi) x 32 NI
// columns go through its own buffer, in which a lane writes NI consecutive
// columns, and leave as whole row segments of 128 NI bytes, whatever the
// alignment of D's rows (the last group of a row whose length is no multiple
// of 4 goes out element by element).  Every value is the fp32 sum, plus the old
// D if accumulating, rounded once for bf16.
template <int MI, int NI>
__device__ __forceinline__ void epilogue(const fp4lib::Fp8GemmArgs& g, floatx16 (&acc)[MI][NI],
                                         int64_t row0, int64_t col0, int lane, float* buf) {
  constexpr int W = 32 * NI, P = W + 4, L = W / 4;      // L: lanes of a row
  const int i = lane & 31, h = lane >> 5;
  const int c = (lane % L) * 4;
  const int n = static_cast<int>(min(g.N - col0 - c, int64_t(4)));     // this lane's columns inside D
  constexpr int R = 32 * L / 64;        // rows of a lane
  const bool add_f32 = g.accumulate && !g.d_bf16 && n == 4;
#pragma unroll
  for (int mi = 0; mi < MI; ++mi) {
    // an fp32 D that is added to: all of its loads at once (6144 x 2048 x 8192
    // 171 us; one before each sum 180), of D's last row for rows outside
    float4_any old[R];
    if (add_f32) {
#pragma unroll
      for (int k = 0; k < R; ++k) {
        const int64_t row = min(row0 + (k * (64 / L) + lane / L) * MI + mi, g.M - 1);
        old[k] = *reinterpret_cast<const float4_any*>(static_cast<float*>(g.D) + row * g.ldd + col0 + c);
      }
    }
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      float* d = buf + i * P + (8 * (k >> 2) + 4 * h + (k & 3)) * NI;
#pragma unroll
      for (int ni = 0; ni < NI; ++ni) d[ni] = acc[mi][ni][k];
    }
    __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
#pragma unroll
    for (int k = 0; k < R; ++k) {
      const int r = k * (64 / L) + lane / L;
      const int64_t row = row0 + r * MI + mi;
      if (row >= g.M || n <= 0) continue;
      float4 v = *reinterpret_cast<const float4*>(buf + r * P + c);
      if (g.d_bf16) {
        uint16_t* d = static_cast<uint16_t*>(g.D) + row * g.ldd + col0 + c;
        if (n == 4) {
          if (g.accumulate) {
            const uint2_any o = *reinterpret_cast<const uint2_any*>(d);
            v.x += __uint_as_float(o.x << 16);
            v.y += __uint_as_float(o.x & 0xFFFF0000u);
            v.z += __uint_as_float(o.y << 16);
            v.w += __uint_as_float(o.y & 0xFFFF0000u);
          }
          *reinterpret_cast<uint2_any*>(d) = uint2_any{fp8dev::pack_bf16(v.x, v.y), fp8dev::pack_bf16(v.z, v.w)};
        } else {
          const float e[3] = {v.x, v.y, v.z};
#pragma unroll
          for (int x = 0; x < 3; ++x)
            if (x < n)
              d[x] = fp8dev::to_bf16(g.accumulate ? e[x] + __uint_as_float(static_cast<uint32_t>(d[x]) << 16) : e[x]);
        }
      } else {
        float* d = static_cast<float*>(g.D) + row * g.ldd + col0 + c;
        if (n == 4) {
          float4_any o = float4_any{v.x, v.y, v.z, v.w};
          if (add_f32) o += old[k];
          *reinterpret_cast<float4_any*>(d) = o;
        } else {
          const float e[3] = {v.x, v.y, v.z};
#pragma unroll
          for (int x = 0; x < 3; ++x)
            if (x < n) d[x] = g.accumulate ? d[x] + e[x] : e[x];
        }
      }
    }
    // these reads precede the next rows' writes
    __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
  }
}

// One K block on stage C.  PREC: bf16 MFMA (fp32 D); else the scaled 8-bit one.
template <int FA, bool PREC, int MI, int NI>
__device__ __forceinline__ void multiply(const Stage<MI, NI>& C, floatx16 (&acc)[MI][NI], uint32_t sa,
                                         uint32_t sb, int wm, int wn, int i, int h) {
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
}

// Tiles of 64 and 128: S stages in a ring, S - 1 blocks on their way while one
// is multiplied, one barrier per block.  Two workgroups per CU, so the reads
// of one are covered by the other's products.
template <int FA, bool PREC, int MI, int NI, int S>
__global__ __launch_bounds__(kThreads) void k_gemm_fp8(Params p) {
  static_assert(S == 2 || S == 3, "stages");
  __shared__ Stage<MI, NI> s0, s1, s2;
  int kb0, nkb;
  const fp4lib::Fp8GemmArgs g = split_args(p.g, kb0, nkb);
  int tm, tn;
  tile_coords(p, blockIdx.x, tm, tn);
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
    src.a[j] = g.codes[0] + r * g.ld[0] + static_cast<int64_t>(kb0) * kStepBytes + 16 * ((lane & 7) ^ swizzle(slot));
  }
#pragma unroll
  for (int j = 0; j < 2 * NI; ++j) {
    const int slot = wave * 16 * NI + 8 * j + (lane >> 3);
    const int64_t r = min(n0 + slot_row<NI>(slot), g.N - 1);
    src.b[j] = g.codes[1] + r * g.ld[1] + static_cast<int64_t>(kb0) * kStepBytes + 16 * ((lane & 7) ^ swizzle(slot));
  }
  // the scales' pitch is a multiple of 16 and at least the rows
  src.sa = g.scales[0] + kb0 * g.s_kblk[0] + min(m0 + wm * 32 * MI + i * MI, g.s_kblk[0] - MI);
  src.sb = g.scales[1] + kb0 * g.s_kblk[1] + min(n0 + wn * 32 * NI + i * NI, g.s_kblk[1] - NI);
  src.ska = g.s_kblk[0];
  src.skb = g.s_kblk[1];

  floatx16 acc[MI][NI];
#pragma unroll
  for (int mi = 0; mi < MI; ++mi)
#pragma unroll
    for (int ni = 0; ni < NI; ++ni) acc[mi][ni] = floatx16{};

  // A block's DMA; its scales are loaded before them, so that a wait that leaves
  // one block's DMA under way has the block before it complete.
  constexpr int kGroup = 2 * MI + 2 * NI;
  uint32_t sa[S], sb[S];
  auto fetch = [&](Stage<MI, NI>& D, int j, int kb) {
    const int k = min(kb, nkb - 1);
    sa[j] = load_scales<MI>(src.sa + k * src.ska);
    sb[j] = load_scales<NI>(src.sb + k * src.skb);
    dma(D, src, k, wave);
    __builtin_amdgcn_sched_barrier(0);
  };
  // Block kb on stage C (number j): it has landed for every wave, and the
  // stage that was multiplied last (F, number f) takes block kb + S - 1 (past
  // the end the last one again, unread).
  auto step = [&](Stage<MI, NI>& C, int j, Stage<MI, NI>& F, int f, int kb) {
    wait_vmcnt<(S - 2) * kGroup>();
    ring_barrier();
    const uint32_t ca = sa[j], cb = sb[j];
    fetch(F, f, kb + S - 1);
    multiply<FA, PREC, MI, NI>(C, acc, ca, cb, wm, wn, i, h);
  };
  if (nkb > 0) {
    fetch(s0, 0, 0);
    if constexpr (S == 3) fetch(s1, 1, 1);
    // whole turns of the ring, then what is left of one (an exit inside the
    // loop makes the compiler move the accumulators)
    int kb = 0;
    if constexpr (S == 3) {
      for (; kb + 2 < nkb; kb += 3) {
        step(s0, 0, s2, 2, kb);
        step(s1, 1, s0, 0, kb + 1);
        step(s2, 2, s1, 1, kb + 2);
      }
      if (kb < nkb) step(s0, 0, s2, 2, kb);
      if (kb + 1 < nkb) step(s1, 1, s0, 0, kb + 1);
    } else {
      for (; kb + 1 < nkb; kb += 2) {
        step(s0, 0, s1, 1, kb);
        step(s1, 1, s0, 0, kb + 1);
      }
      if (kb < nkb) step(s0, 0, s1, 1, kb);
    }
  }
  wait_vmcnt<0>();
  ring_barrier();
  // the stages are done with: the first two hold the waves' buffers
  constexpr int kBuf = 32 * (32 * NI + 4);
  static_assert(2 * kBuf * sizeof(float) <= sizeof(Stage<MI, NI>), "two epilogue buffers per stage");
  float* buf = reinterpret_cast<float*>(wave < 2 ? &s0 : &s1) + (wave & 1) * kBuf;
  epilogue<MI, NI>(g, acc, m0 + wm * 32 * MI, n0 + wn * 32 * NI, lane, buf);
}

// ------------------------------------------------------- 256 x 256, 8-bit --
// The same product to bf16 for large outputs: a wave's 128 x 128 part needs
// half the LDS reads per MFMA of a 64 x 64 one (the LDS pipe bounds the
// smaller tile).  Two stages of 64 KiB; the operands of a step's first half
// are read while the previous step's second half is multiplied, so the one
// barrier of a step (stage Nx landed, stage C read by every wave) stands
// between two halves whose operands are in registers.  sched_barrier(0) pins
// one MFMA and its share of LDS reads and DMA together: left to the scheduler
// the DMA sinks to the next barrier.
//
// 8192 x 21504 x 4096: 600 us, 2.41 PFLOP/s, at the card's power limit (1.6 GHz);
// the MFMAs alone, on registers, take 496, and 515 with their LDS reads.
struct Frags {
  int8v a[4], b[4];
};

// Fragment x (0..7: b0 a0 b1 b2 b3 a1 a2 a3, the order of first use) of half KS.
template <int KS, int X>
__device__ __forceinline__ void read_frag(const Stage<4, 4>& S, Frags& f, int wm, int wn, int i, int h) {
  constexpr bool kIsA = X == 1 || X >= 5;
  constexpr int kT = X == 0 ? 0 : X == 1 ? 0 : X < 5 ? X - 1 : X - 4;
  if constexpr (kIsA) f.a[kT] = frag<KS>(S.a, wm * 128 + kT * 32 + i, h);
  else f.b[kT] = frag<KS>(S.b, wn * 128 + kT * 32 + i, h);
}

// The tile's code rows: a uniform base and a 32-bit offset per DMA (the host
// keeps 256 row pitches below 2^31).
template <int MI>
struct WideSrc {
  const uint8_t *a, *b;
  uint32_t off_a[2 * MI], off_b[8];
};

// The x-th of a stage's 2 MI + 8 DMA of a wave.
template <int MI>
__device__ __forceinline__ void wide_dma(Stage<MI, 4>& W, const WideSrc<MI>& s, int64_t koff, int wave, int x) {
  if (x < 2 * MI) dma16(s.a + koff + s.off_a[x], W.a + wave * 128 * MI + x * 64);
  else dma16(s.b + koff + s.off_b[x - 2 * MI], W.b + wave * 512 + (x - 2 * MI) * 64);
}

// Where a workgroup of the wide kernels stands: its tile, the wave's part, and
// what its lanes load.
template <int MI>
struct WidePos {
  int64_t m0, n0;
  int lane, wave, wm, wn, i, h;
  WideSrc<MI> src;
  const uint8_t *psa, *psb;      // scales of this lane's MI and 4 rows at the first block
  uint32_t shift;                // MI = 3: of the word at psa
};

template <int MI>
__device__ __forceinline__ WidePos<MI> wide_pos(const Params& p, const fp4lib::Fp8GemmArgs& g, int id, int kb0) {
  WidePos<MI> w;
  int tm, tn;
  tile_coords(p, id, tm, tn);
  w.m0 = static_cast<int64_t>(tm) * (64 * MI);
  w.n0 = static_cast<int64_t>(tn) * 256;
  w.lane = threadIdx.x & 63;
  // per tile, not once: addresses kept over the tile loop would be spilled
  asm volatile("" : "+v"(w.lane));
  w.wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  w.wm = w.wave >> 1;
  w.wn = w.wave & 1;
  w.i = w.lane & 31;
  w.h = w.lane >> 5;
  w.src.a = g.codes[0] + w.m0 * g.ld[0] + static_cast<int64_t>(kb0) * kStepBytes;
  w.src.b = g.codes[1] + w.n0 * g.ld[1] + static_cast<int64_t>(kb0) * kStepBytes;
  const uint32_t last_a = static_cast<uint32_t>(min(g.M - 1 - w.m0, int64_t(64 * MI - 1)));
  const uint32_t last_b = static_cast<uint32_t>(min(g.N - 1 - w.n0, int64_t(255)));
#pragma unroll
  for (int x = 0; x < 2 * MI; ++x) {
    const int slot = w.wave * 16 * MI + 8 * x + (w.lane >> 3);
    w.src.off_a[x] = min(static_cast<uint32_t>(slot_row<MI>(slot)), last_a) * static_cast<uint32_t>(g.ld[0]) +
                     16 * ((w.lane & 7) ^ swizzle(slot));
  }
#pragma unroll
  for (int x = 0; x < 8; ++x) {
    const int slot = w.wave * 64 + 8 * x + (w.lane >> 3);
    w.src.off_b[x] = min(static_cast<uint32_t>(slot_row<4>(slot)), last_b) * static_cast<uint32_t>(g.ld[1]) +
                     16 * ((w.lane & 7) ^ swizzle(slot));
  }
  // Three rows' scales are the low bytes of the word at their first one, read
  // from before the end of the block's scales and shifted there.
  const int64_t ra = w.m0 + w.wm * 32 * MI + w.i * MI, at = min(ra, g.s_kblk[0] - 4);
  w.shift = static_cast<uint32_t>(min(ra - at, int64_t(3))) * 8;
  w.psa = g.scales[0] + kb0 * g.s_kblk[0] + at;
  w.psb = g.scales[1] + kb0 * g.s_kblk[1] + min(w.n0 + w.wn * 128 + w.i * 4, g.s_kblk[1] - 4);
  return w;
}

// Half of a step: 16 MFMAs on `cur`, the reads of half KS of stage R into
// `nxt` beside the first 8 and, if DMA, block kb into stage W, one DMA beside
// each: evenly, for a burst holds the wave's next MFMA back (8192 x 4096 x 21504:
// 534 us; two beside each of the first 8: 572, four beside 4: 594).
template <int FA, int KS, bool DMA, int X = 0>
__device__ __forceinline__ void wide_half(floatx16 (&acc)[4][4], const Frags& cur, uint32_t sa,
                                          uint32_t sb, const Stage<4, 4>& R, Frags& nxt,
                                          Stage<4, 4>& W, int64_t koff, const WidePos<4>& w) {
  if constexpr (X < 16) {
    mfma_one<FA, 4, 4, X / 4, X % 4>(acc, cur.a, cur.b, sa, sb);
    if constexpr (X < 8) read_frag<KS, X>(R, nxt, w.wm, w.wn, w.i, w.h);
    if constexpr (DMA) wide_dma(W, w.src, koff, w.wave, X);
    __builtin_amdgcn_sched_barrier(0);
    wide_half<FA, KS, DMA, X + 1>(acc, cur, sa, sb, R, nxt, W, koff, w);
  }
}

// A wave's 128 x 128 part of a bf16 D through 32 x 64 buffers of its own: a
// lane's values of 8 accumulators are 4 consecutive columns each (8 bytes), and
// 8 lanes write a row's 128 bytes.  row0, col: this lane's first row and column.
constexpr int kWidePitch = 72;              // bf16 of a buffer row: 64 and 16 bytes of padding
__device__ __forceinline__ void wide_store_bf16(const fp4lib::Fp8GemmArgs& g, floatx16 (&acc)[4][4],
                                                const WidePos<4>& w, int64_t row0, int64_t col,
                                                uint16_t* buf) {
  uint16_t* d = static_cast<uint16_t*>(g.D) + row0 * g.ldd + col;
#pragma unroll
  for (int mi = 0; mi < 4; ++mi) {
#pragma unroll
    for (int half = 0; half < 2; ++half) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int k = 8 * half + e;
        *reinterpret_cast<uint2*>(buf + w.i * kWidePitch + (8 * (e >> 2) + 4 * w.h + (e & 3)) * 4) =
            make_uint2(fp8dev::pack_bf16(acc[mi][0][k], acc[mi][1][k]),
                       fp8dev::pack_bf16(acc[mi][2][k], acc[mi][3][k]));
      }
      __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const uint4 v = *reinterpret_cast<const uint4*>(buf + (8 * r + (w.lane >> 3)) * kWidePitch + 8 * (w.lane & 7));
        if (row0 + 32 * r + mi < g.M && col + 64 * half < g.N) {
          uint16_t* o = d + (32 * r + mi) * g.ldd + 64 * half;
          if (col + 64 * half + 8 <= g.N) {
            *reinterpret_cast<uint4_any*>(o) = uint4_any{v.x, v.y, v.z, v.w};
          } else {
            const uint32_t e[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int x = 0; x < 7; ++x)
              if (col + 64 * half + x < g.N) o[x] = static_cast<uint16_t>(e[x >> 1] >> (16 * (x & 1)));
          }
        }
      }
      __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
    }
  }
}

// The scales of this lane's MI rows of A, `off` bytes on.
template <int MI>
__device__ __forceinline__ uint32_t wide_scales_a(const WidePos<MI>& w, int64_t off) {
  if constexpr (MI == 4) return load_scales<4>(w.psa + off);
  else return *reinterpret_cast<const uint32_any*>(w.psa + off) >> w.shift;
}

// The scales of the wave's rows of A and B: of the block that is multiplied,
// and of the one after it.
struct WideScales {
  uint32_t a, b, na, nb;
};

__device__ __forceinline__ WideScales wide_scales(const fp4lib::Fp8GemmArgs& g, const WidePos<4>& w, int nkb) {
  const int k1 = min(1, nkb - 1);
  return WideScales{load_scales<4>(w.psa), load_scales<4>(w.psb), load_scales<4>(w.psa + k1 * g.s_kblk[0]),
                    load_scales<4>(w.psb + k1 * g.s_kblk[1])};
}

// Blocks 0 and 1 of a tile on their way into the stages.
__device__ __forceinline__ void wide_begin(Stage<4, 4>& s0, Stage<4, 4>& s1, const WidePos<4>& w, int nkb) {
  __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int x = 0; x < 16; ++x) wide_dma(s0, w.src, 0, w.wave, x);
#pragma unroll
  for (int x = 0; x < 16; ++x) wide_dma(s1, w.src, nkb > 1 ? kStepBytes : 0, w.wave, x);
  __builtin_amdgcn_sched_barrier(0);
}

// Step kb on stage C, whose first half's operands (f0) and scales are in
// registers; block kb + 1 is in (or on its way to) Nx; C takes block kb + 2
// (past the end the last one again).  Steps go in pairs: with an odd number
// of blocks the last one is multiplied again under scales 2^-127 2^-127, whose
// products are zero in fp32 (a loop exit between the two steps makes the
// compiler move the 256 accumulators, and spill).  The scales of block kb + 2
// are loaded before its DMA, a whole step before their use, so that no wait
// for them is a wait for the DMA.
template <int FA>
__device__ __forceinline__ void wide_step(floatx16 (&acc)[4][4], Frags& f0, Frags& f1, WideScales& s,
                                          Stage<4, 4>& C, Stage<4, 4>& Nx, int kb, int nkb,
                                          const fp4lib::Fp8GemmArgs& g, const WidePos<4>& w) {
  const int k2 = min(kb + 2, nkb - 1);
  wide_half<FA, 1, false>(acc, f0, s.a, s.b, C, f1, C, 0, w);
  wait_vmcnt<0>();
  ring_barrier();
  const uint32_t pa = load_scales<4>(w.psa + k2 * g.s_kblk[0]);
  const uint32_t pb = load_scales<4>(w.psb + k2 * g.s_kblk[1]);
  wide_half<FA, 0, true>(acc, f1, s.a, s.b, Nx, f0, C, static_cast<int64_t>(k2) * kStepBytes, w);
  s.a = kb + 1 < nkb ? s.na : 0;
  s.b = kb + 1 < nkb ? s.nb : 0;
  s.na = pa;
  s.nb = pb;
}

__device__ __forceinline__ void wide_first_frags(const Stage<4, 4>& s0, Frags& f0, const WidePos<4>& w) {
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    f0.a[t] = frag<0>(s0.a, w.wm * 128 + t * 32 + w.i, w.h);
    f0.b[t] = frag<0>(s0.b, w.wn * 128 + t * 32 + w.i, w.h);
  }
}

__device__ __forceinline__ void wide_zero(floatx16 (&acc)[4][4]) {
#pragma unroll
  for (int mi = 0; mi < 4; ++mi)
#pragma unroll
    for (int ni = 0; ni < 4; ++ni) acc[mi][ni] = floatx16{};
}

// Any D: one tile per workgroup.
template <int FA>
__global__ __launch_bounds__(kThreads, 1) void k_gemm_fp8_wide(Params p) {
  __shared__ Stage<4, 4> s0, s1;
  int kb0, nkb;
  const fp4lib::Fp8GemmArgs g = split_args(p.g, kb0, nkb);
  const WidePos<4> w = wide_pos<4>(p, g, blockIdx.x, kb0);
  floatx16 acc[4][4];
  wide_zero(acc);
  if (nkb > 0) {
    WideScales sc = wide_scales(g, w, nkb);
    Frags f0, f1;
    wide_begin(s0, s1, w, nkb);
    wait_vmcnt<16>();
    ring_barrier();
    wide_first_frags(s0, f0, w);
    for (int kb = 0; kb < nkb; kb += 2) {
      wide_step<FA>(acc, f0, f1, sc, s0, s1, kb, nkb, g, w);
      wide_step<FA>(acc, f0, f1, sc, s1, s0, kb + 1, nkb, g, w);
    }
  }
  wait_vmcnt<0>();
  ring_barrier();
  constexpr int kBuf = 32 * (32 * 4 + 4);
  float* buf = reinterpret_cast<float*>(w.wave < 2 ? &s0 : &s1) + (w.wave & 1) * kBuf;
  epilogue<4, 4>(g, acc, w.m0 + w.wm * 128, w.n0 + w.wn * 128, w.lane, buf);
}

// A bf16 D, not accumulated: a workgroup per CU takes tile after tile, the first two blocks of the next
// one on their way while a tile is stored.
template <int FA>
__global__ __launch_bounds__(kThreads, 1) void k_gemm_fp8_wide_loop(Params p) {
  __shared__ Stage<4, 4> s0, s1;
  __shared__ __attribute__((aligned(16))) uint16_t ebuf[4][32 * kWidePitch];
  const fp4lib::Fp8GemmArgs& g = p.g;
  const int nkb = static_cast<int>(g.nkb), tiles = p.tiles_m * p.tiles_n;
  int id = blockIdx.x;
  WidePos<4> w = wide_pos<4>(p, g, id, 0);
  WideScales sc = wide_scales(g, w, nkb);
  wide_begin(s0, s1, w, nkb);
  for (;;) {
    floatx16 acc[4][4];
    wide_zero(acc);
    Frags f0, f1;
    wait_vmcnt<0>();
    ring_barrier();
    wide_first_frags(s0, f0, w);
    for (int kb = 0; kb < nkb; kb += 2) {
      wide_step<FA>(acc, f0, f1, sc, s0, s1, kb, nkb, g, w);
      wide_step<FA>(acc, f0, f1, sc, s1, s0, kb + 1, nkb, g, w);
    }
    id += gridDim.x;
    const int64_t row0 = w.m0 + w.wm * 128 + (w.lane >> 3) * 4, col = w.n0 + w.wn * 128 + 8 * (w.lane & 7);
    if (id < tiles) {
      w = wide_pos<4>(p, g, id, 0);
      sc = wide_scales(g, w, nkb);
    }
    wait_vmcnt<0>();
    ring_barrier();           // both stages are done with
    if (id < tiles) wide_begin(s0, s1, w, nkb);
    wide_store_bf16(g, acc, w, row0, col, ebuf[w.wave]);
    if (id >= tiles) break;
  }
}

// ------------------------------------------------------ 256 x 256, bf16 ---
// The product to fp32 for large outputs: the wide tile, of 256 or (where that
// leaves fewer CUs idle) 192 rows, with its codes widened
// to bf16 in registers, two converts beside each MFMA.  A step is four
// quarters of 32 K values; a lane's 16 bytes of each row in a quarter are two
// products' operands (halves).  While a half is multiplied the next one is
// widened, from bytes read from LDS a quarter ahead; the barrier stands before
// the last quarter, whose bytes are then in registers, so the DMA of the
// stage that it frees has most of a step to land.
//
// 6144 x 2048 x 8192: 164 us, 1.26 PFLOP/s (171 added to D).  15 us (22) of it are
// the first blocks' latency and D's own traffic, which nothing covers in a
// single round of tiles; the MFMAs alone take 130.
template <int MI>
struct Raw {
  uint4 a[MI], b[4];
};
template <int MI>
struct Wide {
  uint32_t a[MI][4], b[4][4];
};

// Tile t (0..3 B, then A) of quarter Q.
template <int Q, int MI>
__device__ __forceinline__ void read_raw(const Stage<MI, 4>& S, Raw<MI>& r, int t, const WidePos<MI>& w) {
  const int q = 2 * Q + w.h;
  if (t < 4) {
    const int slot = w.wn * 128 + t * 32 + w.i;
    r.b[t] = S.b[slot * kChunks + (q ^ swizzle(slot))];
  } else {
    const int slot = w.wm * 32 * MI + (t - 4) * 32 + w.i;
    r.a[t - 4] = S.a[slot * kChunks + (q ^ swizzle(slot))];
  }
}

// Word w (0, 1) of tile t's half HALF as four bf16.
template <int FA, int HALF, int MI>
__device__ __forceinline__ void widen_word(const Raw<MI>& r, Wide<MI>& f, int t, int w, const float (&s)[4 + MI]) {
  const uint4& c = t < 4 ? r.b[t & 3] : r.a[t & 3];
  const uint32_t x = HALF ? (w ? c.w : c.z) : (w ? c.y : c.x);
  uint32_t* d = t < 4 ? f.b[t & 3] : f.a[t & 3];
  bf16x2 lo, hi;
  if (t >= 4 && FA == 1) {
    lo = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(x, s[t], false);
    hi = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(x, s[t], true);
  } else {
    lo = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(x, s[t], false);
    hi = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(x, s[t], true);
  }
  d[2 * w] = __builtin_bit_cast(uint32_t, lo);
  d[2 * w + 1] = __builtin_bit_cast(uint32_t, hi);
}

__device__ __forceinline__ bf16x8 as_bf16(const uint32_t (&w)[4]) {
  return __builtin_bit_cast(bf16x8, make_uint4(w[0], w[1], w[2], w[3]));
}

// One half: 4 MI MFMAs on `cur`; beside MFMA x the widening of word x of half
// NHALF of `raw` into `nxt`; if READ, beside the first ones the bytes of quarter RQ
// of stage R; if DMA, beside each the x-th DMA of block koff into stage W.  (MI =
// 3: two words and DMA are left for the first two.)
template <int FA, int NHALF, bool READ, int RQ, bool DMA, int MI>
__device__ __forceinline__ void prec_half(floatx16 (&acc)[MI][4], const Wide<MI>& cur, Wide<MI>& nxt,
                                          const Raw<MI>& raw, const float (&s)[4 + MI], const Stage<MI, 4>& R,
                                          Raw<MI>& rnext, Stage<MI, 4>& W, int64_t koff, const WidePos<MI>& w) {
  constexpr int kMfma = 4 * MI, kWords = 2 * (4 + MI);
#pragma unroll
  for (int x = 0; x < kMfma; ++x) {
    acc[x / 4][x % 4] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(as_bf16(cur.b[x % 4]), as_bf16(cur.a[x / 4]),
                                                                acc[x / 4][x % 4], 0, 0, 0);
#pragma unroll
    for (int y = x; y < kWords; y += kMfma) {
      widen_word<FA, NHALF>(raw, nxt, y >> 1, y & 1, s);
      if constexpr (DMA) wide_dma(W, w.src, koff, w.wave, y);
    }
    if constexpr (READ) {
      if (x < 4 + MI) read_raw<RQ>(R, rnext, x, w);
    }
    __builtin_amdgcn_sched_barrier(0);
  }
}

// MI = 4: 256 x 256 tiles; 3: 192 x 256.
template <int FA, int MI>
__global__ __launch_bounds__(kThreads, 1) void k_gemm_fp8_wide_f32(Params p) {
  __shared__ Stage<MI, 4> s0, s1;
  int kb0, nkb;
  const fp4lib::Fp8GemmArgs g = split_args(p.g, kb0, nkb);
  const WidePos<MI> w = wide_pos<MI>(p, g, blockIdx.x, kb0);

  floatx16 acc[MI][4];
#pragma unroll
  for (int mi = 0; mi < MI; ++mi)
#pragma unroll
    for (int ni = 0; ni < 4; ++ni) acc[mi][ni] = floatx16{};

  Raw<MI> r0, r1;
  Wide<MI> f0, f1;
  float s[4 + MI];            // block scales of B's and A's tiles
  auto set_scales = [&](uint32_t wa, uint32_t wb) {
#pragma unroll
    for (int t = 0; t < 4; ++t) s[t] = scale_of(wb, t);
#pragma unroll
    for (int t = 0; t < MI; ++t) s[4 + t] = scale_of(wa, t);
  };
  // Step kb on stage C: the bytes of its quarter 0 and its first half widened
  // are in registers, with its scales; then as in k_gemm_fp8_wide.
  auto step = [&](Stage<MI, 4>& C, Stage<MI, 4>& Nx, int kb) {
    const int k1 = min(kb + 1, nkb - 1), k2 = min(kb + 2, nkb - 1);
    const uint32_t na = wide_scales_a(w, k1 * g.s_kblk[0]);
    const uint32_t nb = load_scales<4>(w.psb + k1 * g.s_kblk[1]);
    const int64_t koff = static_cast<int64_t>(k2) * kStepBytes;
    prec_half<FA, 1, true, 1, false>(acc, f0, f1, r0, s, C, r1, C, 0, w);
    prec_half<FA, 0, false, 0, false>(acc, f1, f0, r1, s, C, r0, C, 0, w);
    prec_half<FA, 1, true, 2, false>(acc, f0, f1, r1, s, C, r0, C, 0, w);
    prec_half<FA, 0, false, 0, false>(acc, f1, f0, r0, s, C, r1, C, 0, w);
    prec_half<FA, 1, true, 3, false>(acc, f0, f1, r0, s, C, r1, C, 0, w);
    prec_half<FA, 0, false, 0, false>(acc, f1, f0, r1, s, C, r0, C, 0, w);
    wait_vmcnt<0>();
    ring_barrier();
    prec_half<FA, 1, true, 0, true>(acc, f0, f1, r1, s, Nx, r0, C, koff, w);
    set_scales(kb + 1 < nkb ? na : 0, kb + 1 < nkb ? nb : 0);
    prec_half<FA, 0, false, 0, false>(acc, f1, f0, r0, s, C, r1, C, 0, w);
  };
  if (nkb > 0) {
#pragma unroll
    for (int x = 0; x < 2 * MI + 8; ++x) wide_dma(s0, w.src, 0, w.wave, x);
    set_scales(wide_scales_a(w, 0), load_scales<4>(w.psb));
    wait_vmcnt<0>();
    ring_barrier();
#pragma unroll
    for (int x = 0; x < 2 * MI + 8; ++x) wide_dma(s1, w.src, nkb > 1 ? kStepBytes : 0, w.wave, x);
#pragma unroll
    for (int t = 0; t < 4 + MI; ++t) read_raw<0>(s0, r0, t, w);
#pragma unroll
    for (int t = 0; t < 2 * (4 + MI); ++t) widen_word<FA, 0>(r0, f0, t >> 1, t & 1, s);
    for (int kb = 0; kb < nkb; kb += 2) {
      step(s0, s1, kb);
      step(s1, s0, kb + 1);
    }
  }
  wait_vmcnt<0>();
  ring_barrier();
  constexpr int kBuf = 32 * (32 * 4 + 4);
  float* buf = reinterpret_cast<float*>(w.wave < 2 ? &s0 : &s1) + (w.wave & 1) * kBuf;
  static_assert(2 * kBuf * sizeof(float) <= sizeof(s0), "two epilogue buffers per stage");
  epilogue<MI, 4>(g, acc, w.m0 + w.wm * 32 * MI, w.n0 + w.wn * 128, w.lane, buf);
}

template <typename K>
void launch_kernel(K kernel, const fp4lib::Fp8GemmArgs& g, int bm, int bn, hipStream_t s, int max_wgs = 0) {
  Params p{g, static_cast<int>((g.M + bm - 1) / bm), static_cast<int>((g.N + bn - 1) / bn)};
  const int tiles = p.tiles_m * p.tiles_n;
  hipLaunchKernelGGL(kernel, dim3(max_wgs ? std::min(tiles, max_wgs) : tiles, g.splits), dim3(kThreads), 0,
                     s, p);
}

// D from the partial sums of `splits` workgroups per tile, in their order; a
// thread 4 columns.
__global__ __launch_bounds__(256) void k_gemm_fp8_join(fp4lib::Fp8GemmArgs g) {
  const int64_t np = part_pitch(g.N), per_row = np / 4, n = g.M * per_row, plane = g.M * np;
  for (int64_t id = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; id < n;
       id += static_cast<int64_t>(gridDim.x) * 256) {
    const int64_t row = id / per_row, col = (id - row * per_row) * 4;
    const float* src = g.part + row * np + col;
    float4_any v = *reinterpret_cast<const float4_any*>(src);
    int k = 1;
    for (; k + 3 <= g.splits; k += 3) {          // three loads at a time
      const float4_any a = *reinterpret_cast<const float4_any*>(src + k * plane),
                       b = *reinterpret_cast<const float4_any*>(src + (k + 1) * plane),
                       c = *reinterpret_cast<const float4_any*>(src + (k + 2) * plane);
      v += a;
      v += b;
      v += c;
    }
    for (; k < g.splits; ++k) v += *reinterpret_cast<const float4_any*>(src + k * plane);
    const bool whole = col + 4 <= g.N;
    if (g.d_bf16) {
      uint16_t* d = static_cast<uint16_t*>(g.D) + row * g.ldd + col;
      if (whole && !g.accumulate) {
        *reinterpret_cast<uint2_any*>(d) = uint2_any{fp8dev::pack_bf16(v.x, v.y), fp8dev::pack_bf16(v.z, v.w)};
        continue;
      }
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (col + e < g.N)
          d[e] = fp8dev::to_bf16(g.accumulate ? v[e] + __uint_as_float(static_cast<uint32_t>(d[e]) << 16) : v[e]);
    } else {
      float* d = static_cast<float*>(g.D) + row * g.ldd + col;
      if (whole) {
        if (g.accumulate) v += *reinterpret_cast<const float4_any*>(d);
        *reinterpret_cast<float4_any*>(d) = v;
        continue;
      }
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (col + e < g.N) d[e] = g.accumulate ? d[e] + v[e] : v[e];
    }
  }
}

// How a product runs: the kernel, and the workgroups that share a tile's K.
enum Kind { kRows, kTile64, kTile128, kTile192, kTile256, kNone };
struct Plan {
  Kind kind;
  int splits;
};

// A plan that a test asks for (fp4_selftest_set_fp8_plan): rows of a tile, 16 for
// the kernel for few rows; 0: none.  kNone where the kernel cannot run the product.
std::atomic<int> g_rows{0}, g_splits{1};

Plan asked_plan(const fp4lib::Fp8GemmArgs& g, int rows) {
  const int splits = g_splits.load();
  const Plan none{kNone, 1};
  if (splits > 1 && splits > g.nkb) return none;
  if (rows == 16) return g.M <= kMaxRows && splits == 1 ? Plan{kRows, 1} : none;
  if (rows >= 192 && (g.nkb == 0 || g.ld[0] >= (1 << 23) || g.ld[1] >= (1 << 23))) return none;
  if (rows == 192 && g.d_bf16) return none;
  return {rows == 64 ? kTile64 : rows == 128 ? kTile128 : rows == 192 ? kTile192 : kTile256, splits};
}

// The kernel and split (if the caller has a workspace: share) with the least
// estimated time.  A workgroup takes t1 us per K block while at most half of the
// chip's places for such workgroups are taken, and up to t2 when all are (two
// workgroups share a CU as soon as there are more than CUs; the clock falls with
// the power drawn); a round of workgroups has a fixed part (the persistent bf16
// kernel once); the codes come from HBM at 5 TB/s, which hides behind the work
// or hides it (a fourth-power mean joins the two); joining writes and reads the
// parts' fp32 sums.  The constants are a least-squares fit of the times of every
// kernel and split at 61 sizes (fp32 D: 63; M 17 .. 16384, N 320 .. 21504, K 1024 ..
// 21504; 256 CUs): by them the chosen one takes 1 % more than the best on average.
// Measured / estimated in us, bf16 D: M = N = K = 4096: 256-row tiles 55 / 60,
// 128-row 78 / 67; M = 1000, N = 4608, K = 12288: 256-row tiles by 3 67 / 76, 128-row
// unshared 91 / 89; M = 1160, N = 512, K = 6016: 64-row by 3 14.7 / 15.5, 128-row by 6
// 19.2 / 17.3; M = 32, N = 4096, K = 21504: 64-row by 8 21.3 / 27.0, by 3 32.7 / 31.7.
// fp32 D: M = 6144, N = 2048, K = 8192: 192-row 164 / 164, 256-row 167 / 166, 128-row
// 210 / 174; M = 8192, N = K = 4096: 256-row 200 / 195, 192-row 249 / 249, 128-row
// 239 / 223.
//
// Up to 16 rows of A: the kernel of gemm_fp8_rows.hip where 64 x 128 tiles would
// leave half the CUs idle (M = 1: N = 6144, K = 2048 6.4 against 8.8 us; N = 4096,
// K = 21504 17.0 against 19.4), tiles beyond (N = 21504, K = 4096: 19.0 against
// 22.8 us, for every row of A is then read by far fewer workgroups).  With more
// than 8 rows that reading counts where B is long enough to hide the tiles' second
// launch (M = 16: N = 4096, K = 21504 tiles 20.0, rows 23.0; N = 12288, K = 4608
// 14.5, 15.4; N = 2048, K = 6144 9.8, 7.9; M = 8: N = 4096, K = 21504 19.5, 19.7).
Plan plan_of(const fp4lib::Fp8GemmArgs& g, bool share) {
  if (const int rows = g_rows.load()) return asked_plan(g, rows);
  const int64_t cus = fp4lib::device_cu_count();
  auto tiles = [&](int64_t bm, int64_t bn) { return ((g.M + bm - 1) / bm) * ((g.N + bn - 1) / bn); };
  if (g.M <= kMaxRows && tiles(64, 128) * 2 < cus &&
      (g.M <= 8 || !share || static_cast<double>(g.N) * g.nkb * 128 < 48e6))
    return {kRows, 1};
  struct Cost {
    Kind kind;
    int bf16, bm, bn, per_cu;
    double t1, t2, fixed;
  };
  static constexpr Cost kCosts[] = {
      {kTile64, 0, 64, 128, 2, 0.58, 1.05, 3.3}, {kTile128, 0, 128, 128, 2, 0.98, 1.63, 3.5},
      {kTile192, 0, 192, 256, 1, 2.0, 2.43, 8},  {kTile256, 0, 256, 256, 1, 2.15, 2.73, 10},
      {kTile64, 1, 64, 128, 2, 0.38, 0.69, 3.3}, {kTile128, 1, 128, 128, 2, 0.66, 0.94, 3.5},
      {kTile256, 1, 256, 256, 1, 1.04, 1.6, 9}};
  const double size = static_cast<double>(g.M) * static_cast<double>(g.N);
  const double bytes = 4.0 + (static_cast<double>(g.M) + static_cast<double>(g.N)) * g.nkb * 128 / 5e6;
  static constexpr int kSplits[] = {1, 2, 3, 4, 6, 8, 12, 16};
  Plan best{kTile64, 1};
  double least = 0.0;
  for (const Cost& c : kCosts) {
    if (c.bf16 != (g.d_bf16 != 0)) continue;
    // 32-bit offsets within a tile's 256 rows, and no tail test for K = 0
    if (c.bn == 256 && (g.nkb == 0 || g.ld[0] >= (1 << 23) || g.ld[1] >= (1 << 23))) continue;
    for (int splits : kSplits) {
      if (splits > 1 && (!share || g.nkb < 4 * splits)) break;
      const int64_t n = tiles(c.bm, c.bn) * splits, slots = c.per_cu * cus, whole = n / slots, rest = n % slots;
      const double full = static_cast<double>(rest) / static_cast<double>(slots);
      const double more = full <= 0.5 ? 0.0 : c.per_cu == 2 ? 0.8 + 0.2 * (2.0 * full - 1.0) : 2.0 * full - 1.0;
      const double last = rest == 0 ? 0.0 : c.t1 + (c.t2 - c.t1) * more;
      const double blocks = static_cast<double>((g.nkb + splits - 1) / splits);
      const bool once = c.kind == kTile256 && c.bf16 && splits == 1;
      const double starts = once ? 1.0 : static_cast<double>(whole + (rest != 0));
      const double join = splits > 1 ? 3.5 + splits * size * 1.28e-6 : 0.0;
      const double work = (static_cast<double>(whole) * c.t2 + last) * blocks + starts * c.fixed;
      const double t = std::sqrt(std::sqrt(work * work * work * work + bytes * bytes * bytes * bytes)) + join;
      if (least == 0.0 || t < least) {
        least = t;
        best = {c.kind, splits};
      }
    }
  }
  return best;
}

template <int FA>
void run(const fp4lib::Fp8GemmArgs& g, Kind kind, hipStream_t s) {
  const int cus = fp4lib::device_cu_count();
  switch (kind) {
    case kRows:
      launch_rows(g, s);
      break;
    case kTile64:
      if (g.d_bf16) launch_kernel(k_gemm_fp8<FA, false, 1, 2, 3>, g, 64, 128, s);
      else launch_kernel(k_gemm_fp8<FA, true, 1, 2, 3>, g, 64, 128, s);
      break;
    case kTile128:
      if (g.d_bf16) launch_kernel(k_gemm_fp8<FA, false, 2, 2, 2>, g, 128, 128, s);
      else launch_kernel(k_gemm_fp8<FA, true, 2, 2, 2>, g, 128, 128, s);
      break;
    case kTile192:
      launch_kernel(k_gemm_fp8_wide_f32<FA, 3>, g, 192, 256, s);
      break;
    case kTile256:
      if (!g.d_bf16) launch_kernel(k_gemm_fp8_wide_f32<FA, 4>, g, 256, 256, s);
      else if (!g.accumulate && g.splits == 1)
        launch_kernel(k_gemm_fp8_wide_loop<FA>, g, 256, 256, s, cus);
      else launch_kernel(k_gemm_fp8_wide<FA>, g, 256, 256, s);
      break;
    case kNone:
      break;
  }
}

}  // namespace
}  // namespace fp8gemm

namespace fp4lib {

static int64_t part_bytes(const Fp8GemmArgs& g, int splits) {
  return splits > 1 ? splits * g.M * fp8gemm::part_pitch(g.N) * 4 : 0;
}

int64_t gemm_fp8_workspace(const Fp8GemmArgs& g) { return part_bytes(g, fp8gemm::plan_of(g, true).splits); }

void set_fp8_plan(int tile_rows, int splits) {
  fp8gemm::g_rows.store(tile_rows);
  fp8gemm::g_splits.store(splits);
}

hipError_t launch_gemm_fp8(const Fp8GemmArgs& args, hipStream_t s) {
  Fp8GemmArgs g = args;
  fp8gemm::Plan p = fp8gemm::plan_of(g, g.part != nullptr);
  if (part_bytes(g, p.splits) > g.part_bytes) p = fp8gemm::plan_of(g, false);
  // (an asked plan alone can be neither of the two)
  if (p.kind == fp8gemm::kNone || part_bytes(g, p.splits) > g.part_bytes) return hipErrorInvalidValue;
  g.splits = p.splits;
  if (g.a_e5m2) fp8gemm::run<1>(g, p.kind, s);
  else fp8gemm::run<0>(g, p.kind, s);
  if (g.splits > 1) {
    const int64_t n = g.M * fp8gemm::part_pitch(g.N) / 4;
    const int64_t cap = static_cast<int64_t>(device_cu_count()) * 8, want = (n + 255) / 256;
    hipLaunchKernelGGL(fp8gemm::k_gemm_fp8_join, dim3(static_cast<uint32_t>(want < cap ? want : cap)),
                       dim3(256), 0, s, g);
  }
  return hipGetLastError();
}

}  // namespace fp4lib
