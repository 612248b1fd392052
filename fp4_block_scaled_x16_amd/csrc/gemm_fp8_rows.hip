// FP8 block-128 GEMM with few rows of A (a token, a batch of decoding
// requests): D[M, N] for M <= 64.
//
// Bound by reading B once: at M = 32, N = 4096, K = 21504 its 88 MB.  No LDS
// staging, since no byte of B is used twice: every lane loads its own operands
// of v_mfma_f32_16x16x32_bf16 from global memory (the codes widened exactly, as
// for an fp32 D in gemm_fp8.hip; the arithmetic is free here, so bf16 outputs
// have it too).  A workgroup owns 16 NT rows of B; its waves take turns along K,
// so that a few rows of B still put 16 waves of loads in flight on a CU,
// and their sums meet in LDS in a fixed order.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fp4_internal.hpp"
#include "fp8_common.hpp"
#include "gemm_fp8_common.hpp"

namespace fp8gemm {
namespace {

typedef float floatx4 __attribute__((ext_vector_type(4)));

// MT, NT: 16-row tiles of A and B; U: K blocks a wave loads at once.
template <int FA, int MT, int NT, int U>
__global__ __launch_bounds__(64 * (MT == 1 ? 16 : 8)) void k_gemm_fp8_rows(fp4lib::Fp8GemmArgs args) {
  int kb0, nkb;
  const fp4lib::Fp8GemmArgs g = split_args(args, kb0, nkb);
  extern __shared__ __attribute__((aligned(16))) float part[];   // [waves][16 MT][16 NT]
  const int lane = threadIdx.x & 63, waves = blockDim.x >> 6;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int i = lane & 15, q = lane >> 4;
  const int64_t n0 = static_cast<int64_t>(blockIdx.x) * (16 * NT);

  // Lane (i, q) has 16 bytes at 16 q and at 64 + 16 q of each block of row i.
  // Rows outside the operands read their last row; nothing of theirs is stored.
  const uint8_t *pa[MT], *pb[NT], *sa[MT], *sb[NT];
#pragma unroll
  for (int t = 0; t < MT; ++t) {
    const int64_t r = min(static_cast<int64_t>(16 * t + i), g.M - 1);
    pa[t] = g.codes[0] + r * g.ld[0] + static_cast<int64_t>(kb0) * 128 + 16 * q;
    sa[t] = g.scales[0] + kb0 * g.s_kblk[0] + r;
  }
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int64_t r = min(n0 + 16 * t + i, g.N - 1);
    pb[t] = g.codes[1] + r * g.ld[1] + static_cast<int64_t>(kb0) * 128 + 16 * q;
    sb[t] = g.scales[1] + kb0 * g.s_kblk[1] + r;
  }

  floatx4 acc[MT][NT];
#pragma unroll
  for (int t = 0; t < MT; ++t)
#pragma unroll
    for (int u = 0; u < NT; ++u) acc[t][u] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};

  for (int k0 = wave * U; k0 < nkb; k0 += waves * U) {
    uint4 b[U][NT][2], a[U][MT][2];
    uint32_t eb[U][NT], ea[U][MT];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      // past the end: the last block again, not multiplied
      const int64_t kb = min(k0 + u, nkb - 1);
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        b[u][t][0] = *reinterpret_cast<const uint4*>(pb[t] + kb * 128);
        b[u][t][1] = *reinterpret_cast<const uint4*>(pb[t] + kb * 128 + 64);
        eb[u][t] = sb[t][kb * g.s_kblk[1]];
      }
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        a[u][t][0] = *reinterpret_cast<const uint4*>(pa[t] + kb * 128);
        a[u][t][1] = *reinterpret_cast<const uint4*>(pa[t] + kb * 128 + 64);
        ea[u][t] = sa[t][kb * g.s_kblk[0]];
      }
    }
    // every load of the U blocks is issued before the first is waited for
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (k0 + u >= nkb) break;
#pragma unroll
      for (int p = 0; p < 4; ++p) {          // 8 bytes of each half of the block
        bf16x8 wa[MT], wb[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const uint4& c = b[u][t][p >> 1];
          wb[t] = widen8<false>(p & 1 ? c.z : c.x, p & 1 ? c.w : c.y, scale_of(eb[u][t], 0));
        }
#pragma unroll
        for (int t = 0; t < MT; ++t) {
          const uint4& c = a[u][t][p >> 1];
          wa[t] = widen8<FA == 1>(p & 1 ? c.z : c.x, p & 1 ? c.w : c.y, scale_of(ea[u][t], 0));
        }
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
          for (int v = 0; v < NT; ++v)
            acc[t][v] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wb[v], wa[t], acc[t][v], 0, 0, 0);
      }
    }
  }

  // lane (i, q): row i of A's tile, rows 4 q .. 4 q + 3 of B's
  constexpr int W = 16 * NT, P = 16 * MT * W;
#pragma unroll
  for (int t = 0; t < MT; ++t)
#pragma unroll
    for (int v = 0; v < NT; ++v)
      *reinterpret_cast<floatx4*>(part + wave * P + (16 * t + i) * W + 16 * v + 4 * q) = acc[t][v];
  __syncthreads();
  for (int o = threadIdx.x; o < P; o += blockDim.x) {
    const int64_t row = o / W, col = n0 + o % W;
    if (row >= g.M || col >= g.N) continue;
    float v = 0.0f;
    for (int w = 0; w < waves; ++w) v += part[w * P + o];
    if (g.d_bf16) {
      uint16_t* d = static_cast<uint16_t*>(g.D) + row * g.ldd + col;
      if (g.accumulate) v += __uint_as_float(static_cast<uint32_t>(*d) << 16);
      *d = fp8dev::to_bf16(v);
    } else {
      float* d = static_cast<float*>(g.D) + row * g.ldd + col;
      *d = g.accumulate ? *d + v : v;
    }
  }
}

// Workgroups and waves for one variant.
struct Shape {
  int64_t tiles;
  int splits, waves;
};

// Enough waves for 16 on every CU: first along K within the workgroup (at
// most kMax of them, 64 KiB of partial sums), then along K over workgroups,
// each wave keeping at least 2 blocks.
template <int MT, int NT>
Shape shape_of(const fp4lib::Fp8GemmArgs& g) {
  constexpr int kMax = MT == 1 ? 16 : 8;
  Shape p{(g.N + 16 * NT - 1) / (16 * NT), 1, 4};
  const int64_t want = 16 * fp4lib::device_cu_count() / p.tiles;
  while (p.waves < kMax && p.waves * MT * NT * 2 <= 64 && p.waves < want && p.waves * 4 <= g.nkb) p.waves *= 2;
  while (p.splits < 16 && p.splits * p.waves * 2 <= want && p.splits * p.waves * 4 <= g.nkb) p.splits *= 2;
  return p;
}

template <int FA, int MT, int NT, int U>
void launch(const fp4lib::Fp8GemmArgs& g, hipStream_t s) {
  const Shape p = shape_of<MT, NT>(g);
  hipLaunchKernelGGL((k_gemm_fp8_rows<FA, MT, NT, U>), dim3(static_cast<uint32_t>(p.tiles), g.splits),
                     dim3(64 * p.waves), static_cast<size_t>(p.waves) * MT * NT * 1024, s, g);
}

template <int FA>
void by_rows(const fp4lib::Fp8GemmArgs& g, hipStream_t s) {
  if (g.M <= 16) launch<FA, 1, 1, 4>(g, s);
  else if (g.M <= 32) launch<FA, 2, 4, 2>(g, s);
  else launch<FA, 4, 4, 1>(g, s);
}

}  // namespace

int rows_splits(const fp4lib::Fp8GemmArgs& g) {
  return g.M <= 16 ? shape_of<1, 1>(g).splits : g.M <= 32 ? shape_of<2, 4>(g).splits : shape_of<4, 4>(g).splits;
}

void launch_rows(const fp4lib::Fp8GemmArgs& g, hipStream_t s) {
  if (g.a_e5m2) by_rows<1>(g, s);
  else by_rows<0>(g, s);
}

}  // namespace fp8gemm
