// FP8 block-128 GEMM with few rows of A (a token, a batch of decoding
// requests): D[M, N] for M <= 16.
//
// Bound by reading B once: at M = 1, N = 4096, K = 21504 its 88 MB (16.9 us, 5.2
// TB/s).  No LDS staging, since no byte of B is used twice: every lane loads its
// own operands of v_mfma_f32_16x16x32_bf16 from global memory (the codes widened
// as for an fp32 D in gemm_fp8.hip; the arithmetic is free here, so bf16 outputs
// have it too).  A workgroup owns 16 rows of B; its waves take turns
// along K, so that a few rows of B still put 16 waves of loads in flight on a CU,
// and their sums meet in LDS in a fixed order.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fp4_internal.hpp"
#include "fp8_common.hpp"
#include "gemm_fp8_common.hpp"

namespace fp8gemm {
namespace {

typedef float floatx4 __attribute__((ext_vector_type(4)));

constexpr int kU = 4;             // K blocks a wave loads at once
constexpr int kMaxWaves = 16;

template <int FA>
__global__ __launch_bounds__(64 * kMaxWaves) void k_gemm_fp8_rows(fp4lib::Fp8GemmArgs g) {
  extern __shared__ __attribute__((aligned(16))) float part[];   // [waves][16 rows of A][16 of B]
  const int lane = threadIdx.x & 63, waves = blockDim.x >> 6;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int i = lane & 15, q = lane >> 4;
  const int64_t n0 = static_cast<int64_t>(blockIdx.x) * 16;
  const int nkb = static_cast<int>(g.nkb);

  // Lane (i, q) has 16 bytes at 16 q and at 64 + 16 q of each block of row i.
  // Rows outside the operands read their last row; nothing of theirs is stored.
  const int64_t ra = min(static_cast<int64_t>(i), g.M - 1), rb = min(n0 + i, g.N - 1);
  const uint8_t* pa = g.codes[0] + ra * g.ld[0] + 16 * q;
  const uint8_t* pb = g.codes[1] + rb * g.ld[1] + 16 * q;
  const uint8_t* sa = g.scales[0] + ra;
  const uint8_t* sb = g.scales[1] + rb;

  floatx4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int k0 = wave * kU; k0 < nkb; k0 += waves * kU) {
    uint4 b[kU][2], a[kU][2];
    uint32_t eb[kU], ea[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      // past the end: the last block again, not multiplied
      const int64_t kb = min(k0 + u, nkb - 1);
      b[u][0] = *reinterpret_cast<const uint4*>(pb + kb * 128);
      b[u][1] = *reinterpret_cast<const uint4*>(pb + kb * 128 + 64);
      eb[u] = sb[kb * g.s_kblk[1]];
      a[u][0] = *reinterpret_cast<const uint4*>(pa + kb * 128);
      a[u][1] = *reinterpret_cast<const uint4*>(pa + kb * 128 + 64);
      ea[u] = sa[kb * g.s_kblk[0]];
    }
    // every load of the blocks is issued before the first is waited for
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      if (k0 + u >= nkb) break;
      const float fa = scale_of(ea[u], 0), fb = scale_of(eb[u], 0);
#pragma unroll
      for (int p = 0; p < 4; ++p) {          // 8 bytes of each half of the block
        const uint4 &x = b[u][p >> 1], &y = a[u][p >> 1];
        acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
            widen8<false>(p & 1 ? x.z : x.x, p & 1 ? x.w : x.y, fb),
            widen8<FA == 1>(p & 1 ? y.z : y.x, p & 1 ? y.w : y.y, fa), acc, 0, 0, 0);
      }
    }
  }

  // lane (i, q): row i of A's tile, rows 4 q .. 4 q + 3 of B's
  *reinterpret_cast<floatx4*>(part + wave * 256 + i * 16 + 4 * q) = acc;
  __syncthreads();
  const int o = threadIdx.x;
  const int64_t row = o / 16, col = n0 + o % 16;
  if (o >= 256 || row >= g.M || col >= g.N) return;
  float v = 0.0f;
  for (int w = 0; w < waves; ++w) v += part[w * 256 + o];
  if (g.d_bf16) {
    uint16_t* d = static_cast<uint16_t*>(g.D) + row * g.ldd + col;
    if (g.accumulate) v += __uint_as_float(static_cast<uint32_t>(*d) << 16);
    *d = fp8dev::to_bf16(v);
  } else {
    float* d = static_cast<float*>(g.D) + row * g.ldd + col;
    *d = g.accumulate ? *d + v : v;
  }
}

}  // namespace

// Waves per workgroup: enough for 16 on every CU where the rows of B are few,
// and no more than the K blocks give work to; at least 4 (256 outputs).
void launch_rows(const fp4lib::Fp8GemmArgs& g, hipStream_t s) {
  const int64_t tiles = (g.N + 15) / 16, want = kMaxWaves * fp4lib::device_cu_count() / tiles;
  int waves = 4;
  while (waves < kMaxWaves && waves < want && waves * kU < g.nkb) waves *= 2;
  const dim3 grid(static_cast<uint32_t>(tiles)), block(64 * waves);
  if (g.a_e5m2) hipLaunchKernelGGL(k_gemm_fp8_rows<1>, grid, block, waves * 1024, s, g);
  else hipLaunchKernelGGL(k_gemm_fp8_rows<0>, grid, block, waves * 1024, s, g);
}

}  // namespace fp8gemm
