// Shared by the FP8 GEMM's translation units: codes and scales to bf16, and
// the launchers.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fp4_internal.hpp"
#include "fp8_common.hpp"

namespace fp8gemm {

using fp8dev::bf16x2;
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

// 8 codes (two words) with their block's scale as bf16: exact from 2^-126 to below
// 2^128 (a code of 2^-9 with the scale 2^-127 is below bf16's subnormals).
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

// ------------------------------------------------- products split along K --
// With few output tiles, `splits` workgroups (blockIdx.y) share a tile's K
// blocks; each writes its fp32 sums to its part of the caller's workspace,
// [splits][M][part_pitch(N)], and k_gemm_fp8_join adds them in order.
__host__ __device__ __forceinline__ int64_t part_pitch(int64_t n) { return (n + 3) & ~int64_t(3); }

// This workgroup's arguments: blocks kb0 .. kb0 + nkb - 1 and, if split, its
// part of the workspace as D.
__device__ __forceinline__ fp4lib::Fp8GemmArgs split_args(const fp4lib::Fp8GemmArgs& g, int& kb0, int& nkb) {
  fp4lib::Fp8GemmArgs r = g;
  const int n = static_cast<int>(g.nkb), k = blockIdx.y;
  kb0 = static_cast<int>(static_cast<int64_t>(n) * k / g.splits);
  nkb = static_cast<int>(static_cast<int64_t>(n) * (k + 1) / g.splits) - kb0;
  if (g.splits > 1) {
    r.D = g.part + k * g.M * part_pitch(g.N);
    r.ldd = part_pitch(g.N);
    r.d_bf16 = 0;
    r.accumulate = 0;
  }
  return r;
}

// Few rows of A (gemm_fp8_rows.hip): M at most kMaxRows.
constexpr int kMaxRows = 16;
void launch_rows(const fp4lib::Fp8GemmArgs& g, hipStream_t s);

}  // namespace fp8gemm
