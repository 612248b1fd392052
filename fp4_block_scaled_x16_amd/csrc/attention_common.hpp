// Shared by the attention kernels: how a request's tokens are shared among
// workgroups, and the launchers of the formats.
#pragma once

#include "kv_common.hpp"

namespace fp4attn {

constexpr int kWaves = 4, kTile = 32;
constexpr int kWideWaves = 8, kWideDim = 128; // of a workgroup that has a short request alone, heads up to 128
constexpr int kLoneTokens = 384;              // many requests of up to as many: one wave each
constexpr int kMaxParts = 512;
constexpr int kStep = kWaves * kTile;         // tokens that a workgroup takes at once

// Waves on a SIMD: as many as the registers of a lane's part of out and of the tiles
// under way leave room for (128 elements: 4 instead of 3 spills 27 registers and takes
// 220 instead of 128 us for 64 requests of up to 8192 tokens; 256: 3 instead of 2, 150
// instead of 66 us for 16 of 8000).
__host__ __device__ constexpr int waves_per_simd(int head_dim) { return head_dim == 64 ? 4 : head_dim == 128 ? 3 : 2; }

// Requests whose parts may go by their lengths (a wave looks at 64 of these at once; with
// 512 what it costs is more than it gives: 500 of up to 3000 MXFP4 tokens 177 -> 188 us).
constexpr int kPlanned = 256;

// Tokens of a part (the last may have fewer) of a request of len tokens where the parts
// do not go by the lengths: at most a.splits parts of at least a.min_part, whole steps each.
__host__ __device__ __forceinline__ int part_tokens(int len, const fp4lib::AttnArgs& a) {
  const int even = (len + a.splits - 1) / a.splits;
  return even <= a.min_part ? a.min_part : (even + kStep - 1) / kStep * kStep;
}

__device__ __forceinline__ int tokens_of(const fp4lib::AttnArgs& a, int request) {
  const int64_t room = static_cast<int64_t>(a.table_width) << a.cache.page_shift;
  const int len = a.lens[request];
  return len < 0 ? 0 : len > room ? static_cast<int>(room) : len;
}

// The workspace: the parts' sums [key head][part][query head of it][head_dim], behind
// them each one's maximum (in powers of two) and sum of p, and behind these each request's
// first part and number of parts.
__device__ __forceinline__ float2* part_sums(const fp4lib::AttnArgs& a) {
  return reinterpret_cast<float2*>(a.part + a.items * a.q.heads * a.cache.head_dim);
}
__device__ __forceinline__ int2* request_parts(const fp4lib::AttnArgs& a) {
  return reinterpret_cast<int2*>(part_sums(a) + a.items * a.q.heads);
}

}  // namespace fp4attn

namespace fp4lib {
template <int FMT>
hipError_t launch_attention_fmt(const AttnArgs& a, uint32_t grid, hipStream_t s);
}  // namespace fp4lib
