// Shared by the attention kernels: the requests' lengths, where the workspace holds the
// parts' sums, and the launchers of the formats.
#pragma once

#include "attention_plan.hpp"
#include "kv_common.hpp"

namespace fp4attn {

// Waves on a SIMD: as many as the registers of a lane's part of out and of the tiles
// under way leave room for (128 elements: 4 instead of 3 spills 27 registers and takes
// 220 instead of 128 us for 64 requests of up to 8192 tokens; 256: 3 instead of 2, 150
// instead of 66 us for 16 of 8000).
__host__ __device__ constexpr int waves_per_simd(int head_dim) { return head_dim == 64 ? 4 : head_dim == 128 ? 3 : 2; }

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
