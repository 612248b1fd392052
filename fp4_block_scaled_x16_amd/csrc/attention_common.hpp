// Shared by the attention kernels: how a request's tokens are shared among
// workgroups, and the launchers of the formats.
#pragma once

#include "kv_common.hpp"

namespace fp4attn {

constexpr int kWaves = 4, kTile = 32;
constexpr int kMinPart = kWaves * kTile;      // tokens of a part: at least a tile for each wave

// Tokens of a part (the last may have fewer) of a request of len tokens in at
// most `splits` parts.
__host__ __device__ __forceinline__ int part_tokens(int len, int splits) {
  const int even = (len + splits - 1) / splits;
  return even <= kMinPart ? kMinPart : (even + kMinPart - 1) / kMinPart * kMinPart;
}

__device__ __forceinline__ int tokens_of(const fp4lib::AttnArgs& a, int request) {
  const int64_t room = static_cast<int64_t>(a.table_width) << a.cache.page_shift;
  const int len = a.lens[request];
  return len < 0 ? 0 : len > room ? static_cast<int>(room) : len;
}

}  // namespace fp4attn

namespace fp4lib {
template <int FMT>
hipError_t launch_attention_fmt(const AttnArgs& a, uint32_t grid, hipStream_t s);
}  // namespace fp4lib
