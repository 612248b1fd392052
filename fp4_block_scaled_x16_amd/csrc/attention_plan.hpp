// How requests' tokens are shared among workgroups: the plan that the host makes from
// the sizes, and the arithmetic by which each workgroup finds its part from the lengths
// (attention.hip: planned_item).  Both are here, and plain C++, since they have to agree: the
// launch and the workspace hold as many parts as the plan says, whatever the lengths.
#pragma once

#include <algorithm>

#include "kv_internal.hpp"

namespace fp4attn {

constexpr int kWaves = 4, kTile = 32;
constexpr int kWideWaves = 8, kWideDim = 128; // of a workgroup that has a short request alone, heads up to 128
constexpr int kLoneTokens = 384;              // many requests of up to as many: one wave each
constexpr int kMaxParts = 512;
constexpr int kStep = kWaves * kTile;         // tokens that a workgroup takes at once

// Requests whose parts may go by their lengths (a wave looks at 64 of these at once; with
// 512 what it costs is more than it gives: 500 of up to 3000 MXFP4 tokens 177 -> 188 us).
// In tables with room for 131072 tokens each, 256 / 257 requests of up to 3000 MXFP8 tokens take
// 139 / 170 us, of up to 500 tokens 40 / 39; 400 of up to 500 87, with room for 500 each 54.
constexpr int kPlanned = 256;

// Tokens of a part (the last may have fewer) of a request of len tokens where the parts
// do not go by the lengths: at most a.splits parts of at least a.min_part, whole steps each.
__host__ __device__ __forceinline__ int part_tokens(int len, const fp4lib::AttnArgs& a) {
  const int even = (len + a.splits - 1) / a.splits;
  return even <= a.min_part ? a.min_part : (even + kStep - 1) / kStep * kStep;
}

// x / d rounded down, for x below 2^24 and d of 1 or more, from a reciprocal that is at most
// a step of fp32 off (and exact where d is a power of two: v_rcp_f32).  For d in (2^k, 2^(k+1)) that
// step moves the product by up to 2^-k, rounding it by up to 2^-(k+1): by less than 1 together,
// which one correction makes good.
__host__ __device__ __forceinline__ int quotient(int x, int d, float reciprocal) {
  const int q = static_cast<int>(static_cast<float>(x) * reciprocal);
  const int rest = x - q * d;
  return rest < 0 ? q - 1 : rest >= d ? q + 1 : q;
}
__host__ __device__ __forceinline__ int quotient(int x, int d) {
#ifdef __HIP_DEVICE_COMPILE__
  return quotient(x, d, __builtin_amdgcn_rcpf(static_cast<float>(d)));
#else
  return quotient(x, d, 1.0f / static_cast<float>(d));
#endif
}

// Lengths, and those of parts, in steps (kStep tokens): a request has at most this many.
constexpr int kMostSteps = 1 << 23;

// n / d rounded up, exact below kMostSteps, and else too much by a step; kMostSteps at most.
__host__ __device__ __forceinline__ int share(uint32_t n, int d) {
  if (n < static_cast<uint32_t>(kMostSteps)) return quotient(n + d - 1, d);
  const int q = static_cast<int>(n / static_cast<uint32_t>(d)) + 1;
  return q < kMostSteps ? q : kMostSteps;
}

// Parts of `step` steps that there are `want` of all requests' tokens together, but for
// each request's rounding up: at most want + requests.
struct Shares {
  int want, step;
};

// For `all` steps of all requests: target[0] parts, fewer (target[1]: one to a CU) if they were
// short.
template <int D>
__host__ __device__ __forceinline__ Shares first_shares(uint32_t all, const fp4lib::AttnArgs& a) {
  Shares s{a.target[0], 0};
  s.step = share(all, s.want);
  if (D == 64 && s.step < 16) {
    s.want = s.want > 3 ? s.want / 2 : 1;
    s.step = share(all, s.want);
  }
  if (s.step < (D == 64 ? 5 : 8)) {
    s.want = a.target[1];
    s.step = share(all, s.want);
  }
  const int least = a.min_part / kStep;
  if (s.step < least) s.step = least;
  return s;
}

// The step with which `count` parts, more than `want` and below twice as many, become about
// `want`: step * count / want, rounded up.  (The product is not formed: it may pass 32 bits.)
// Never below `step`, so no request gets more parts than it had.
__host__ __device__ __forceinline__ int longer_step(int step, int count, int want) {
  const int whole = quotient(step, want), rest = step - whole * want;
  const int longer = whole * count + quotient(rest * count + want - 1, want);
  return longer < kMostSteps ? longer : kMostSteps;
}

// Parts of a request of `size` steps, and the steps of each.
__host__ __device__ __forceinline__ int parts_of(int size, int step) {
  const int n = quotient(size + step - 1, step);
  return n > 1 ? n : 1;
}
__host__ __device__ __forceinline__ int steps_of(int size, int parts) { return quotient(size + parts - 1, parts); }

// At most `splits` parts of a request (and where they go by the lengths, no more than
// target[0] together but for each request's rounding up).
inline void set_parts(fp4lib::AttnArgs& a, int splits) {
  a.splits = splits;
  a.items = static_cast<int64_t>(a.requests) * splits;
  if (a.planned && splits > 1) a.items = std::min<int64_t>(a.items, a.requests + a.target[0]);
}

// How a request's tokens are shared.  Up to kPlanned requests' parts go by their lengths,
// which are on the device (attention.hip: planned_item): the page table may have room for far
// more (64 requests of up to 500 MXFP8 tokens take 16 us with room for 131072 each; parts
// planned from the room took 57).  Two workgroups on every CU (heads of 64: four), if that
// leaves a part 8 steps of 128 tokens, else as many as there are CUs, but not more: 4 requests of
// 120000 NVFP4 tokens in 8 / 16 / 24 / 64 parts 126 / 109 / 112 / 116 us, 1 of 30000 FP8 tokens in
// 32 / 64 / 128 parts 17.4 / 19.2 / 22, 6 of 3084 MXFP8 tokens of 8 heads in 4 / 5 / 6 / 8 parts
// 16.0 / 15.2 / 18.9 / 18.2.  Against parts alike for every request: 16 of up to 30000 FP8 tokens
// 104 -> 95, 200 of up to 4000 MXFP8 tokens 159 -> 144, 1 of 30000 18.4 -> 19.1.
// More requests: two parts of over 2048 tokens even out lengths (300 of up to 2500 of 2 heads
// 55 -> 51), up to eight of 4096, while the workgroups are not too many: where the table has
// more room than that, most of them find nothing to do (1000 of up to 200 MXFP4 tokens with
// room for 131072 each 241 -> 38).  Where one part per request will do, the join is not launched
// (72 of 551 tokens of 2 heads in 1 / 2 parts 11.1 / 15.6, 256 of up to 1024 15.4 / 21.6).
// The figures are from kernels that took p in two parts; a third adds up to 7 % to either side.
inline void plan(fp4lib::AttnArgs& a, int64_t cu, int forced) {
  const int64_t room = static_cast<int64_t>(a.table_width) << a.cache.page_shift;
  a.group = a.q.heads / a.cache.heads;
  a.tiles = a.group <= 8 ? 1 : (a.group + 15) / 16;
  const int64_t each = static_cast<int64_t>(a.requests) * a.cache.heads * a.tiles;
  const int64_t slots = 2 * cu;
  const int64_t most = (room + kStep - 1) / kStep, full = slots / each > 1 ? slots / each : 1;
  int64_t want = full;
  if (room < 1024 * full) want = cu / each;
  auto at_most = [&](int64_t tokens, int64_t cap) { return std::min((room + tokens - 1) / tokens, cap); };
  want = std::max({want, at_most(2048, 2 * full), at_most(4096, 8 * full)});
  if (a.requests > kPlanned) want = std::min(want, std::max<int64_t>(1, 16 * slots / each));
  a.min_part = 2 * each >= slots ? 4 * kStep : kStep;
  if (forced) {
    want = forced;
    a.min_part = kStep;
  }
  // More codes than half of the 256 MB last-level cache do not come from there again:
  // they are read past it (64 requests of up to 8192 MXFP8 tokens 122 -> 115 us, 32 of 6000
  // FP8 tokens, 197 MB, 45 -> 40; but 1 of 30000, 61 MB, 17.9 -> 19.1 when they are).
  // More than 16 query heads to a key head: several workgroups read the same codes.
  const int row = a.cache.head_dim >> (a.cache.fmt != fp4lib::kKvFp8 && a.cache.fmt != fp4lib::kKvMx8);
  a.stream = a.tiles == 1 && 2.0 * room * a.requests * a.cache.heads * row > 0x1p27;
  want = want > most ? most : want;
  // Short requests whole, eight waves each: one launch instead of two (1 of 200 / 500 / 1000
  // FP8 tokens 7.6 / 9.5 / 12.4 us instead of 8.9 / 8.8 / 9.4, and 8.3 / 10.0 / 12.8 instead of
  // 11.6 / 11.7 / 11.8 a call where the host's part counts; heads of 64, MXFP4: 5.5 / 6.5 / 8.4
  // instead of 7.3 / 7.3 / 7.9, and 8.2 / 8.1 / 9.1 instead of 12).
  // Many of them, a wave each: no meeting at the end (8 heads of 128: 2000 of up to 64 FP8 tokens with
  // 4 / 2 / 1 waves 98 / 59 / 50 us, 2000 of up to 256 MXFP4 tokens 117 / 83 / 75, 128 of up to 200 MXFP8
  // tokens 14.4 / - / 11.7; but 256 of up to 512 MXFP4 tokens of 4 heads of 64 11.8 / - / 15.1, and
  // 512 of up to 1024 MXFP4 tokens 66 / 69 / 78).
  const int steps = a.cache.head_dim == 64 ? 4 : 2;
  a.waves = kWaves;
  if (!forced) {
    if (4 * room <= each && room <= kLoneTokens) {
      a.waves = 1;
      want = 1;
    } else if (a.cache.head_dim <= kWideDim && want > 1 && room <= steps * kWideWaves * kTile) {
      a.waves = kWideWaves;
      want = 1;
    }
  }
  const int64_t ht = static_cast<int64_t>(a.cache.heads) * a.tiles, first = a.cache.head_dim == 64 ? 4 * cu : slots;
  a.target[0] = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(kMaxParts, first / ht)));
  a.target[1] = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(kMaxParts, cu / ht)));
  a.planned = a.requests <= kPlanned && a.waves == kWaves && !forced && (want > 1 || each > cu);
  if (a.planned && want > 1) want = std::min<int64_t>(most, a.target[0]);
  set_parts(a, static_cast<int>(want < 1 ? 1 : want > kMaxParts ? kMaxParts : want));
}

inline int64_t part_bytes(const fp4lib::AttnArgs& a) {
  return a.splits <= 1 ? 0
                       : a.items * a.q.heads * (a.cache.head_dim + 2) * static_cast<int64_t>(sizeof(float)) +
                             a.requests * static_cast<int64_t>(sizeof(int2));
}

// Workgroups of a launch: a grid has fewer than 2^32 threads, and the kernel divides a part's
// number, which is smaller, by up to 1024 with a product.
constexpr int64_t kMostGroups = int64_t(1) << 22;

// Calls launch with the arguments of each launch of planned ones, until one fails.
template <typename F>
hipError_t by_launches(const fp4lib::AttnArgs& planned, F&& launch) {
  fp4lib::AttnArgs a = planned;
  const int64_t groups = static_cast<int64_t>(a.cache.heads) * a.tiles * (a.items / a.requests);
  const int most = a.planned ? a.requests : static_cast<int>(groups < kMostGroups ? kMostGroups / groups : 1);
  const int64_t row = static_cast<int64_t>(a.q.heads) * a.cache.head_dim * (a.out_f32 ? 4 : 2);
  for (int64_t first = 0; first < planned.requests; first += most) {         // (an int may pass 2^31)
    a.requests = static_cast<int>(std::min<int64_t>(planned.requests - first, most));
    if (!a.planned) set_parts(a, a.splits);
    a.q.x = planned.q.x + first * planned.q.token;
    a.table = planned.table + first * planned.table_stride;
    a.lens = planned.lens + first;
    a.out = static_cast<uint8_t*>(planned.out) + first * row;
    a.lse = planned.lse ? planned.lse + first * a.q.heads : nullptr;
    const hipError_t e = launch(a);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace fp4attn
