// Launch of the attention of one new token per request (attention.hip): how many
// parts a request's tokens are shared among, and the kernel that joins them.
#include <atomic>

#include "attention_common.hpp"

using namespace kvdev;
using namespace fp4attn;

namespace {

constexpr float kLog2e = 1.44269504088896340736f;

// The parts of a request, in order: a workgroup per query head, D / 2 threads
// (two elements each) times 8 shares of the parts.
template <int D>
__global__ __launch_bounds__(4 * D) void k_attention_join(fp4lib::AttnArgs a) {
  constexpr int kShares = 8, kPair = D / 2;
  __shared__ float2 sums[kShares - 1][kPair];
  __shared__ float totals[kShares - 1];
  const int64_t row = blockIdx.x;
  const int request = static_cast<int>(row / a.q.heads);
  const int len = tokens_of(a, request), per = part_tokens(len, a.splits);
  const int parts = (len + per - 1) / per;
  if (parts <= 1) return;
  const int share = threadIdx.x / kPair, d = threadIdx.x % kPair * 2;
  const float* p = a.part + row * a.splits * (D + 2);
  float top = -__builtin_inff();
  for (int s = 0; s < parts; ++s) top = fmaxf(top, p[s * (D + 2) + D]);
  const float ref = top == -__builtin_inff() ? 0.0f : top;
  float total = 0.0f;
  float2 o = make_float2(0.0f, 0.0f);
#pragma unroll 4
  for (int s = share; s < parts; s += kShares) {
    const float* e = p + s * (D + 2);
    const float2 ml = *reinterpret_cast<const float2*>(e + D), v = *reinterpret_cast<const float2*>(e + d);
    const float by = __builtin_amdgcn_exp2f(ml.x - ref);
    total += by * ml.y;
    o.x += by * v.x;
    o.y += by * v.y;
  }
  if (share) {
    sums[share - 1][d / 2] = o;
    if (d == 0) totals[share - 1] = total;
  }
  __syncthreads();
  if (share) return;
  for (int s = 0; s < kShares - 1; ++s) {
    o.x += sums[s][d / 2].x;
    o.y += sums[s][d / 2].y;
    total += totals[s];
  }
  const float by = total > 0.0f || total != total ? 1.0f / total : 0.0f;
  if (a.out_f32)
    *reinterpret_cast<float2*>(static_cast<float*>(a.out) + row * D + d) = make_float2(o.x * by, o.y * by);
  else
    *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.out) + row * D + d) =
        fp8dev::pack_bf16(o.x * by, o.y * by);
  if (a.lse && d == 0) a.lse[row] = (top + __builtin_log2f(total)) / kLog2e;
}


std::atomic<int> g_splits{0};

// Parts per request: enough workgroups for kPerCu on every CU where every
// request has as many tokens as the page table has room for, and none of fewer
// than kMinPart tokens.  A shorter request is shared among as many workgroups, as
// far as that leaves each kMinPart tokens: the kernel goes by its length.
constexpr int kPerCu = 8;

int splits_of(const fp4lib::AttnArgs& a) {
  const int64_t room = static_cast<int64_t>(a.table_width) << a.cache.page_shift;
  const int64_t most = (room + kMinPart - 1) / kMinPart;
  const int group = a.q.heads / a.cache.heads, tiles = (group + (group <= 8 ? 7 : 15)) / (group <= 8 ? 8 : 16);
  const int64_t each = static_cast<int64_t>(a.requests) * a.cache.heads * tiles;
  int64_t want = (static_cast<int64_t>(fp4lib::device_cu_count()) * kPerCu + each - 1) / each;
  if (const int forced = g_splits.load()) want = forced;
  want = want > most ? most : want;
  return static_cast<int>(want < 1 ? 1 : want > 512 ? 512 : want);
}

int64_t part_bytes(const fp4lib::AttnArgs& a, int splits) {
  return splits <= 1 ? 0
                     : static_cast<int64_t>(a.requests) * a.q.heads * splits * (a.cache.head_dim + 2) *
                           static_cast<int64_t>(sizeof(float));
}

}  // namespace

namespace fp4lib {

void set_attention_splits(int splits) { g_splits.store(splits); }

int64_t attention_workspace(const AttnArgs& a) { return part_bytes(a, splits_of(a)); }

hipError_t launch_attention(const AttnArgs& args, hipStream_t s) {
  AttnArgs a = args;
  a.splits = splits_of(a);
  if (!a.part || a.part_bytes < part_bytes(a, a.splits)) a.splits = 1;
  const int group = a.q.heads / a.cache.heads, tiles = (group + (group <= 8 ? 7 : 15)) / (group <= 8 ? 8 : 16);
  const int64_t grid = static_cast<int64_t>(a.requests) * a.cache.heads * tiles * a.splits;
  if (grid >= (int64_t(1) << 31)) return hipErrorInvalidConfiguration;
  const hipError_t e = with_format(a.cache.fmt, [&](auto f) {
    return launch_attention_fmt<decltype(f)::value>(a, static_cast<uint32_t>(grid), s);
  });
  if (e != hipSuccess || a.splits == 1) return e;
  return with_dim(a.cache.head_dim, [&](auto d) {
    constexpr int D = decltype(d)::value;
    hipLaunchKernelGGL(k_attention_join<D>, dim3(a.requests * a.q.heads), dim3(4 * D), 0, s, a);
    return hipGetLastError();
  });
}

}  // namespace fp4lib
