// Launch of the attention of one new token per request (attention.hip), and the
// kernel that joins the parts that a request's tokens are shared among (attention_plan.hpp):
//   m = max_s m_s,  out = sum_s 2^(m_s - m) o_s / sum_s 2^(m_s - m) l_s
// of each part's maximum m_s, sum l_s and sum of p v o_s.  Few bytes (64 requests of up to
// 8192 tokens, 32 heads on 8 of 128: 1.1 MB read), so it is bound by its launch and two
// rounds of loads: 3 to 5 us.
#include <algorithm>
#include <atomic>

#include "attention_common.hpp"

using namespace kvdev;
using namespace fp4attn;

namespace {

constexpr float kLog2e = 1.44269504088896340736f;

// out and lse of a row from its parts' sums o (the thread's four elements), the
// largest of their maxima and their sum.
template <int D>
__device__ __forceinline__ void finish(const fp4lib::AttnArgs& a, int64_t row, int d, float4 o, float top, float total) {
  const float by = total > 0.0f || total != total ? 1.0f / total : 0.0f;
  if (a.out_f32)
    *reinterpret_cast<float4*>(static_cast<float*>(a.out) + row * D + 4 * d) =
        make_float4(o.x * by, o.y * by, o.z * by, o.w * by);
  else
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + row * D + 4 * d) =
        make_uint2(fp8dev::pack_bf16(o.x * by, o.y * by), fp8dev::pack_bf16(o.z * by, o.w * by));
  if (a.lse && d == 0) a.lse[row] = (top + __builtin_log2f(total)) / kLog2e;
}

// A row's parts: every a.group-th row of sums from `first` on.
struct Parts {
  int64_t first;
  int count;
  __device__ __forceinline__ Parts(const fp4lib::AttnArgs& a, uint32_t row) {
    const uint32_t heads = a.q.heads, request = row / heads, head = row - request * heads;
    const uint32_t kv = head / static_cast<uint32_t>(a.group);
    const int2 p = request_parts(a)[request];
    // (within the workspace in any case: lengths that change while the kernels run may cost
    // results, and no more)
    const int64_t base = std::min<uint32_t>(p.x, static_cast<uint32_t>(a.items - 1));
    first = (kv * a.items + base) * a.group + (head - kv * a.group);
    count = static_cast<int>(std::min<int64_t>(std::min(p.y, a.splits), a.items - base));
  }
};

// Few parts: D / 4 lanes per query head, four elements each.
constexpr int kFewParts = 16;
template <int D>
__global__ __launch_bounds__(256) void k_attention_join_few(fp4lib::AttnArgs a) {
  constexpr int kQuads = D / 4;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (256 / kQuads) + threadIdx.x / kQuads;
  if (row >= static_cast<int64_t>(a.requests) * a.q.heads) return;
  const int d = threadIdx.x % kQuads;
  const Parts in(a, static_cast<uint32_t>(row));
  const int parts = in.count;
  if (parts <= 1) return;
  const int step = a.group;
  const float4* p = reinterpret_cast<const float4*>(a.part + in.first * D) + d;
  const float2* ml = part_sums(a) + in.first;
  float top = -__builtin_inff(), total = 0.0f;
  float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
  for (int s = 0; s < parts; ++s) top = fmaxf(top, ml[s * step].x);
  const float ref = top == -__builtin_inff() ? 0.0f : top;
#pragma unroll 4
  for (int s = 0; s < parts; ++s) {
    const float4 v = p[s * step * kQuads];
    const float2 m = ml[s * step];
    const float by = __builtin_amdgcn_exp2f(m.x - ref);
    total += by * m.y;
    o.x += by * v.x;
    o.y += by * v.y;
    o.z += by * v.z;
    o.w += by * v.w;
  }
  finish<D>(a, row, d, o, top, total);
}

// The parts of a request, in order: a workgroup per query head, whose threads take
// four elements each of every kShares-th part.
template <int D>
__global__ __launch_bounds__(256) void k_attention_join(fp4lib::AttnArgs a) {
  constexpr int kQuads = D / 4, kShares = 256 / kQuads;
  __shared__ float4 sums[kShares][kQuads];
  __shared__ float weights[kMaxParts];
  __shared__ float2 most[4];
  const int64_t row = blockIdx.x;
  const Parts in(a, static_cast<uint32_t>(row));
  const int parts = in.count;
  if (parts <= 1) return;
  const float* p = a.part + in.first * D;
  const float2* ml = part_sums(a) + in.first;
  // what each part's sums count for: 2^(its maximum - the largest)
  float2 mine[kMaxParts / 256];
  float top = -__builtin_inff();
#pragma unroll
  for (int i = 0; i < kMaxParts / 256; ++i) {
    const int s = threadIdx.x + 256 * i;
    mine[i] = s < parts ? ml[s * a.group] : make_float2(-__builtin_inff(), 0.0f);
    top = fmaxf(top, mine[i].x);
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor(top, o, 64));
  if ((threadIdx.x & 63) == 0) most[threadIdx.x >> 6].x = top;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 4; ++i) top = fmaxf(top, most[i].x);
  const float ref = top == -__builtin_inff() ? 0.0f : top;
  float total = 0.0f;
#pragma unroll
  for (int i = 0; i < kMaxParts / 256; ++i) {
    const int s = threadIdx.x + 256 * i;
    const float by = __builtin_amdgcn_exp2f(mine[i].x - ref);
    if (s < parts) {
      weights[s] = by;
      total += by * mine[i].y;
    }
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) total += __shfl_xor(total, o, 64);
  if ((threadIdx.x & 63) == 0) most[threadIdx.x >> 6].y = total;
  __syncthreads();
  total = ((most[0].y + most[1].y) + most[2].y) + most[3].y;

  const int share = threadIdx.x / kQuads, d = threadIdx.x % kQuads;
  float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
  for (int s = share; s < parts; s += kShares) {
    const float4 v = *reinterpret_cast<const float4*>(p + static_cast<int64_t>(s) * a.group * D + 4 * d);
    const float by = weights[s];
    o.x += by * v.x;
    o.y += by * v.y;
    o.z += by * v.z;
    o.w += by * v.w;
  }
  sums[share][d] = o;
  __syncthreads();
  if (threadIdx.x >= kQuads) return;
#pragma unroll
  for (int s = 1; s < kShares; ++s) {
    o.x += sums[s][d].x;
    o.y += sums[s][d].y;
    o.z += sums[s][d].z;
    o.w += sums[s][d].w;
  }
  finish<D>(a, row, d, o, top, total);
}

std::atomic<int> g_splits{0};

void plan(fp4lib::AttnArgs& a) { fp4attn::plan(a, fp4lib::device_cu_count(), g_splits.load()); }

}  // namespace

namespace fp4lib {

void set_attention_splits(int splits) { g_splits.store(splits); }

int64_t attention_workspace(const AttnArgs& args) {
  AttnArgs a = args;
  plan(a);
  return part_bytes(a);
}

namespace {

// One launch's requests.
hipError_t launch_some(const AttnArgs& a, hipStream_t s) {
  int64_t grid = a.items * a.cache.heads;
  if (a.tiles > 1) grid = (grid + 7) / 8 * 8 * a.tiles;
  const hipError_t e = with_format(a.cache.fmt, [&](auto f) {
    return launch_attention_fmt<decltype(f)::value>(a, static_cast<uint32_t>(grid), s);
  });
  if (e != hipSuccess || a.splits == 1) return e;
  return with_dim(a.cache.head_dim, [&](auto d) {
    constexpr int D = decltype(d)::value;
    const int64_t rows = static_cast<int64_t>(a.requests) * a.q.heads;
    if (a.splits <= kFewParts || (a.planned && a.requests * a.q.heads >= 2048))
      hipLaunchKernelGGL(k_attention_join_few<D>, dim3(static_cast<uint32_t>((rows * (D / 4) + 255) / 256)),
                         dim3(256), 0, s, a);
    else
      hipLaunchKernelGGL(k_attention_join<D>, dim3(static_cast<uint32_t>(rows)), dim3(256), 0, s, a);
    return hipGetLastError();
  });
}

}  // namespace

hipError_t launch_attention(const AttnArgs& args, hipStream_t s) {
  AttnArgs a = args;
  plan(a);
  if (!a.part || a.part_bytes < part_bytes(a)) set_parts(a, 1);
  auto inverse = [](int n) { return static_cast<uint32_t>(((int64_t(1) << 32) + n - 1) / n); };
  a.by_splits = inverse(a.splits);
  a.by_heads = inverse(a.cache.heads);
  return by_launches(a, [&](const AttnArgs& some) { return launch_some(some, s); });
}

}  // namespace fp4lib
