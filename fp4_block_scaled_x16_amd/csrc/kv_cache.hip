// Slots of a paged key-value cache back to values.  (The cache is written by
// qk_rows.hip.)
//
// Bound by memory, mostly by what it writes: 1 (0.5) bytes in and 2 out per
// element (32768 NVFP4 slots of 8 heads of 128 in 31 us, 172 MB at 5.5 TB/s; 1000 MXFP4
// slots of 4 heads of 256 in 3.1, a launch's time).  A thread takes 8 elements of K and the same
// 8 of V: 16-byte stores, a wave 1 KiB of the output.
#include "kv_common.hpp"

using namespace kvdev;

namespace {

// per_wg slots at once.
template <int D, int FMT>
__global__ __launch_bounds__(256) void k_kv_read(fp4lib::KvReadArgs a, int per_wg) {
  using F = KvTraits<FMT>;
  constexpr int kLanes = D / 8;
  constexpr int kBlockLanes = (D < F::kBlock ? D : F::kBlock) / 8;
  const int chunks = a.cache.heads * kLanes;      // of a slot
  const int sub = threadIdx.x / static_cast<uint32_t>(chunks);
  if (sub >= per_wg) return;
  float s_dec[2], s_enc;
  tensor_scales<FMT>(a.cache, 0, s_enc, s_dec[0]);
  tensor_scales<FMT>(a.cache, 1, s_enc, s_dec[1]);
  const int mask = (1 << a.cache.page_shift) - 1;
  for (int64_t n = static_cast<int64_t>(blockIdx.x) * per_wg + sub; n < a.n;
       n += static_cast<int64_t>(gridDim.x) * per_wg) {
    const int64_t slot = a.slots[n], page = slot >> a.cache.page_shift;
    const int place = static_cast<int>(slot) & mask;
    const bool held = slot >= 0 && page < a.cache.pages;       // else zeros
    for (int c = threadIdx.x - sub * chunks; c < chunks; c += 256) {
      const int head = c / kLanes, l = c % kLanes;
      Coded<FMT> q[2];
#pragma unroll
      for (int i = 0; i < 2; ++i)
        q[i].load(a.cache.codes[i] + code_at(a.cache, page, place, head) + l * F::kBits,
                  a.cache.scales[i] + scale_at(a.cache, page, place, head, l / kBlockLanes), held);
      const int64_t at = (n * a.cache.heads + head) * D + 8 * l;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if (!a.out[i]) continue;
        float v[8];
        q[i].values(s_dec[i], v);
        if (a.out_f32) {
          float* p = static_cast<float*>(a.out[i]) + at;
          __builtin_nontemporal_store(floats4{v[0], v[1], v[2], v[3]}, reinterpret_cast<floats4*>(p));
          __builtin_nontemporal_store(floats4{v[4], v[5], v[6], v[7]}, reinterpret_cast<floats4*>(p + 4));
        } else {
          store8(static_cast<uint16_t*>(a.out[i]) + at, v);
        }
      }
    }
  }
}

// Workgroups enough that each has a slot or two; several slots' loads under way in a
// thread, and fewer workgroups, measured no better (32768 NVFP4 slots of 8 heads of 128: 1
// slot at once in 64 workgroups per CU 30.8 us, 2 in 8 34.7).
constexpr int kReadPerCu = 64;

}  // namespace

namespace fp4lib {

hipError_t launch_kv_read(const KvReadArgs& a, hipStream_t s) {
  const int chunks = a.cache.heads * a.cache.head_dim / 8;
  const int per_wg = chunks >= 256 ? 1 : 256 / chunks;
  const int64_t want = (a.n + per_wg - 1) / per_wg, cap = static_cast<int64_t>(device_cu_count()) * kReadPerCu;
  const dim3 grid(static_cast<uint32_t>(want < cap ? want : cap));
  return kvdev::with_dim(a.cache.head_dim, [&](auto d) {
    return kvdev::with_format(a.cache.fmt, [&](auto f) {
      hipLaunchKernelGGL((k_kv_read<decltype(d)::value, decltype(f)::value>), grid, dim3(256), 0, s, a, per_wg);
      return hipGetLastError();
    });
  });
}

}  // namespace fp4lib
