// Device helpers of the attention operators: the formats of a cache, sums and
// maxima over the lanes of a row, encoding and decoding of 8 elements.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fp4_device.hpp"
#include "fp8_common.hpp"
#include "gemm_common.hpp"
#include "kv_internal.hpp"

namespace kvdev {

// A constant as an argument.
template <int V>
struct Const {
  static constexpr int value = V;
};

using fp4lib::kKvFp8;
using fp4lib::kKvMx4;
using fp4lib::kKvMx8;
using fp4lib::kKvNv4;
using fp4lib::kKvUe4;

template <int FMT>
struct KvTraits {
  static constexpr bool kTwoLevel = FMT == kKvNv4 || FMT == kKvUe4;     // E4M3 / UE5M3 scales, tensor scale
  static constexpr int kBits = FMT == kKvFp8 || FMT == kKvMx8 ? 8 : 4;
  static constexpr int kBlock = FMT == kKvFp8 ? 128 : kTwoLevel ? 16 : 32;
  static constexpr int kDev = FMT == kKvUe4 ? fp4dev::kUE : fp4dev::kNV;
};

// Tensor scales of K (i = 0) or V (fp4_device.hpp: global_scales).
template <int FMT>
__device__ __forceinline__ void tensor_scales(const fp4lib::KvCacheArgs& c, int i, float& enc, float& dec) {
  enc = dec = 1.0f;
  if constexpr (KvTraits<FMT>::kTwoLevel) fp4dev::global_scales(c.amax[i], c.target, enc, dec);
}

// ------------------------------------------ over the 2, 4, .. lanes of a row --
template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
  return __builtin_amdgcn_update_dpp(0, static_cast<int>(v), CTRL, 0xF, 0xF, true);
}
constexpr int kXor1 = 0xB1, kXor2 = 0x4E;      // within a quad
constexpr int kHalfMirror = 0x141;             // lane i of 8 <-> 7 - i: the other quad
constexpr int kMirror = 0x140;                 // lane i of 16 <-> 15 - i: the other half

// In a fixed order, the same in every lane (a + b = b + a).
template <int N>
__device__ __forceinline__ float lane_sum(float v) {
  auto add = [](float a, uint32_t b) { return a + __uint_as_float(b); };
  if constexpr (N > 1) v = add(v, dpp<kXor1>(__float_as_uint(v)));
  if constexpr (N > 2) v = add(v, dpp<kXor2>(__float_as_uint(v)));
  if constexpr (N > 4) v = add(v, dpp<kHalfMirror>(__float_as_uint(v)));
  if constexpr (N > 8) v = add(v, dpp<kMirror>(__float_as_uint(v)));
  if constexpr (N > 16) v += __shfl_xor(v, 16, 64);
  return v;
}
template <int N>
__device__ __forceinline__ double lane_sum(double v) {
  auto moved = [&](auto ctrl) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    constexpr int kCtrl = decltype(ctrl)::value;
    return __builtin_bit_cast(double, static_cast<uint64_t>(dpp<kCtrl>(static_cast<uint32_t>(b >> 32))) << 32 |
                                          dpp<kCtrl>(static_cast<uint32_t>(b)));
  };
  if constexpr (N > 1) v += moved(Const<kXor1>());
  if constexpr (N > 2) v += moved(Const<kXor2>());
  if constexpr (N > 4) v += moved(Const<kHalfMirror>());
  if constexpr (N > 8) v += moved(Const<kMirror>());
  if constexpr (N > 16) v += __shfl_xor(v, 16, 64);
  return v;
}
template <int N>
__device__ __forceinline__ uint32_t lane_max(uint32_t v) {
  if constexpr (N > 1) v = fp8dev::umax(v, dpp<kXor1>(v));
  if constexpr (N > 2) v = fp8dev::umax(v, dpp<kXor2>(v));
  if constexpr (N > 4) v = fp8dev::umax(v, dpp<kHalfMirror>(v));
  if constexpr (N > 8) v = fp8dev::umax(v, dpp<kMirror>(v));
  return v;
}

typedef uint32_t words2 __attribute__((ext_vector_type(2)));
typedef float floats4 __attribute__((ext_vector_type(4)));
typedef uint32_t words4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ void load8(float (&v)[8], const uint16_t* p) {
  fp4quant::unpack8(*reinterpret_cast<const uint4*>(p), v);
}
// Past the caches: what is written here is as large as what is read and is not read
// again by the kernel (8192 tokens normed and rotated 39 -> 34.6 us, 32768 slots read back
// 60 -> 31; no loss at 64 tokens).
__device__ __forceinline__ void store8(uint16_t* p, const float (&v)[8]) {
  const words4 w = {fp8dev::pack_bf16(v[0], v[1]), fp8dev::pack_bf16(v[2], v[3]),
                    fp8dev::pack_bf16(v[4], v[5]), fp8dev::pack_bf16(v[6], v[7])};
  __builtin_nontemporal_store(w, reinterpret_cast<words4*>(p));
}

// Where slot `at` (page and place within it) of a head lies.
__device__ __forceinline__ int64_t code_at(const fp4lib::KvCacheArgs& c, int64_t page, int place, int head) {
  return page * c.page + head * c.head + place * c.token;
}
__device__ __forceinline__ int64_t scale_at(const fp4lib::KvCacheArgs& c, int64_t page, int place, int head,
                                            int block) {
  return page * c.s_page + head * c.s_head + block * c.s_block + place;
}

// A row of D elements, 8 in each of D / 8 neighbouring lanes (this one's from
// element 8 lane on), encoded as fp4_quantize encodes a row of D columns (fp8:
// blocks of 128, a row of 64 being one block).
template <int FMT, int D>
__device__ __forceinline__ void encode_row(const float (&v)[8], int lane, const fp4lib::KvCacheArgs& c, int i,
                                           int64_t page, int place, int head, float s_enc, float s_dec) {
  using F = KvTraits<FMT>;
  constexpr int kLanes = (D < F::kBlock ? D : F::kBlock) / 8;
  const uint32_t amax = lane_max<kLanes>(fp8dev::absmax8(v));
  uint8_t* codes = c.codes[i] + code_at(c, page, place, head) + lane * F::kBits;
  uint32_t code;
  if constexpr (F::kBits == 8) {
    code = fp8dev::scale_code<false>(amax);
    const float s = fp8dev::code_scale(code);
    const words2 w = {fp8dev::pack4<false>(v[0], v[1], v[2], v[3], s), fp8dev::pack4<false>(v[4], v[5], v[6], v[7], s)};
    __builtin_nontemporal_store(w, reinterpret_cast<words2*>(codes));
  } else {
    float s;
    if constexpr (F::kTwoLevel) {
      fp4dev::ScaleEvents ev{0, 0, 0};
      code = fp4dev::block_scale_two_level<F::kDev>(__uint_as_float(amax), s_enc, s_dec, s, ev);
    } else {
      code = fp4dev::block_scale_mx(__uint_as_float(amax), s);
    }
    uint32_t w = 0;
    w = fp4dev::e2m1_rne_pair<0>(w, v[0] * s, v[1] * s);
    w = fp4dev::e2m1_rne_pair<1>(w, v[2] * s, v[3] * s);
    w = fp4dev::e2m1_rne_pair<2>(w, v[4] * s, v[5] * s);
    w = fp4dev::e2m1_rne_pair<3>(w, v[6] * s, v[7] * s);
    __builtin_nontemporal_store(w, reinterpret_cast<uint32_t*>(codes));
  }
  if (lane % kLanes == 0)
    c.scales[i][scale_at(c, page, place, head, lane / kLanes)] = static_cast<uint8_t>(code);
}

// 8 elements of one block as they lie in the cache; `held` false: zeros.
template <int FMT>
struct Coded {
  using F = KvTraits<FMT>;
  uint32_t w[F::kBits / 4], scale;
  __device__ __forceinline__ void load(const uint8_t* codes, const uint8_t* at, bool held) {
    w[0] = w[F::kBits / 4 - 1] = scale = 0u;
    if (!held) return;
    if constexpr (F::kBits == 8) {
      const words2 v = *reinterpret_cast<const words2*>(codes);
      w[0] = v.x;
      w[1] = v.y;
    } else {
      w[0] = *reinterpret_cast<const uint32_t*>(codes);
    }
    scale = *at;
  }
  // as fp4_dequantize forms them
  __device__ __forceinline__ void values(float s_dec, float (&v)[8]) const {
    if constexpr (F::kBits == 8) {
      const float s = fp8dev::code_scale(scale);
      fp8dev::unpack4<false>(w[0], v, s);
      fp8dev::unpack4<false>(w[1], v + 4, s);
    } else {
      float s = 1.0f;
      if constexpr (FMT == kKvMx4) s = fp4dev::ue8m0_decode(scale);
      if constexpr (FMT == kKvNv4) s = fp4dev::scale_m3_decode<7>(scale);
      if constexpr (FMT == kKvUe4) s = fp4dev::scale_m3_decode<15>(scale);
      const fp8dev::float2v p[4] = {__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[0], 1.0f, 0),
                                    __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[0], 1.0f, 1),
                                    __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[0], 1.0f, 2),
                                    __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[0], 1.0f, 3)};
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = (p[i / 2][i % 2] * s) * s_dec;
    }
  }
};

// Calls f with the format and head dimension as constants.
template <typename F>
hipError_t with_dim(int head_dim, F&& f) {
  return head_dim == 64 ? f(Const<64>()) : head_dim == 128 ? f(Const<128>()) : f(Const<256>());
}
template <typename F>
hipError_t with_format(int fmt, F&& f) {
  switch (fmt) {
    case kKvFp8: return f(Const<kKvFp8>());
    case kKvMx8: return f(Const<kKvMx8>());
    case kKvMx4: return f(Const<kKvMx4>());
    case kKvNv4: return f(Const<kKvNv4>());
    default: return f(Const<kKvUe4>());
  }
}

}  // namespace kvdev
