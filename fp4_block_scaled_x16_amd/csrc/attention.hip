// Attention of one new token per request over its pages of a quantized
// key-value cache:  out = softmax(scale q K^T) V  over the request's tokens.
//
// Bound by reading the codes once, where there are many: 64 requests of up to 8192
// MXFP8 tokens (8 heads of 128 for 32 query heads) take 101.5 us, 5.5 TB/s of codes and
// scales, 64 of 8192 174 us, 6.4 TB/s; 1000 of up to 4000 of heads of 64 329 us, 6.4 TB/s.
// With 4-bit codes and block scales that are no powers of two by the vector instructions
// as well (4 of 120000 NVFP4 tokens: 71 % of cycles; 103 to 108 us, 5.1 to 5.4 TB/s).  Few
// or short requests by their steps, one after the other: about 1 us for 128 tokens of
// heads of 128 (a tile's 240 vector and 90 scalar instructions, and the wait for its
// codes), and about 5 for the launch, the loads that wait for one another at the start,
// and the meeting of the waves (1 request of 1000 FP8 tokens: 6 us and 3 for the join).
//
// A workgroup of four waves has one request, one key head, up to 16 of the query heads
// that share it, and a part of the request's tokens; its waves take turns at tiles of
// 32 tokens, each with a running maximum and sum of its own, and meet in LDS at the
// end.  Where a request has several parts, their sums go to the caller's workspace and
// k_attention_join brings them together in order (no atomics: the same bits every
// time).  Which part a workgroup takes goes by the lengths of all requests, the longest
// first (planned_item).  Short requests have a workgroup of eight waves each where they are
// few, and one of a single wave where they are many (attention_plan.hpp: plan).
//
// Codes go from global memory into registers and, widened, straight into MFMA
// operands: no byte of the cache is used twice, so nothing is staged in LDS.
//   scores^T [token, head] = K q^T.  Lane (c, g) (c = lane % 16, g = lane / 16) has a
//     token of each half tile, elements g D/4 .. of its row; q's operand is laid out
//     to match.  The tokens stand in the operand's rows such that it gets back
//     tokens g, 4 + g, 8 + g and 12 + g of head c.
//   out^T [element, head] += V^T p^T.  The four scores of each half are the lane's
//     own part of p's operand: p never leaves its lane.  V^T's operand holds elements
//     of the same 8 tokens (four of each half), so a lane loads elements c D/16 ..
//     of those 8 rows (four neighbouring rows to an instruction of the wave) and pairs
//     tokens with byte permutes.
// FP8, MXFP8 and MXFP4 are widened to bf16, their power-of-two scales applied by
// the same convert; NVFP4 and UE5M3 to fp16, in which code times block scale is
// exact (UE5M3 times 2^-5), q's row being scaled into fp16's range by a power of
// two.  Either way the operands are exact.  So is p in bf16, in three parts of 8 bits; in
// fp16 a rounded part and what that leaves hold 2^-22 of it.  For up to 8 heads the second
// part takes the other 8 of the matrix's 16 columns, for more a second MFMA; the third takes
// one more.  (Two bf16 parts, 2^-17 of p, leave 2.2 of 1000 outputs in bf16 beside the
// nearest one, 64 requests of up to 8192 MXFP8 tokens, where elementary fp32 operations leave
// 0.6; three leave 0.3.  They cost nothing where memory bounds, 101.9 and 101.5 us there, and
// up to 7 % where vector instructions do: 256 of up to 1024 MXFP4 tokens 14.8 and 15.4 us, 8 of
// 30000 with 64 heads on one 29.2 and 31.2.  Figures below and beside the plan that compare two
// ways of one step are from kernels with two parts.)
#include "attention_common.hpp"

using namespace kvdev;
using namespace fp4attn;

namespace {

typedef float floatx4 __attribute__((ext_vector_type(4)));
typedef uint32_t uintx4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 halfx8 __attribute__((ext_vector_type(8)));
typedef _Float16 halfx2 __attribute__((ext_vector_type(2)));

constexpr float kLog2e = 1.44269504088896340736f;
// A running maximum is raised only when a score exceeds it by this many powers
// of two: what it guards against is overflow, and until then nothing has to be
// rescaled.
constexpr float kSlack = 8.0f;

template <bool F16>
__device__ __forceinline__ floatx4 mfma(uintx4 a, uintx4 b, floatx4 c) {
  if constexpr (F16)
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(halfx8, a),
                                                  __builtin_bit_cast(halfx8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// A float's upper half, and those of two (with kZeros: zeros) as bf16.
__device__ __forceinline__ float upper(float x) { return __uint_as_float(__float_as_uint(x) & 0xFFFF0000u); }
constexpr uint32_t kUpperHalves = 0x07060302u, kZeros = 0x0C0C0C0Cu;
__device__ __forceinline__ uint32_t upper_pair(float x, float y, uint32_t which) {
  return __builtin_amdgcn_perm(__float_as_uint(y), __float_as_uint(x), which);
}

// Two floats as fp16, to nearest even.
__device__ __forceinline__ uint32_t pack2(float x, float y) {
  return __builtin_bit_cast(uint32_t, halfx2{static_cast<_Float16>(x), static_cast<_Float16>(y)});
}
// The halves of a word, of bf16 or fp16.
template <bool F16>
__device__ __forceinline__ float unpack_lo(uint32_t w) {
  if constexpr (F16) return static_cast<float>(__builtin_bit_cast(halfx2, w)[0]);
  return __uint_as_float(w << 16);
}
template <bool F16>
__device__ __forceinline__ float unpack_hi(uint32_t w) {
  if constexpr (F16) return static_cast<float>(__builtin_bit_cast(halfx2, w)[1]);
  return __uint_as_float(w & 0xFFFF0000u);
}

// Codes of pair P of a word (8-bit: 0, 1; 4-bit: 0 .. 3) widened: `s` is the
// block scale, as a float (bf16) or as an fp16 pair of which HALF is it.
template <int FMT, int P, int HALF>
__device__ __forceinline__ uint32_t widen2(uint32_t w, uint32_t s) {
  using F = KvTraits<FMT>;
  if constexpr (F::kTwoLevel) {
    const halfx2 sp = __builtin_bit_cast(halfx2, s);
    const halfx2 v = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, P);
    return __builtin_bit_cast(uint32_t, v * (HALF ? halfx2{sp[1], sp[1]} : halfx2{sp[0], sp[0]}));
  } else if constexpr (F::kBits == 8) {
    return __builtin_bit_cast(uint32_t,
                              __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, __uint_as_float(s), P == 1));
  } else {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, __uint_as_float(s), P));
  }
}

// Pair i of a lane's words (a constant once the loops around it are unrolled).
template <int FMT, int N>
__device__ __forceinline__ uint32_t widen_pair(const uint32_t (&w)[N], int i, uint32_t s, int half) {
  if constexpr (KvTraits<FMT>::kBits == 8)
    return i % 2 ? widen2<FMT, 1, 0>(w[i / 2], s) : widen2<FMT, 0, 0>(w[i / 2], s);
  switch (i % 4 + 4 * half) {
    case 0: return widen2<FMT, 0, 0>(w[i / 4], s);
    case 1: return widen2<FMT, 1, 0>(w[i / 4], s);
    case 2: return widen2<FMT, 2, 0>(w[i / 4], s);
    case 3: return widen2<FMT, 3, 0>(w[i / 4], s);
    case 4: return widen2<FMT, 0, 1>(w[i / 4], s);
    case 5: return widen2<FMT, 1, 1>(w[i / 4], s);
    case 6: return widen2<FMT, 2, 1>(w[i / 4], s);
    default: return widen2<FMT, 3, 1>(w[i / 4], s);
  }
}

// Scale B of a word of four scale codes as widen2 takes it: a float's bits, or
// the fp16 pair that holds it in half B % 2.
template <int FMT, int B>
__device__ __forceinline__ uint32_t scale_for(uint32_t word) {
  if constexpr (KvTraits<FMT>::kTwoLevel)
    return fp4gemm::scale_pair_f16<KvTraits<FMT>::kDev, B & 2>(word);
  else
    return ((word >> (8 * B)) & 0xFFu) << 23;
}

// An address in scalar registers, of global memory: without this the compiler adds the
// lane's offset to the loop's invariant part and keeps 64-bit sums for every load in
// vector registers.
typedef const __attribute__((address_space(1))) uint8_t* GlobalBytes;
__device__ __forceinline__ GlobalBytes uniform(const uint8_t* p) {
  GlobalBytes q = (GlobalBytes)p;
  asm("" : "+s"(q));
  return q;
}

// N bytes (2, 4, 8 or a multiple of 16) into words.  STREAM: past the caches, where
// one instruction of the wave takes the whole of every line that it touches.
template <bool STREAM, typename T>
__device__ __forceinline__ T load_as(GlobalBytes p, uint32_t at) {
  typedef const __attribute__((address_space(1))) T* Ptr;
  asm("" : "+v"(at));          // 32 bits here, too: widened where it is made, it is no operand of the load
  if constexpr (STREAM) return __builtin_nontemporal_load((Ptr)(p + at));
  return *(Ptr)(p + at);
}
template <int N, bool STREAM>
struct Raw {
  uint32_t w[N < 4 ? 1 : N / 4];
  __device__ __forceinline__ void load(GlobalBytes p, uint32_t at) {
    if constexpr (N == 2) {
      w[0] = load_as<STREAM, uint16_t>(p, at);
    } else if constexpr (N == 4) {
      w[0] = load_as<STREAM, uint32_t>(p, at);
    } else if constexpr (N == 8) {
      const words2 v = load_as<STREAM, words2>(p, at);
      w[0] = v.x, w[1] = v.y;
    } else {
#pragma unroll
      for (int i = 0; i < N / 16; ++i) {
        const words4 v = load_as<STREAM, words4>(p + 16 * i, at);
        w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
      }
    }
  }
};

template <int FMT, int D>
struct Shape {
  using F = KvTraits<FMT>;
  static constexpr int kSteps = D / 32;                       // MFMAs over a row of K
  static constexpr int kKBytes = D / 4 * F::kBits / 8;        // of a lane's part of a row of K
  static constexpr int kKBlocks = D / 4 <= F::kBlock ? 1 : D / 4 / F::kBlock;
  static constexpr int kElems = D / 16;                       // of a lane's part of a row of V
  static constexpr int kVBytes = kElems * F::kBits / 8;
  // A quad whose elements lie in one block shares the loading of its tokens' scales.
  // (Pairs could too, but NVFP4's step is short of instructions, not of loads: 4 requests
  // of 120000 in 107 instead of 104 us.)
  static constexpr int kShare = F::kBlock / kElems >= 4 ? 4 : 1;
};

// Where a half's codes and scales begin, and how many of its tokens there are: the
// same for the whole wave, so a load is that address plus the lane's own offset.
struct HalfPos {
  uint64_t code, scale;
  int n;                        // 16 or more: all; 0 or less: none
};

template <int FMT, int D, bool STREAM>
struct KHalf {
  using S = Shape<FMT, D>;
  Raw<S::kKBytes, STREAM && S::kKBytes <= 16> w;
  uint32_t s[S::kKBlocks];
};
template <int FMT, int D, bool STREAM>
struct VHalf {
  using S = Shape<FMT, D>;
  Raw<S::kVBytes, STREAM> w[4];
  Raw<16 / S::kShare, false> s;      // this lane's share of the scale codes of the half's 16 tokens
};

// The scale codes of the lane's tokens g, 4 + g, 8 + g and 12 + g, in a word: byte g
// of each of four words, of which the lane holds one (SHARE lanes together the four) or all.
struct ScalePick {
  uint32_t own, pair, quad;
  __device__ __forceinline__ explicit ScalePick(int c, int g) {
    own = 0x0C0C0400u + 0x0101u * g;                       // byte g of two words
    pair = c & 1 ? 0x0C0C0004u + 0x0101u * g : own;        // the even lane's first
    quad = c & 2 ? 0x01000504u : 0x05040100u;              // two halves, the lower lanes' first
  }
  template <int SHARE>
  __device__ __forceinline__ uint32_t take(const uint32_t* w) const {
    if constexpr (SHARE == 4) {
      const uint32_t t = __builtin_amdgcn_perm(dpp<kXor1>(w[0]), w[0], pair);
      return __builtin_amdgcn_perm(dpp<kXor2>(t), t, quad);
    } else {
      return __builtin_amdgcn_perm(__builtin_amdgcn_perm(w[3], w[2], own), __builtin_amdgcn_perm(w[1], w[0], own),
                                   0x05040100u);
    }
  }
};

// A workgroup's part of a request: tokens part * per .., as one of `parts`, the first of
// which is part number `base` of its key head's.
struct Item {
  int request, len, part, parts, per, base;
};

__device__ __forceinline__ uint32_t wave_sum(uint32_t v) {
  v += dpp<kXor1>(v);
  v += dpp<kXor2>(v);
  v += dpp<kHalfMirror>(v);
  v += dpp<kMirror>(v);
  return __builtin_amdgcn_readlane(v, 0) + __builtin_amdgcn_readlane(v, 16) + __builtin_amdgcn_readlane(v, 32) +
         __builtin_amdgcn_readlane(v, 48);
}

// Sum over the lanes up to this one.
__device__ __forceinline__ int wave_scan(int v) {
  auto moved = [&](auto ctrl, auto rows) {
    return __builtin_amdgcn_update_dpp(0, v, decltype(ctrl)::value, decltype(rows)::value, 0xF, false);
  };
  v += moved(Const<0x111>(), Const<0xF>());      // row_shr:1, 2, 4, 8
  v += moved(Const<0x112>(), Const<0xF>());
  v += moved(Const<0x114>(), Const<0xF>());
  v += moved(Const<0x118>(), Const<0xF>());
  v += moved(Const<0x142>(), Const<0xA>());      // row_bcast:15 into the odd rows, row_bcast:31 into the upper two
  v += moved(Const<0x143>(), Const<0xC>());
  return v;
}

// Parts by the lengths; the one that has place nth when the longest come first (in 16
// classes; in each by request): where more workgroups wait than the chip holds, those
// that come last should have least to do.  parts = 0: there is no nth.
// kWhole: every request is one part.
template <int D, bool kWhole>
__device__ __forceinline__ Item planned_item(const fp4lib::AttnArgs& a, int nth, int lane) {
  constexpr int kChunks = kPlanned / 64, kClasses = 16;
  if (!kWhole && a.requests == 1) {
    const int len = tokens_of(a, 0), size = (len + kStep - 1) / kStep;
    const int parts = parts_of(size, first_shares<D>(size, a).step);
    return {0, len, nth, parts, steps_of(size, parts) * kStep, 0};
  }
  int len[kChunks], parts[kChunks], size[kChunks];       // size: steps, then steps of a part
  uint32_t all = 0;
#pragma unroll
  for (int k = 0; k < kChunks; ++k) len[k] = tokens_of(a, min(64 * k + lane, a.requests - 1));
#pragma unroll
  for (int k = 0; k < kChunks; ++k) {
    size[k] = 64 * k + lane < a.requests ? (len[k] + kStep - 1) / kStep : 0;
    all += size[k];
  }
  Shares s{1, 1};
  if constexpr (!kWhole) s = first_shares<D>(wave_sum(all), a);
  auto split = [&] {
    uint32_t count = 0;
#pragma unroll
    for (int k = 0; k < kChunks; ++k) {
      if (64 * k >= a.requests) break;
      parts[k] = 64 * k + lane < a.requests ? parts_of(size[k], s.step) : 0;
      count += parts[k];
    }
    return static_cast<int>(wave_sum(count));
  };
  int count = a.requests;
  if constexpr (kWhole) {
#pragma unroll
    for (int k = 0; k < kChunks; ++k) parts[k] = 64 * k + lane < a.requests;
  } else {
    count = split();
  }
  // what rounding up each request's number has added comes off again: a round of workgroups that
  // is not full costs as much as one that is
  if (!kWhole && count > s.want && a.requests < s.want) {
    s.step = longer_step(s.step, count, s.want);
    count = split();
  }
  const bool order = kWhole || count > a.target[1];      // (else each has a CU to itself)
  uint32_t longest = 0;
#pragma unroll
  for (int k = 0; k < kChunks; ++k) {
    if (64 * k >= a.requests) break;
    const int n = max(parts[k], 1);
    if constexpr (!kWhole) size[k] = steps_of(size[k], n);
    longest = fp8dev::umax(longest, size[k]);
  }
  int c = 0;
  float by = 0.0f;               // all in class 0
  if (order) {
    longest = lane_max<16>(longest);
    longest = fp8dev::umax(fp8dev::umax(__builtin_amdgcn_readlane(longest, 0), __builtin_amdgcn_readlane(longest, 16)),
                           fp8dev::umax(__builtin_amdgcn_readlane(longest, 32), __builtin_amdgcn_readlane(longest, 48)));
    by = kClasses * __builtin_amdgcn_rcpf(static_cast<float>(longest) + 1.0f);
    auto class_of = [&](int k) { return min(static_cast<int>(static_cast<float>(size[k]) * by), kClasses - 1); };
    // the class: the highest with more than nth parts in it and above; `above` it
    int above = 0;
#pragma unroll
    for (int bit = kClasses / 2; bit; bit /= 2) {
      uint32_t over = 0;
#pragma unroll
      for (int k = 0; k < kChunks; ++k) {
        if (64 * k >= a.requests) break;
        if constexpr (kWhole) over += __popcll(__ballot(parts[k] && class_of(k) >= c + bit));
        else over += class_of(k) >= c + bit ? parts[k] : 0;
      }
      if constexpr (!kWhole) over = wave_sum(over);
      if (static_cast<int>(over) > nth) c += bit;
      else above = over;
    }
    nth = __builtin_amdgcn_readfirstlane(nth - above);
  }
  Item found{0, 0, 0, 0, 0, 0};
  int base = 0;
#pragma unroll
  for (int k = 0; k < kChunks; ++k) {
    if (64 * k >= a.requests) break;
    const bool mine = min(static_cast<int>(static_cast<float>(size[k]) * by), kClasses - 1) == c;
    if constexpr (kWhole) {
      const uint64_t in = __ballot(mine && parts[k]);
      const int many = __popcll(in);
      if (nth >= 0 && nth < many) {
        const int before = __builtin_amdgcn_mbcnt_hi(static_cast<uint32_t>(in >> 32),
                                                     __builtin_amdgcn_mbcnt_lo(static_cast<uint32_t>(in), 0));
        const int at = __builtin_amdgcn_readfirstlane(
            __ffsll(static_cast<unsigned long long>(__ballot(mine && parts[k] && before == nth))) - 1);
        found = {64 * k + at, __builtin_amdgcn_readlane(len[k], at), 0, 1,
                 __builtin_amdgcn_readlane(size[k], at) * kStep, 64 * k + at};
      }
      nth -= many;
      continue;
    }
    const int up_to = wave_scan(parts[k]), in = wave_scan(mine ? parts[k] : 0);
    const uint64_t here = __ballot(mine && nth < in && nth >= in - parts[k]);
    if (here) {
      const int at = __builtin_amdgcn_readfirstlane(__ffsll(static_cast<unsigned long long>(here)) - 1);
      const int n = __builtin_amdgcn_readlane(parts[k], at);
      found = {64 * k + at, __builtin_amdgcn_readlane(len[k], at), nth - (__builtin_amdgcn_readlane(in, at) - n), n,
               __builtin_amdgcn_readlane(size[k], at) * kStep, base + __builtin_amdgcn_readlane(up_to, at) - n};
    }
    nth -= __builtin_amdgcn_readlane(in, 63);
    base += __builtin_amdgcn_readlane(up_to, 63);
  }
  return found;
}

// Read through the scalar cache (the kernel does not write the page table), whose
// waits are apart from the vector loads'.
typedef const __attribute__((address_space(4))) int32_t* ConstInts;

template <int FMT, int D, int NP, bool STREAM, int W>
__global__ __launch_bounds__(64 * W, W == kWideWaves ? 2 : waves_per_simd(D)) void k_attention(fp4lib::AttnArgs a) {
  using F = KvTraits<FMT>;
  using S = Shape<FMT, D>;
  constexpr bool kF16 = F::kTwoLevel;
  constexpr int kHeads = NP == 1 ? 8 : 16;                   // query heads of a workgroup
  // fp16 holds p down to 2^-24: its largest, 2^kSlack, is moved up by 2^7
  constexpr float kShift = kF16 ? 7.0f : 0.0f;
  __shared__ float meet[W > 1 ? W - 1 : 1][S::kElems * 4 + 2][64];

  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c = lane & 15, g = lane >> 4;
  const int group = a.group, tiles = a.tiles;
  // Workgroups go round the 8 XCDs: those of one part (more than 16 query heads to a key
  // head) are 8 apart, so that they find its codes in one L2 (64 requests of 4096 MXFP8
  // tokens, 64 heads on one, 47.8 -> 35.9 us; 64 of 8000 in FP8, 32 heads of 256 on one, 86 -> 69).
  uint32_t id = blockIdx.x;
  int tile = 0;
  if (tiles > 1) {
    const uint32_t eight = id / 8, part = eight / tiles;
    tile = eight - part * tiles;
    id = 8 * part + id % 8;
  }
  // (the quotients are exact: id < 2^32 / 1024)
  const bool planned = W == kWaves && a.planned;
  const uint32_t part = !planned && a.splits > 1 ? __umulhi(id, a.by_splits) : id;
  const int split = id - part * a.splits;
  id = a.cache.heads > 1 ? __umulhi(part, a.by_heads) : part;
  const int kv = part - id * a.cache.heads;
  Item item;
  if (planned) {
    item = a.splits > 1 ? planned_item<D, false>(a, id, lane) : planned_item<D, true>(a, id, lane);
  } else {
    if (id >= static_cast<uint32_t>(a.requests)) return;
    item.request = id;
    item.len = tokens_of(a, id);
    item.part = split;
    item.per = part_tokens(item.len, a);
    item.parts = max(1, (item.len + item.per - 1) / item.per);
    item.base = item.request * a.splits;
  }
  if (item.part >= item.parts || item.base + item.part >= a.items) return;
  const int request = __builtin_amdgcn_readfirstlane(item.request);
  const int begin = __builtin_amdgcn_readfirstlane(item.part * item.per);
  const int end = __builtin_amdgcn_readfirstlane(min(item.len, begin + item.per));
  const int first = kv * group + tile * kHeads, heads = min(kHeads, group - tile * kHeads);
  // (every thread: the compiler fails where one of them is chosen)
  if (a.splits > 1 && kv == 0 && tile == 0 && item.part == 0)
    request_parts(a)[request] = make_int2(item.base, item.parts);
  const int col = NP == 1 ? c & 7 : c;
  const bool mine = col < heads;
  const int64_t row = static_cast<int64_t>(request) * a.q.heads + first + (mine ? col : 0);

  // q, elements g D/4 .. of the lane's head: the operand of each step.  The sign of
  // the scale goes into it, so that the largest score is that of the largest product.
  uintx4 q[S::kSteps];
  float factor = fabsf(a.scale) * kLog2e;
  const uint32_t flip = a.scale < 0.0f ? 0x80008000u : 0u, keep = a.scale == 0.0f ? 0u : ~0u;
  {
    const uint16_t* p = a.q.x + request * a.q.token + static_cast<int64_t>(first + (mine ? col : 0)) * a.q.head +
                        g * (D / 4);
#pragma unroll
    for (int k = 0; k < S::kSteps; ++k) {
      const uint4 w = *reinterpret_cast<const uint4*>(p + 8 * k);
      q[k] = (uintx4{w.x, w.y, w.z, w.w} ^ flip) & keep;
    }
    if constexpr (kF16) {
      float s_enc, s_dec;
      tensor_scales<FMT>(a.cache, 0, s_enc, s_dec);
      uint32_t big = 0;
#pragma unroll
      for (int k = 0; k < S::kSteps; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          big = fp8dev::umax(big, fp8dev::umax((q[k][i] << 16) & 0x7FFFFFFFu, q[k][i] & 0x7FFF0000u));
      big = fp8dev::umax(big, __shfl_xor(big, 16, 64));
      big = fp8dev::umax(big, __shfl_xor(big, 32, 64));
      const int e = 14 - (static_cast<int>(big >> 23) - 127);      // largest element to 2^14 .. 2^15
#pragma unroll
      for (int k = 0; k < S::kSteps; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          q[k][i] = pack2(__builtin_ldexpf(unpack_lo<false>(q[k][i]), e),
                                __builtin_ldexpf(unpack_hi<false>(q[k][i]), e));
      factor = __builtin_ldexpf(factor * s_dec, (FMT == kKvUe4 ? 5 : 0) - e);
    }
  }

  // masked scores are -infinity, which a factor of 0 would make a NaN (a scale of 0,
  // or one that a tiny q brings to 0: no score differs from 0 then)
  if (factor == 0.0f) factor = 0x1p-126f;

  floatx4 acc[S::kElems];
#pragma unroll
  for (int i = 0; i < S::kElems; ++i) acc[i] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
  float top = -__builtin_inff(), total = 0.0f;

  const ConstInts table = (ConstInts)(a.table + request * a.table_stride);
  const int mask = ((1 << a.cache.page_shift) - 1) & ~15;
  // (behind the last token: the 16 tokens with the last one, whose lines are near)
  auto page_at = [&](int t) { return table[min(t, end - 1) >> a.cache.page_shift]; };
  const uint32_t count = static_cast<uint32_t>(a.cache.pages), stride = static_cast<uint32_t>(a.cache.page);
  const uint32_t s_stride = static_cast<uint32_t>(a.cache.s_page), token = static_cast<uint32_t>(a.cache.token);
  const uint32_t block = static_cast<uint32_t>(a.cache.s_block);
  auto half_at = [&](int t, int number) {
    HalfPos h;
    const bool there = static_cast<uint32_t>(number) < count;       // else its tokens are masked
    const uint32_t place = min(t, end - 1) & mask, page = there ? number : 0;
    h.n = there ? end - t : 0;
    h.code = static_cast<uint64_t>(page) * stride + place * token;
    h.scale = static_cast<uint64_t>(page) * s_stride + place;
    return h;
  };
  // the lane's offsets (below 2^31: kv_api.cpp)
  const uint8_t* const codes[2] = {a.cache.codes[0] + kv * a.cache.head, a.cache.codes[1] + kv * a.cache.head};
  const uint8_t* const scales[2] = {a.cache.scales[0] + kv * a.cache.s_head,
                                    a.cache.scales[1] + kv * a.cache.s_head};
  const uint32_t k_row = 4 * (c & 3) + (c >> 2);
  const uint32_t k_code = k_row * token + g * S::kKBytes, k_scale = k_row + g * (D / 4) / F::kBlock * block;
  const uint32_t v_code = g * token + c * S::kVBytes;
  const uint32_t v_scale = c * S::kElems / F::kBlock * block + c % S::kShare * (16 / S::kShare);
  auto load_k = [&](KHalf<FMT, D, STREAM>& k, const HalfPos& h) {
    k.w.load(uniform(codes[0] + h.code), k_code);
    const GlobalBytes p = uniform(scales[0] + h.scale);
#pragma unroll
    for (int b = 0; b < S::kKBlocks; ++b) k.s[b] = load_as<false, uint8_t>(p, k_scale + b * block);
  };
  auto load_v = [&](VHalf<FMT, D, STREAM>& v, const HalfPos& h) {
#pragma unroll
    for (int j = 0; j < 4; ++j) v.w[j].load(uniform(codes[1] + h.code), v_code + 4 * j * token);
    v.s.load(uniform(scales[1] + h.scale), v_scale);
  };

  // A tile's loads are issued while the tile before it is worked on: K's when its
  // scores are done, V's when its products are; its pages are looked up a tile earlier
  // still.  They are not branched around at the end (the compiler would wait for all of
  // them at once): the last 16 tokens are loaded again then, and not used.  (Two tiles
  // under way at lower occupancy were no faster at any size.)
  const ScalePick pick(c, g);
  const uint32_t third_of = NP == 2 || c < 8 ? kUpperHalves : kZeros;     // (once for each head)
  HalfPos h[2];
  KHalf<FMT, D, STREAM> k[2];
  VHalf<FMT, D, STREAM> v[2];
  int t = begin + wave * kTile;
  if (t < end) {
    int pages[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      h[i] = half_at(t + 16 * i, page_at(t + 16 * i));
      load_k(k[i], h[i]);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      load_v(v[i], h[i]);
      pages[i] = page_at(t + W * kTile + 16 * i);
    }
    do {
      t += W * kTile;
      const HalfPos next[2] = {half_at(t, pages[0]), half_at(t + 16, pages[1])};
      floatx4 x[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        x[i] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int n = 0; n < S::kSteps; ++n) {
          // elements 8 n .. of the lane's part lie in one block
          const uint32_t sc = scale_for<FMT, 0>(k[i].s[8 * n / F::kBlock < S::kKBlocks ? 8 * n / F::kBlock : 0]);
          uintx4 w;
#pragma unroll
          for (int e = 0; e < 4; ++e) w[e] = widen_pair<FMT>(k[i].w.w, 4 * n + e, sc, 0);
          x[i] = mfma<kF16>(w, q[n], x[i]);
        }
        if (h[i].n < 16) {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (4 * j + g >= h[i].n) x[i][j] = -__builtin_inff();
        }
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        load_k(k[i], next[i]);
        pages[i] = page_at(t + W * kTile + 16 * i);
      }

      float best = fmaxf(fmaxf(fmaxf(x[0][0], x[0][1]), fmaxf(x[0][2], x[0][3])),
                         fmaxf(fmaxf(x[1][0], x[1][1]), fmaxf(x[1][2], x[1][3]))) * factor;
      if (__any(best > top + kSlack)) {
        best = fmaxf(best, __shfl_xor(best, 16, 64));
        best = fmaxf(best, __shfl_xor(best, 32, 64));
        const float to = fmaxf(top, best);
        const float by = to == top ? 1.0f : __builtin_amdgcn_exp2f(top - to);
        top = to;
        total *= by;
#pragma unroll
        for (int i = 0; i < S::kElems; ++i) acc[i] *= by;
      }
      const float from = top == -__builtin_inff() ? 0.0f : top - kShift;
      uintx4 p, rest, third;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float u = __builtin_amdgcn_exp2f(__builtin_fmaf(x[j / 2][2 * (j % 2)], factor, -from));
        const float w = __builtin_amdgcn_exp2f(__builtin_fmaf(x[j / 2][2 * (j % 2) + 1], factor, -from));
        total += u + w;
        uint32_t hi, lo;
        if constexpr (kF16) {
          hi = pack2(u, w);
          lo = pack2(u - unpack_lo<true>(hi), w - unpack_hi<true>(hi));
        } else {
          // cut off, not rounded, so that the third part is all that the two leave
          const float u1 = u - upper(u), w1 = w - upper(w);
          hi = upper_pair(u, w, kUpperHalves);
          lo = upper_pair(u1, w1, kUpperHalves);
          third[j] = upper_pair(u1 - upper(u1), w1 - upper(w1), third_of);
        }
        if constexpr (NP == 1) {
          p[j] = c < 8 ? hi : lo;
        } else {
          p[j] = hi;
          rest[j] = lo;
        }
      }

      // V: what is not there is zero codes and scales, whatever the memory holds;
      // pairs of elements of the eight tokens, then pairs of tokens
      uint32_t own[2];              // scale codes of the lane's four tokens
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        own[i] = pick.take<S::kShare>(v[i].s.w);
        if (h[i].n < 16) {
          const int n = h[i].n - g;                 // token 4 j + g is there if 4 j < n
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (4 * j >= n) {
#pragma unroll
              for (auto& w : v[i].w[j].w) w = 0;
              own[i] &= ~(0xFFu << (8 * j));
            }
        }
      }
      uint32_t sc[8];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        sc[4 * i] = scale_for<FMT, 0>(own[i]);
        sc[4 * i + 1] = scale_for<FMT, 1>(own[i]);
        sc[4 * i + 2] = scale_for<FMT, 2>(own[i]);
        sc[4 * i + 3] = scale_for<FMT, 3>(own[i]);
      }
      constexpr int kPart = S::kElems < 8 ? S::kElems : 8;      // elements at once
#pragma unroll
      for (int e0 = 0; e0 < S::kElems; e0 += kPart) {
        uint32_t w[8][kPart / 2];
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
          for (int e = 0; e < kPart / 2; ++e)
            w[j][e] = widen_pair<FMT>(v[j / 4].w[j % 4].w, e0 / 2 + e, sc[j], j & 1);
#pragma unroll
        for (int e = 0; e < kPart; ++e) {
          const uint32_t sel = e % 2 ? 0x07060302u : 0x05040100u;
          uintx4 o;
#pragma unroll
          for (int j = 0; j < 4; ++j) o[j] = __builtin_amdgcn_perm(w[2 * j + 1][e / 2], w[2 * j][e / 2], sel);
          acc[e0 + e] = mfma<kF16>(o, p, acc[e0 + e]);
          if constexpr (NP == 2) acc[e0 + e] = mfma<kF16>(o, rest, acc[e0 + e]);
          if constexpr (!kF16) acc[e0 + e] = mfma<kF16>(o, third, acc[e0 + e]);
        }
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        h[i] = next[i];
        load_v(v[i], h[i]);
      }
    } while (t < end);
  }

  // the waves' sums, lane by lane, in the first
  total += __shfl_xor(total, 16, 64);
  total += __shfl_xor(total, 32, 64);
  if (wave) {
    float(*to)[64] = meet[wave - 1];
#pragma unroll
    for (int e = 0; e < S::kElems; ++e)
#pragma unroll
      for (int i = 0; i < 4; ++i) to[4 * e + i][lane] = acc[e][i];
    to[4 * S::kElems][lane] = top;
    to[4 * S::kElems + 1][lane] = total;
  }
  if constexpr (W > 1) __syncthreads();
  if (wave) return;
  float all = top;
#pragma unroll
  for (int w = 0; w < W - 1; ++w) all = fmaxf(all, meet[w][4 * S::kElems][lane]);
  const float ref = all == -__builtin_inff() ? 0.0f : all;
  {
    const float by = __builtin_amdgcn_exp2f(top - ref);
    total *= by;
#pragma unroll
    for (int e = 0; e < S::kElems; ++e) acc[e] *= by;
  }
#pragma unroll
  for (int w = 0; w < W - 1; ++w) {
    const float by = __builtin_amdgcn_exp2f(meet[w][4 * S::kElems][lane] - ref);
    total += by * meet[w][4 * S::kElems + 1][lane];
#pragma unroll
    for (int e = 0; e < S::kElems; ++e)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[e][i] += by * meet[w][4 * e + i][lane];
  }
  if constexpr (NP == 1) {
    // columns 8 .. hold the sums with p's second part
#pragma unroll
    for (int e = 0; e < S::kElems; ++e)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        acc[e][i] += __uint_as_float(dpp<0x128>(__float_as_uint(acc[e][i])));     // row_ror:8
    if (c >= 8) return;
  }
  if (!mine) return;

  // lane (c, g) has elements (4 g + i) D/16 + e
  const bool whole = item.parts == 1;
  float s_enc, s_dec;
  tensor_scales<FMT>(a.cache, 1, s_enc, s_dec);
  if constexpr (FMT == kKvUe4) s_dec *= 32.0f;
  if (whole) {
    const float by = total > 0.0f || total != total ? s_dec / total : 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t at = row * D + (4 * g + i) * S::kElems;
#pragma unroll
      for (int e = 0; e < S::kElems; e += 4) {
        const float o[4] = {acc[e][i] * by, acc[e + 1][i] * by, acc[e + 2][i] * by, acc[e + 3][i] * by};
        if (a.out_f32)
          *reinterpret_cast<float4*>(static_cast<float*>(a.out) + at + e) = make_float4(o[0], o[1], o[2], o[3]);
        else
          *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + at + e) =
              make_uint2(fp8dev::pack_bf16(o[0], o[1]), fp8dev::pack_bf16(o[2], o[3]));
      }
    }
    if (a.lse && g == 0) a.lse[row] = (all + __builtin_log2f(total) - kShift) / kLog2e;
  } else {
    // sums with V's tensor scale; the maximum and the sum of p apart
    const int64_t at = (kv * a.items + item.base + item.part) * group + (tile * kHeads + col);
    float* o = a.part + at * D;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int e = 0; e < S::kElems; e += 4)
        *reinterpret_cast<float4*>(o + (4 * g + i) * S::kElems + e) =
            make_float4(acc[e][i] * s_dec, acc[e + 1][i] * s_dec, acc[e + 2][i] * s_dec, acc[e + 3][i] * s_dec);
    if (g == 0) part_sums(a)[at] = make_float2(all - kShift, total);
  }
}

}  // namespace

namespace fp4lib {

// One translation unit per format of the cache.
template <>
hipError_t launch_attention_fmt<FP4_KV_FMT>(const AttnArgs& a, uint32_t grid, hipStream_t s) {
  return with_dim(a.cache.head_dim, [&](auto d) {
    constexpr int D = decltype(d)::value;
    auto launch = [&](auto np, auto stream, auto waves) {
      constexpr int W = decltype(waves)::value;
      hipLaunchKernelGGL((k_attention<FP4_KV_FMT, D, decltype(np)::value, decltype(stream)::value, W>), dim3(grid),
                         dim3(64 * W), 0, s, a);
    };
    const bool few = a.q.heads / a.cache.heads <= 8;
    auto by_heads = [&](auto stream, auto waves) {
      if (few) launch(Const<1>(), stream, waves);
      else launch(Const<2>(), stream, waves);
    };
    if (a.waves == 1) by_heads(Const<0>(), Const<1>());
    else if (D <= kWideDim && a.waves == kWideWaves) by_heads(Const<0>(), Const<(D <= kWideDim ? kWideWaves : kWaves)>());
    else if (a.stream) by_heads(Const<1>(), Const<kWaves>());
    else by_heads(Const<0>(), Const<kWaves>());
    return hipGetLastError();
  });
}

}  // namespace fp4lib
