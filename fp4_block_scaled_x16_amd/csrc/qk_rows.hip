// Queries and keys between the projection and attention: RMS norm of each
// head's row, a weight, and rotation by the token's position, forward (also
// straight into a cache, with V) and backward.
//
//   r = (mean(x^2) + eps)^(-1/2),  z = x r w,  y = R z
//   R turns the pair (a, b) of angle t into (a cos t - b sin t, b cos t + a sin t)
//   dz = R^T dy;  dw = sum dz x r;  g = dz w;  dx = r (g - x r^2 mean(g x))
//
// Bound by memory: 2 bytes in and 2 out per element (backward 4 in, 2 out).  8192 tokens
// of 32 + 8 heads of 128 take 33.9 us, 5.1 TB/s, where a large copy reaches 5.0 to 5.2;
// backward 53.4 us, 4.8 TB/s; 8192 tokens normed, turned and written to an MXFP8 cache 41.5 us,
// 4.6 TB/s (MXFP4 44.0, NVFP4 47.0), without a norm K and V alone 12 us (NVFP4 14.5); 64 of them
// normed to an FP8 cache 4.0 us, of which a launch is 3.
//
// A row lies in D / 8 lanes, 16 bytes each.  A rotated pair's other half ("half"
// style: D / 2 lanes' distance or less) is not exchanged between lanes but loaded a
// second time, from the line that is in flight already.  Forward, a workgroup has
// one token (up to 512 / 64 waves of its rows), whose angles a wave holds for all of
// its heads; backward, a wave has a run of consecutive rows.
#include "kv_common.hpp"

using namespace kvdev;

namespace {

constexpr int kThreads = 256, kWaves = kThreads / 64;
constexpr int kManyRows = 4;
constexpr int kRowWaves = 8;      // of a workgroup of the forward pass, at most
// Rows of k or v that go into a cache, where q has r: 64-bit sums take registers.
constexpr int coded_rows_of(int r) { return r > 1 ? 2 : 1; }

// "half" style: element from which the partners of the lane's elements d0 .. lie;
// -1 where they are neighbours, or not turned.
__device__ __forceinline__ int partner_of(const fp4lib::NormArgs& n, int d0) {
  if (!n.table || n.interleaved || d0 >= 2 * n.pairs) return -1;
  return d0 < n.pairs ? d0 + n.pairs : d0 - n.pairs;
}

// The rotation of the lane's 8 elements: y = x c + xp s, xp being their partners
// (the sign of sin is in s).
struct Turn {
  float c[8], s[8];
};

__device__ __forceinline__ Turn turn_of(const fp4lib::NormArgs& n, int64_t token, int d0, int partner) {
  Turn t;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    t.c[i] = 1.0f;
    t.s[i] = 0.0f;
  }
  if (!n.table || d0 >= 2 * n.pairs) return t;
  const int64_t pos = n.positions[token];
  const bool in = pos >= 0 && pos < n.table_rows;       // outside the table: NaN, and no access
  const float* row = n.table + (in ? pos : 0) * (2 * n.pairs);
  if (partner < 0) {
    const float4 c = *reinterpret_cast<const float4*>(row + d0 / 2);
    const float4 s = *reinterpret_cast<const float4*>(row + n.pairs + d0 / 2);
    const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      t.c[i] = cc[i / 2];
      t.s[i] = i % 2 ? ss[i / 2] : -ss[i / 2];
    }
  } else {
    const bool first = d0 < n.pairs;
    const float* p = row + (first ? d0 : partner);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float4 c = *reinterpret_cast<const float4*>(p + 4 * h);
      const float4 s = *reinterpret_cast<const float4*>(p + n.pairs + 4 * h);
      const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        t.c[4 * h + i] = cc[i];
        t.s[4 * h + i] = first ? -ss[i] : ss[i];
      }
    }
  }
  if (!in) {
#pragma unroll
    for (int i = 0; i < 8; ++i) t.c[i] = __builtin_nanf("");
  }
  return t;
}

// A lane's elements of a row and, in "half" style, their partners, as they lie in memory.
struct RawRow {
  uint4 v, p;
  __device__ __forceinline__ void load(const uint16_t* row, int d0, int partner) {
    v = *reinterpret_cast<const uint4*>(row + d0);
    if (partner >= 0) p = *reinterpret_cast<const uint4*>(row + partner);
  }
  __device__ __forceinline__ void values(float (&x)[8], float (&xp)[8], int partner) const {
    fp4quant::unpack8(v, x);
    if (partner >= 0) {
      fp4quant::unpack8(p, xp);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) xp[i] = x[i ^ 1];
    }
  }
};

__device__ __forceinline__ void weights(float (&w)[8], const fp4lib::NormArgs& n, int which, int d) {
  if (!n.w[which]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = 1.0f;
  } else if (n.w_f32) {
    const float* p = static_cast<const float*>(n.w[which]) + d;
    const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
    w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w, w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
  } else {
    load8(w, static_cast<const uint16_t*>(n.w[which]) + d);
  }
}

template <int D>
__device__ __forceinline__ float inv_rms(const float (&v)[8], float eps) {
  float q = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) q = __builtin_fmaf(v[i], v[i], q);
  return __builtin_amdgcn_rsqf(lane_sum<D / 8>(q) * (1.0f / D) + eps);      // within an ulp
}

// The same in 64 bits, in which the squares of bf16 elements are exact.
template <int D>
__device__ __forceinline__ double inv_rms64(const float (&v)[8], float eps) {
  double q = 0.0;
#pragma unroll
  for (int i = 0; i < 8; ++i) q = __builtin_fma(static_cast<double>(v[i]), static_cast<double>(v[i]), q);
  const double a = lane_sum<D / 8>(q) * (1.0 / D) + eps, r = __builtin_amdgcn_rsq(a);
  const double off = __builtin_fma(-a * r, r, 1.0);
  return __builtin_fabs(off) < 0.5 ? __builtin_fma(0.5 * r, off, r) : r;       // (0 and infinity as they are)
}

// To fp32 such that a second rounding, to fewer bits, gives what one from z gives: what
// is cut off leaves a mark in the last bit.
__device__ __forceinline__ float to_odd(double z) {
  const float f = static_cast<float>(z);
  const double back = f;
  uint32_t b = __float_as_uint(f);
  if (__builtin_fabs(back) > __builtin_fabs(z)) b -= 1;       // (of the magnitude)
  return __uint_as_float(back == z || z != z ? b : b | 1u);
}

// Rows of k or v into their slot: from head0 on, every kRows-th.
//
// What a norm or a rotation gives is formed in 64 bits and, rounded to odd in fp32, handed to the
// encoder.  A scale that is a power of two then gives the code of one rounding (NVFP4's and UE5M3's
// are none: their product with the inverse scale is rounded in fp32 as fp4_quantize rounds it).
// With all of it in fp32 a value next to a border between two codes would now and then fall on
// its other side, 6 or 12 % away (12 of 8 million elements, as many as in elementary fp32
// operations; 8192 tokens to an MXFP8 cache took 40.7 us, and 64 to an FP8 one 3.4).
template <int D, int FMT, int R>
__device__ __forceinline__ void coded_rows(const fp4lib::QkRowsArgs& a, int kind, int64_t token, int head0, int lane) {
  constexpr int kLanes = D / 8, kRows = 64 / kLanes;
  const fp4lib::HeadsArgs& in = a.in[kind];
  const int d0 = lane % kLanes * 8;
  const int partner = kind == 1 ? partner_of(a.norm, d0) : -1;
  RawRow raw[R];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int head = head0 + i * kRows < in.heads ? head0 + i * kRows : 0;
    raw[i].load(in.x + token * in.token + static_cast<int64_t>(head) * in.head, d0, partner);
  }
  const int64_t slot = a.slots[token], page = slot >> a.cache.page_shift;
  const int place = static_cast<int>(slot & ((1 << a.cache.page_shift) - 1));
  if (slot < 0 || page >= a.cache.pages) return;
  float s_enc = 1.0f, s_dec = 1.0f;
  tensor_scales<FMT>(a.cache, kind - 1, s_enc, s_dec);
  const bool norm = a.norm.w[1] != nullptr, turned = a.norm.table && d0 < 2 * a.norm.pairs;
  if (kind == 1 && (norm || a.norm.table)) {
    // y = r (x wc + xp ws): w c, and the partner's w s (products of two fp32 numbers: exact)
    double wc[8], ws[8];
    {
      const Turn t = turn_of(a.norm, token, d0, partner);
      float w[8];
      weights(w, a.norm, 1, d0);
#pragma unroll
      for (int e = 0; e < 8; ++e) wc[e] = static_cast<double>(w[e]) * t.c[e];
      if (partner >= 0) weights(w, a.norm, 1, partner);
#pragma unroll
      for (int e = 0; e < 8; ++e) ws[e] = static_cast<double>(w[partner >= 0 ? e : e ^ 1]) * t.s[e];
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
      float v[8], vp[8];
      raw[i].values(v, vp, partner);
      const double r = norm ? inv_rms64<D>(v, a.norm.eps) : 1.0;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        double z = v[e] * wc[e];
        if (turned) z = __builtin_fma(static_cast<double>(vp[e]), ws[e], z);
        v[e] = to_odd(z * r);
      }
      if (head0 + i * kRows < in.heads)          // a row's lanes together
        encode_row<FMT, D>(v, lane % kLanes, a.cache, 0, page, place, head0 + i * kRows, s_enc, s_dec);
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < R; ++i) {
    float v[8];
    fp4quant::unpack8(raw[i].v, v);
    if (head0 + i * kRows < in.heads)
      encode_row<FMT, D>(v, lane % kLanes, a.cache, kind - 1, page, place, head0 + i * kRows, s_enc, s_dec);
  }
}

// A wave has R times (k and v for a cache: coded_rows_of(R) times) 64 / (D / 8) rows of one
// token, all of q, of k or of v (a.part[kind] is the first wave of the kind), whose
// loads it issues before anything else; a workgroup has neighbouring rows of a token.
template <int D, int FMT, int R>
__global__ __launch_bounds__(64 * kRowWaves) void k_qk_rows(fp4lib::QkRowsArgs a) {
  constexpr int kLanes = D / 8, kRows = 64 / kLanes;
  const int lane = threadIdx.x & 63;
  const int64_t token = blockIdx.x;
  const int part = blockIdx.y * (blockDim.x >> 6) + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (part >= a.part[3]) return;
  const int kind = part < a.part[1] ? 0 : part < a.part[2] ? 1 : 2;
  if constexpr (FMT >= 0) {
    if (kind > 0) {
      coded_rows<D, FMT, coded_rows_of(R)>(a, kind, token,
                                           (part - a.part[kind]) * (coded_rows_of(R) * kRows) + lane / kLanes, lane);
      return;
    }
  }
  const fp4lib::HeadsArgs& in = a.in[kind];
  const int d0 = lane % kLanes * 8, head0 = (part - a.part[kind]) * (R * kRows) + lane / kLanes;
  const int partner = partner_of(a.norm, d0);
  RawRow raw[R];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int head = head0 + i * kRows < in.heads ? head0 + i * kRows : 0;
    raw[i].load(in.x + token * in.token + static_cast<int64_t>(head) * in.head, d0, partner);
  }
  // y = r (x wc + xp ws): w c, and the partner's w s
  float wc[8], ws[8];
  const Turn t = turn_of(a.norm, token, d0, partner);
  weights(wc, a.norm, kind, d0);
  if (partner >= 0) {
    weights(ws, a.norm, kind, partner);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) ws[i] = wc[i ^ 1];
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    wc[i] *= t.c[i];
    ws[i] *= t.s[i];
  }
  const bool norm = a.norm.w[0] != nullptr, turned = a.norm.table && d0 < 2 * a.norm.pairs;
  const fp4lib::HeadsArgs& out = a.out[kind];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int head = head0 + i * kRows;
    float v[8], vp[8];
    raw[i].values(v, vp, partner);
    const float r = norm ? inv_rms<D>(v, a.norm.eps) : 1.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      float y = v[e] * wc[e];
      if (turned) y = __builtin_fmaf(vp[e], ws[e], y);
      v[e] = y * r;
    }
    if (head < in.heads) store8(out.x + token * out.token + head * out.head + d0, v);      // a row's lanes together
  }
}

// Backward: a persistent grid, its first groups[0] workgroups on q and the rest
// on k; a wave takes consecutive (token, rows) tasks and keeps its lanes' part
// of the weight's gradient in registers.
template <int D>
__global__ __launch_bounds__(kThreads) void k_qk_grad(fp4lib::QkGradArgs a) {
  constexpr int kLanes = D / 8, kRows = 64 / kLanes;
  __shared__ float sum[kWaves * kRows][D];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int row = lane / kLanes, d0 = lane % kLanes * 8;
  const int which = static_cast<int>(blockIdx.x) >= a.groups[0];
  const int group = blockIdx.x - (which ? a.groups[0] : 0);
  const fp4lib::HeadsArgs &hx = a.x[which], &hdy = a.dy[which], &hdx = a.dx[which];
  const bool norm = a.norm.w[which] != nullptr;
  const int iters = (hx.heads + kRows - 1) / kRows;
  const int64_t tasks = a.tokens * iters, waves = static_cast<int64_t>(a.groups[which]) * kWaves;
  const int64_t w = static_cast<int64_t>(group) * kWaves + wave;
  // tasks w * tasks / waves .. (the products stay below 2^63: tasks < 2^42)
  const int64_t begin = tasks * w / waves, end = tasks * (w + 1) / waves;
  float wt[8], dw[8];
  weights(wt, a.norm, which, d0);
#pragma unroll
  for (int i = 0; i < 8; ++i) dw[i] = 0.0f;
  int64_t token = begin / iters;
  int it = static_cast<int>(begin - token * iters);
  const int partner = partner_of(a.norm, d0);
  const bool turned = a.norm.table && d0 < 2 * a.norm.pairs;
  Turn t;
  RawRow rx, ry;
  auto load = [&](RawRow& x, RawRow& y, int64_t token, int it) {
    const int64_t h = it * kRows + row < hx.heads ? it * kRows + row : 0;
    // read once, past the caches (57 instead of 65 us for 8192 tokens; dy's line is read
    // again for the partners)
    x.v = __builtin_bit_cast(uint4, __builtin_nontemporal_load(reinterpret_cast<const words4*>(
                                        hx.x + token * hx.token + h * hx.head + d0)));
    y.load(hdy.x + token * hdy.token + h * hdy.head, d0, partner);
  };
  if (begin < end) {
    load(rx, ry, token, it);
    t = turn_of(a.norm, token, d0, partner);
  }
  for (int64_t task = begin; task < end; ++task) {
    const int64_t h = it * kRows + row;
    const bool valid = h < hx.heads;
    uint16_t* out = hdx.x + token * hdx.token + h * hdx.head + d0;
    float x[8], dz[8], dp[8];
    fp4quant::unpack8(rx.v, x);
    ry.values(dz, dp, partner);
    if (turned) {
#pragma unroll
      for (int i = 0; i < 8; ++i) dz[i] = dz[i] * t.c[i] - dp[i] * t.s[i];
    }
    // the next rows' loads, before these are worked on (behind the last: these again)
    const bool turn_page = it + 1 == iters && task + 1 < end;
    if (task + 1 < end) it = turn_page ? 0 : it + 1;
    if (turn_page) ++token;
    load(rx, ry, token, it);
    if (turn_page) t = turn_of(a.norm, token, d0, partner);
    if (norm) {
      const float r = inv_rms<D>(x, a.norm.eps);
      float gx = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float xr = x[i] * r;
        if (valid) dw[i] = __builtin_fmaf(dz[i], xr, dw[i]);
        dz[i] *= wt[i];
        x[i] = xr;
        gx = __builtin_fmaf(dz[i], xr, gx);
      }
      const float m = lane_sum<D / 8>(gx) * (1.0f / D);
#pragma unroll
      for (int i = 0; i < 8; ++i) dz[i] = r * (dz[i] - x[i] * m);
    }
    if (valid) store8(out, dz);
  }
  if (!norm || !a.part) return;
#pragma unroll
  for (int i = 0; i < 8; ++i) sum[wave * kRows + row][d0 + i] = dw[i];
  __syncthreads();
  for (int d = threadIdx.x; d < D; d += kThreads) {
    float v = 0.0f;
#pragma unroll
    for (int k = 0; k < kWaves * kRows; ++k) v += sum[k][d];
    a.part[static_cast<int64_t>(blockIdx.x) * D + d] = v;
  }
}

// The workgroups' sums in their order: 32 columns per workgroup, 32 threads each.
__global__ __launch_bounds__(1024) void k_qk_grad_join(fp4lib::QkGradArgs a) {
  __shared__ float sum[32][33];
  const int which = blockIdx.y, col = threadIdx.x & 31, r = threadIdx.x >> 5;
  if (!a.dw[which]) return;
  const int n = a.groups[which];
  const float* p = a.part + (which ? static_cast<int64_t>(a.groups[0]) * a.head_dim : 0) + blockIdx.x * 32 + col;
  float v = 0.0f;
  for (int g = r; g < n; g += 16 * 32) {
    float w[16];           // all under way at once, behind the last the last again
#pragma unroll
    for (int k = 0; k < 16; ++k) w[k] = p[static_cast<int64_t>(min(g + 32 * k, n - 1)) * a.head_dim];
#pragma unroll
    for (int k = 0; k < 16; ++k) v += g + 32 * k < n ? w[k] : 0.0f;
  }
  sum[r][col] = v;
  __syncthreads();
  // thread (row r, column col): sums of column r of this workgroup's 32
  v = sum[col][r];
  v = lane_sum<32>(v);
  if (col) return;
  float* dw = a.dw[which] + blockIdx.x * 32 + r;
  *dw = a.accumulate ? *dw + v : v;
}

// What the registers leave room for at once (8192 tokens of 32 + 8 heads of 128: 3 / 4 / 5 / 8
// per CU 62.6 / 56.7 / 53.4 / 58.2 us).
constexpr int kGradGroupsPerCu = 5;

}  // namespace

namespace fp4lib {

// kManyRows for long sequences (8192 tokens of 32 + 8 heads of 128, before the stores went past
// the caches: R = 1 / 2 / 3 / 4 / 5 50 / 41.5 / 40.2 / 39.2 / 41.4 us; of one token's waves in one
// workgroup, with 4 tokens' waves of one kind instead 41.3); 1 where that leaves CUs with
// fewer than 8 waves.
hipError_t launch_qk_rows(const QkRowsArgs& args, hipStream_t s) {
  QkRowsArgs a = args;
  auto parts = [&](int r) {
    for (int i = 0; i < 3; ++i) {
      const int rows = (a.cached && i > 0 ? coded_rows_of(r) : r) * 512 / a.head_dim;       // of a wave
      a.part[i + 1] = a.part[i] + (a.in[i].x ? (a.in[i].heads + rows - 1) / rows : 0);
    }
    return a.part[3];
  };
  const bool many = a.tokens * parts(kManyRows) >= 8 * static_cast<int64_t>(device_cu_count());
  const int all = many ? a.part[3] : parts(1), waves = all < kRowWaves ? all : kRowWaves;
  // a grid has fewer than 2^32 threads along x
  constexpr int64_t kMostTokens = int64_t(1) << 22;
  if (a.tokens > kMostTokens) {
    for (int64_t first = 0; first < args.tokens; first += kMostTokens) {
      a = args;
      a.tokens = args.tokens - first < kMostTokens ? args.tokens - first : kMostTokens;
      for (auto& h : a.in)
        if (h.x) h.x += first * h.token;
      for (auto& h : a.out)
        if (h.x) h.x += first * h.token;
      if (a.norm.positions) a.norm.positions += first;
      if (a.slots) a.slots += first;
      const hipError_t e = launch_qk_rows(a, s);
      if (e != hipSuccess) return e;
    }
    return hipSuccess;
  }
  const dim3 grid(static_cast<uint32_t>(a.tokens), (all + waves - 1) / waves), block(64 * waves);
  return with_dim(a.head_dim, [&](auto d) {
    constexpr int D = decltype(d)::value;
    auto launch = [&](auto f) {
      constexpr int F = decltype(f)::value;
      if (many) hipLaunchKernelGGL((k_qk_rows<D, F, kManyRows>), grid, block, 0, s, a);
      else hipLaunchKernelGGL((k_qk_rows<D, F, 1>), grid, block, 0, s, a);
      return hipGetLastError();
    };
    return a.cached ? with_format(a.cache.fmt, launch) : launch(Const<-1>());
  });
}

// The most workgroups that a backward pass has: the workspace does not
// depend on the other sizes.
int64_t qk_grad_workspace(int head_dim) {
  return static_cast<int64_t>(device_cu_count()) * kGradGroupsPerCu * head_dim * sizeof(float);
}

hipError_t launch_qk_grad(const QkGradArgs& args, hipStream_t s) {
  QkGradArgs a = args;
  const int rows = 512 / a.head_dim;
  int64_t tasks[2], all = 0;
  for (int i = 0; i < 2; ++i) {
    tasks[i] = a.x[i].x ? a.tokens * ((a.x[i].heads + rows - 1) / rows) : 0;
    all += tasks[i];
  }
  // As few workgroups as give no wave more tasks than it has with all of them (1001 tokens
  // of 32 + 32 heads of 64: 1001 workgroups of two tasks a wave 12.0 us, 1280 13.3, 2002 of
  // one 17.5); in proportion to the rows, at least one for each side that has any.
  const int64_t cap = static_cast<int64_t>(device_cu_count()) * kGradGroupsPerCu;
  const int64_t each = all ? (all + cap * kWaves - 1) / (cap * kWaves) * kWaves : 1;
  const int64_t total = (all + each - 1) / each < cap ? (all + each - 1) / each : cap;
  const int64_t k = tasks[1] ? total * tasks[1] / all : 0;
  a.groups[1] = static_cast<int>(tasks[1] && k < 1 ? 1 : k);
  a.groups[0] = static_cast<int>(tasks[0] ? (total - a.groups[1] < 1 ? 1 : total - a.groups[1]) : 0);
  return with_dim(a.head_dim, [&](auto d) {
    constexpr int D = decltype(d)::value;
    if (all) hipLaunchKernelGGL(k_qk_grad<D>, dim3(a.groups[0] + a.groups[1]), dim3(kThreads), 0, s, a);
    if (a.dw[0] || a.dw[1]) hipLaunchKernelGGL(k_qk_grad_join, dim3(D / 32, 2), dim3(1024), 0, s, a);
    return hipGetLastError();
  });
}

}  // namespace fp4lib
