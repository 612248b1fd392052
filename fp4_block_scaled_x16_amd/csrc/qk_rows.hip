// Queries and keys between the projection and attention: RMS norm of each
// head's row, a weight, and rotation by the token's position, forward (also
// straight into a cache, with V) and backward.
//
//   r = (mean(x^2) + eps)^(-1/2),  z = x r w,  y = R z
//   R turns the pair (a, b) of angle t into (a cos t - b sin t, b cos t + a sin t)
//   dz = R^T dy;  dw = sum dz x r;  g = dz w;  dx = r (g - x r^2 mean(g x))
//
// Bound by memory: 2 bytes in and 2 out per element (backward 4 in).  A row
// lies in D / 8 lanes, 16 bytes each.  A rotated pair's other half ("half"
// style: D / 2 lanes' distance or less) is not exchanged between lanes but
// loaded a second time, from the line that is in flight already.  A wave stays
// with one token, whose angles it holds in registers for all of its heads.
#include "kv_common.hpp"

using namespace kvdev;

namespace {

constexpr int kThreads = 256, kWaves = kThreads / 64;

// The lane's 8 elements of a rotation: y = x c + xp s, xp being their partners
// (the sign of sin is in s).
struct Turn {
  float c[8], s[8];
  int partner;          // "half": element from which the partners lie; else -1
  bool turned;
};

template <int D>
__device__ __forceinline__ Turn turn_of(const fp4lib::NormArgs& n, int64_t token, int d0) {
  Turn t;
  t.turned = n.table && d0 < 2 * n.pairs;
  t.partner = -1;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    t.c[i] = 1.0f;
    t.s[i] = 0.0f;
  }
  if (!t.turned) return t;
  const int64_t pos = n.positions[token];
  const bool in = pos >= 0 && pos < n.table_rows;       // outside the table: NaN, and no access
  const float* row = n.table + (in ? pos : 0) * (2 * n.pairs);
  if (n.interleaved) {
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
    t.partner = first ? d0 + n.pairs : d0 - n.pairs;
    const float* p = row + (first ? d0 : d0 - n.pairs);
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

// The partners of the lane's elements v of the row at p.
__device__ __forceinline__ void partners(float (&vp)[8], const float (&v)[8], const uint16_t* p, const Turn& t) {
  if (t.partner >= 0) {
    load8(vp, p + t.partner);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) vp[i] = v[i ^ 1];
  }
}

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
  return 1.0f / __builtin_sqrtf(lane_sum<D / 8>(q) * (1.0f / D) + eps);
}

// Iterations of a token: ceil(heads / rows of a wave) for q, then k, then v.
template <int D, int FMT>
__global__ __launch_bounds__(kThreads) void k_qk_rows(fp4lib::QkRowsArgs a) {
  constexpr int kLanes = D / 8, kRows = 64 / kLanes;
  const int lane = threadIdx.x & 63;
  const int64_t token =
      static_cast<int64_t>(blockIdx.x) * kWaves + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (token >= a.tokens) return;
  const int row = lane / kLanes, d0 = lane % kLanes * 8;
  const Turn t = turn_of<D>(a.norm, token, d0);
  const bool norm = a.norm.w[0] != nullptr;
  int64_t page = 0;
  int place = 0;
  bool kept = false;
  float s_enc[2], s_dec[2];
  if constexpr (FMT >= 0) {
    const int64_t slot = a.slots[token];
    page = slot >> a.cache.page_shift;
    place = static_cast<int>(slot & ((1 << a.cache.page_shift) - 1));
    kept = slot >= 0 && page < a.cache.pages;
    tensor_scales<FMT>(a.cache, 0, s_enc[0], s_dec[0]);
    tensor_scales<FMT>(a.cache, 1, s_enc[1], s_dec[1]);
  }
  const int first = blockIdx.y * a.per_wave, last = min(first + a.per_wave, a.part[3]);
  for (int kind = 0; kind < 3; ++kind) {
    const int lo = max(first, a.part[kind]), hi = min(last, a.part[kind + 1]);
    if (lo >= hi) continue;
    if (FMT >= 0 && kind > 0 && !kept) continue;
    const fp4lib::HeadsArgs& in = a.in[kind];
    // w c and (partner's w) s: y = r (x wc + xp ws)
    float wc[8], ws[8];
    if (kind < 2) {
      weights(wc, a.norm, kind, d0);
      if (t.partner >= 0) {
        weights(ws, a.norm, kind, t.partner);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) ws[i] = wc[i ^ 1];
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        wc[i] *= t.c[i];
        ws[i] *= t.s[i];
      }
    }
    for (int it = lo; it < hi; ++it) {
      const int head = (it - a.part[kind]) * kRows + row;
      const bool valid = head < in.heads;
      const uint16_t* p = in.x + token * in.token + static_cast<int64_t>(valid ? head : 0) * in.head;
      float v[8];
      load8(v, p + d0);
      if (kind < 2) {
        float vp[8];
        if (t.turned) partners(vp, v, p, t);
        const float r = norm ? inv_rms<D>(v, a.norm.eps) : 1.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float y = v[i] * wc[i];
          if (t.turned) y = __builtin_fmaf(vp[i], ws[i], y);
          v[i] = y * r;
        }
      }
      if constexpr (FMT >= 0) {
        if (kind > 0) {
          // a row's lanes are valid together, and so are those of a block
          if (valid)
            encode_row<FMT, D>(v, lane % kLanes, a.cache, kind - 1, page, place, head, s_enc[kind - 1],
                               s_dec[kind - 1]);
          continue;
        }
      }
      if (valid && kind < 2) {
        const fp4lib::HeadsArgs& out = a.out[kind];
        store8(out.x + token * out.token + head * out.head + d0, v);
      }
    }
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
  Turn t;
  bool fresh = true;
  for (int64_t task = begin; task < end; ++task) {
    if (fresh) t = turn_of<D>(a.norm, token, d0);
    fresh = false;
    const int head = it * kRows + row;
    const bool valid = head < hx.heads;
    const int64_t h = valid ? head : 0;
    const uint16_t* px = hx.x + token * hx.token + h * hx.head;
    const uint16_t* py = hdy.x + token * hdy.token + h * hdy.head;
    float x[8], dz[8];
    load8(x, px + d0);
    load8(dz, py + d0);
    if (t.turned) {
      float dp[8];
      partners(dp, dz, py, t);
#pragma unroll
      for (int i = 0; i < 8; ++i) dz[i] = dz[i] * t.c[i] - dp[i] * t.s[i];
    }
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
    if (valid) store8(hdx.x + token * hdx.token + h * hdx.head + d0, dz);
    if (++it == iters) {
      it = 0;
      ++token;
      fresh = true;
    }
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

// The workgroups' sums in their order: 32 columns per workgroup, 8 threads each.
__global__ __launch_bounds__(256) void k_qk_grad_join(fp4lib::QkGradArgs a) {
  __shared__ float sum[8][32];
  const int which = blockIdx.y, col = threadIdx.x & 31, r = threadIdx.x >> 5;
  if (!a.dw[which]) return;
  const float* p = a.part + (which ? static_cast<int64_t>(a.groups[0]) * a.head_dim : 0) + blockIdx.x * 32 + col;
  float v = 0.0f;
#pragma unroll 8
  for (int g = r; g < a.groups[which]; g += 8) v += p[static_cast<int64_t>(g) * a.head_dim];
  sum[r][col] = v;
  __syncthreads();
  if (r) return;
  for (int k = 1; k < 8; ++k) v += sum[k][col];
  float* dw = a.dw[which] + blockIdx.x * 32 + col;
  *dw = a.accumulate ? *dw + v : v;
}

constexpr int kGradGroupsPerCu = 4;

}  // namespace

namespace fp4lib {

hipError_t launch_qk_rows(const QkRowsArgs& args, hipStream_t s) {
  QkRowsArgs a = args;
  const int rows = 512 / a.head_dim;       // of a wave
  for (int i = 0; i < 3; ++i) a.part[i + 1] = a.part[i] + (a.in[i].x ? (a.in[i].heads + rows - 1) / rows : 0);
  // enough waves for 16 on a CU before a wave takes several rows
  const int64_t want = a.tokens * a.part[3] / (16 * static_cast<int64_t>(device_cu_count()));
  a.per_wave = static_cast<int>(want < 1 ? 1 : want < a.part[3] ? want : a.part[3]);
  const dim3 grid(static_cast<uint32_t>((a.tokens + kWaves - 1) / kWaves),
                  (a.part[3] + a.per_wave - 1) / a.per_wave);
  return with_dim(a.head_dim, [&](auto d) {
    constexpr int D = decltype(d)::value;
    if (!a.cached) {
      hipLaunchKernelGGL((k_qk_rows<D, -1>), grid, dim3(kThreads), 0, s, a);
      return hipGetLastError();
    }
    return with_format(a.cache.fmt, [&](auto f) {
      hipLaunchKernelGGL((k_qk_rows<D, decltype(f)::value>), grid, dim3(kThreads), 0, s, a);
      return hipGetLastError();
    });
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
  // workgroups in proportion to the rows, at least one for each side that has any
  const int64_t cap = static_cast<int64_t>(device_cu_count()) * kGradGroupsPerCu;
  const int64_t total = all < cap * kWaves ? (all + kWaves - 1) / kWaves + 1 : cap;
  const int64_t k = tasks[1] ? total * tasks[1] / all : 0;
  a.groups[1] = static_cast<int>(tasks[1] && k < 1 ? 1 : k);
  a.groups[0] = static_cast<int>(tasks[0] ? (total - a.groups[1] < 1 ? 1 : total - a.groups[1]) : 0);
  return with_dim(a.head_dim, [&](auto d) {
    constexpr int D = decltype(d)::value;
    if (all) hipLaunchKernelGGL(k_qk_grad<D>, dim3(a.groups[0] + a.groups[1]), dim3(kThreads), 0, s, a);
    if (a.dw[0] || a.dw[1]) hipLaunchKernelGGL(k_qk_grad_join, dim3(D / 32, 2), dim3(256), 0, s, a);
    return hipGetLastError();
  });
}

}  // namespace fp4lib
