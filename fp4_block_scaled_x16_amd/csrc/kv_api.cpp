// The C ABI's attention calls (include/fp4.h): norm and rotation of queries and
// keys, the paged key-value cache, attention of one new token.  Host-side argument
// checks, then launches; no check touches a HIP API, so rejected calls work
// without a GPU.
#include <cmath>

#include "../../include/fp4_selftest.h"
#include "api_common.hpp"
#include "kv_internal.hpp"

using namespace fp4api;

namespace {

constexpr int64_t kMaxTokens = int64_t(1) << 31;
constexpr int64_t kMaxHeads = 1024;

bool aligned(const void* p, size_t bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }

bool head_dim_ok(int64_t d) { return d == 64 || d == 128 || d == 256; }

fp4_status check_tokens(const char* what, int64_t n) {
  if (n < 0) return fail(FP4_ERR_SHAPE, "negative %s=%lld", what, (long long)n);
  if (n >= kMaxTokens) return fail(FP4_ERR_SHAPE, "%s=%lld must be below 2^31", what, (long long)n);
  return FP4_OK;
}

fp4_status check_head_dim(int64_t d) {
  if (!head_dim_ok(d))
    return fail(FP4_ERR_UNSUPPORTED, "head_dim=%lld: 64, 128 and 256 are supported", (long long)d);
  return FP4_OK;
}

// Rows of heads; outputs must not overlap.
fp4_status check_heads(const char* name, const fp4_heads* h, int64_t tokens, int64_t head_dim, bool output) {
  if (!h) return fail(FP4_ERR_ARG, "%s is null", name);
  if (h->heads < 1 || h->heads > kMaxHeads)
    return fail(FP4_ERR_SHAPE, "%s: heads=%lld must be 1 .. %lld", name, (long long)h->heads, (long long)kMaxHeads);
  if (tokens == 0) return FP4_OK;
  if (!h->x) return fail(FP4_ERR_ARG, "%s: x is null", name);
  if (!aligned16(h->x)) return fail(FP4_ERR_ARG, "%s must be 16-byte aligned", name);
  if (h->token_stride < 0 || h->head_stride < 0 || h->token_stride % 8 || h->head_stride % 8)
    return fail(FP4_ERR_ARG, "%s: strides must be multiples of 8, not negative", name);
  if (output) {
    // one of the two strides steps over the other's whole extent (which may pass 63 bits)
    using Wide = __int128;
    const Wide by_head = Wide(h->heads - 1) * h->head_stride + head_dim;
    const Wide by_token = Wide(tokens - 1) * h->token_stride + head_dim;
    const bool heads_apart = h->heads == 1 || h->head_stride >= head_dim;
    const bool tokens_outer = heads_apart && (tokens == 1 || h->token_stride >= by_head);
    const bool heads_outer = (tokens == 1 || h->token_stride >= head_dim) &&
                             (h->heads == 1 || h->head_stride >= by_token);
    if (!tokens_outer && !heads_outer) return fail(FP4_ERR_ARG, "%s: rows overlap", name);
  }
  return FP4_OK;
}

fp4lib::HeadsArgs heads_args(const fp4_heads* h) {
  return h ? fp4lib::HeadsArgs{h->x, h->token_stride, h->head_stride, static_cast<int>(h->heads)}
           : fp4lib::HeadsArgs{};
}

fp4_status check_norm(const fp4_qk_norm* n, const int64_t* positions, int64_t tokens, int64_t head_dim) {
  if (!n) return fail(FP4_ERR_ARG, "norm is null");
  if (!n->q_weight != !n->k_weight) return fail(FP4_ERR_ARG, "q_weight and k_weight are given together or not at all");
  if (!n->q_weight && !n->table) return fail(FP4_ERR_ARG, "neither weights nor a table");
  if (n->q_weight) {
    if (!aligned16(n->q_weight) || !aligned16(n->k_weight))
      return fail(FP4_ERR_ARG, "weights must be 16-byte aligned");
    if (!std::isfinite(n->eps) || n->eps < 0) return fail(FP4_ERR_ARG, "eps must be finite and not negative");
  }
  if (n->table) {
    if (!aligned16(n->table)) return fail(FP4_ERR_ARG, "the table must be 16-byte aligned");
    if (n->rotary_dim < 16 || n->rotary_dim > head_dim || n->rotary_dim % 16)
      return fail(FP4_ERR_SHAPE, "rotary_dim=%d must be a multiple of 16 up to head_dim", n->rotary_dim);
    if (n->table_rows < 1) return fail(FP4_ERR_SHAPE, "table_rows=%lld must be positive", (long long)n->table_rows);
    if (tokens > 0 && !positions) return fail(FP4_ERR_ARG, "positions is null");
    if (!aligned(positions, 8)) return fail(FP4_ERR_ARG, "positions must be aligned to their elements");
  }
  return FP4_OK;
}

fp4lib::NormArgs norm_args(const fp4_qk_norm* n, const int64_t* positions) {
  fp4lib::NormArgs a{};
  if (!n) return a;
  a.w[0] = n->q_weight;
  a.w[1] = n->k_weight;
  a.w_f32 = n->weight_f32;
  a.eps = n->eps;
  a.table = n->table;
  a.table_rows = n->table_rows;
  a.pairs = n->rotary_dim / 2;
  a.interleaved = n->interleaved;
  a.positions = positions;
  return a;
}

// The launcher's number of a format, -1 for one that no cache has.
int cache_format(int f) {
  switch (f) {
    case FP4_FP8_E4M3: return fp4lib::kKvFp8;
    case FP4_MXFP8: return fp4lib::kKvMx8;
    case FP4_MXFP4: return fp4lib::kKvMx4;
    case FP4_NVFP4: return fp4lib::kKvNv4;
    case FP4_UE5M3: return fp4lib::kKvUe4;
    default: return -1;
  }
}

int log2_of(int v) {
  int k = 0;
  while (v >> (k + 1)) ++k;
  return k;
}

fp4_status check_cache(const fp4_kv_cache* c) {
  if (!c) return fail(FP4_ERR_ARG, "cache is null");
  if (cache_format(c->format) < 0)
    return fail(FP4_ERR_UNSUPPORTED, "format %d: a cache is FP8_E4M3, MXFP8, MXFP4, NVFP4 or UE5M3", (int)c->format);
  fp4_status st = check_head_dim(c->head_dim);
  if (st) return st;
  if (c->heads < 1 || c->heads > kMaxHeads)
    return fail(FP4_ERR_SHAPE, "cache heads=%d must be 1 .. %lld", c->heads, (long long)kMaxHeads);
  if (c->page_size < 16 || c->page_size > 1024 || (c->page_size & (c->page_size - 1)))
    return fail(FP4_ERR_SHAPE, "page_size=%d must be a power of two, 16 .. 1024", c->page_size);
  if (c->pages < 1 || c->pages >= kMaxTokens)
    return fail(FP4_ERR_SHAPE, "pages=%lld must be 1 .. 2^31 - 1", (long long)c->pages);
  const void* p[4] = {c->k_codes, c->k_scales, c->v_codes, c->v_scales};
  for (const void* q : p) {
    if (!q) return fail(FP4_ERR_ARG, "cache: codes/scales are null");
    if (!aligned16(q)) return fail(FP4_ERR_ARG, "cache: codes and scales must be 16-byte aligned");
  }
  const int64_t codes[3] = {c->page_stride, c->head_stride, c->token_stride};
  const int64_t scales[3] = {c->scale_page_stride, c->scale_head_stride, c->scale_block_stride};
  constexpr int64_t kMost = int64_t(1) << 31;
  for (int i = 0; i < 3; ++i)
    if (codes[i] <= 0 || codes[i] % 16 || scales[i] <= 0 || scales[i] % 16)
      return fail(FP4_ERR_ARG, "cache: strides must be positive multiples of 16");
  if (codes[0] >= 2 * kMost || scales[0] >= 2 * kMost)
    return fail(FP4_ERR_SHAPE, "cache: page strides must be below 2^32");
  // within a page the kernels' offsets are 32 bits wide
  if (codes[1] >= kMost || codes[2] >= kMost || scales[1] >= kMost || scales[2] >= kMost ||
      (c->heads - 1) * codes[1] + c->page_size * codes[2] >= kMost ||
      (c->heads - 1) * scales[1] + 16 * scales[2] + c->page_size >= kMost)
    return fail(FP4_ERR_SHAPE, "cache: offsets within a page must be below 2^31");
  const int row = c->head_dim / (c->format == FP4_FP8_E4M3 || c->format == FP4_MXFP8 ? 1 : 2);
  if (codes[2] < row) return fail(FP4_ERR_ARG, "cache: token_stride=%lld below a row's %d bytes", (long long)codes[2], row);
  if (c->format == FP4_NVFP4 || c->format == FP4_UE5M3) {
    if (!c->amax || !aligned(c->amax, 4))
      return fail(FP4_ERR_ARG, "cache: amax must be non-null and aligned to its elements");
    if (!std::isfinite(c->target) || c->target <= 0) return fail(FP4_ERR_ARG, "cache: target must be finite and positive");
  }
  return FP4_OK;
}

fp4lib::KvCacheArgs cache_args(const fp4_kv_cache* c) {
  fp4lib::KvCacheArgs a{};
  a.codes[0] = c->k_codes;
  a.codes[1] = c->v_codes;
  a.scales[0] = c->k_scales;
  a.scales[1] = c->v_scales;
  a.page = c->page_stride;
  a.head = c->head_stride;
  a.token = c->token_stride;
  a.s_page = c->scale_page_stride;
  a.s_head = c->scale_head_stride;
  a.s_block = c->scale_block_stride;
  a.pages = c->pages;
  a.amax = c->amax;
  a.target = c->target;
  a.fmt = cache_format(c->format);
  a.heads = c->heads;
  a.head_dim = c->head_dim;
  a.page_shift = log2_of(c->page_size);
  return a;
}

// An input and its output: both there or neither, with the same heads.
fp4_status check_pair(const char* in_name, const fp4_heads* in, const char* out_name, const fp4_heads* out,
                      int64_t tokens, int64_t head_dim) {
  if (!in && !out) return FP4_OK;
  fp4_status st = check_heads(in_name, in, tokens, head_dim, false);
  if (!st) st = check_heads(out_name, out, tokens, head_dim, true);
  if (st) return st;
  if (in->heads != out->heads)
    return fail(FP4_ERR_SHAPE, "%s has %lld heads, %s %lld", in_name, (long long)in->heads, out_name,
                (long long)out->heads);
  return FP4_OK;
}

}  // namespace

FP4_EXPORT fp4_status fp4_qk_norm_rope(const fp4_qk_norm* norm, const fp4_heads* q, const fp4_heads* k,
                                       const int64_t* positions, int64_t tokens, int64_t head_dim,
                                       const fp4_heads* q_out, const fp4_heads* k_out, void* stream) {
  fp4_status st = check_tokens("tokens", tokens);
  if (!st) st = check_head_dim(head_dim);
  if (!st) st = check_norm(norm, positions, tokens, head_dim);
  if (!st) st = check_pair("q", q, "q_out", q_out, tokens, head_dim);
  if (!st) st = check_pair("k", k, "k_out", k_out, tokens, head_dim);
  if (st) return st;
  if (!q && !k) return fail(FP4_ERR_ARG, "q and k are null");
  if (tokens == 0) return ok();
  fp4lib::QkRowsArgs a{};
  a.in[0] = heads_args(q);
  a.in[1] = heads_args(k);
  a.out[0] = heads_args(q_out);
  a.out[1] = heads_args(k_out);
  a.norm = norm_args(norm, positions);
  a.tokens = tokens;
  a.head_dim = static_cast<int>(head_dim);
  return device_status(fp4lib::launch_qk_rows(a, static_cast<hipStream_t>(stream)), "fp4_qk_norm_rope launch");
}

FP4_EXPORT int64_t fp4_qk_norm_workspace(int64_t head_dim) {
  return head_dim_ok(head_dim) ? fp4lib::qk_grad_workspace(static_cast<int>(head_dim)) : 0;
}

FP4_EXPORT fp4_status fp4_qk_norm_rope_backward(const fp4_qk_norm* norm, const fp4_heads* q, const fp4_heads* k,
                                                const int64_t* positions, int64_t tokens, int64_t head_dim,
                                                const fp4_heads* dq, const fp4_heads* dk,
                                                const fp4_heads* dq_in, const fp4_heads* dk_in,
                                                float* dq_weight, float* dk_weight, int accumulate,
                                                void* workspace, int64_t workspace_bytes, void* stream) {
  fp4_status st = check_tokens("tokens", tokens);
  if (!st) st = check_head_dim(head_dim);
  if (!st) st = check_norm(norm, positions, tokens, head_dim);
  if (!st) st = check_pair("q", q, "dq_in", dq_in, tokens, head_dim);
  if (!st) st = check_pair("k", k, "dk_in", dk_in, tokens, head_dim);
  if (st) return st;
  if (!q && !k) return fail(FP4_ERR_ARG, "q and k are null");
  const fp4_heads *x[2] = {q, k}, *dy[2] = {dq, dk};
  for (int i = 0; i < 2; ++i) {
    if (!x[i]) continue;
    st = check_heads(i ? "dk" : "dq", dy[i], tokens, head_dim, false);
    if (st) return st;
    if (dy[i]->heads != x[i]->heads)
      return fail(FP4_ERR_SHAPE, "%s has %lld heads, its input %lld", i ? "dk" : "dq", (long long)dy[i]->heads,
                  (long long)x[i]->heads);
  }
  const bool sums = dq_weight || dk_weight;
  if (sums && !norm->q_weight) return fail(FP4_ERR_ARG, "a weight's gradient is asked for without a norm");
  if (!aligned(dq_weight, 4) || !aligned(dk_weight, 4))
    return fail(FP4_ERR_ARG, "weight gradients must be aligned to their elements");
  if (sums && (!workspace || !aligned16(workspace)))
    return fail(FP4_ERR_ARG, "the workspace must be non-null and 16-byte aligned");
  if (sums && workspace_bytes < fp4lib::qk_grad_workspace(static_cast<int>(head_dim)))
    return fail(FP4_ERR_ARG, "workspace_bytes=%lld: fp4_qk_norm_workspace bytes are needed",
                (long long)workspace_bytes);
  if (tokens == 0 && !sums) return ok();
  fp4lib::QkGradArgs a{};
  for (int i = 0; i < 2; ++i) {
    a.x[i] = heads_args(x[i]);
    a.dy[i] = heads_args(x[i] ? dy[i] : nullptr);
  }
  a.dx[0] = heads_args(dq_in);
  a.dx[1] = heads_args(dk_in);
  a.norm = norm_args(norm, positions);
  a.dw[0] = dq_weight;
  a.dw[1] = dk_weight;
  a.accumulate = accumulate != 0;
  a.part = sums ? static_cast<float*>(workspace) : nullptr;
  a.tokens = tokens;
  a.head_dim = static_cast<int>(head_dim);
  return device_status(fp4lib::launch_qk_grad(a, static_cast<hipStream_t>(stream)),
                       "fp4_qk_norm_rope_backward launch");
}

FP4_EXPORT fp4_status fp4_kv_cache_write(const fp4_kv_cache* cache, const fp4_heads* k, const fp4_heads* v,
                                         const int64_t* slots, int64_t tokens, const fp4_qk_norm* norm,
                                         const int64_t* positions, const fp4_heads* q, const fp4_heads* q_out,
                                         void* stream) {
  fp4_status st = check_tokens("tokens", tokens);
  if (!st) st = check_cache(cache);
  if (st) return st;
  const int64_t d = cache->head_dim;
  st = check_heads("k", k, tokens, d, false);
  if (!st) st = check_heads("v", v, tokens, d, false);
  if (st) return st;
  if (k->heads != cache->heads || v->heads != cache->heads)
    return fail(FP4_ERR_SHAPE, "k has %lld heads and v %lld, the cache %d", (long long)k->heads,
                (long long)v->heads, cache->heads);
  if (tokens > 0 && !slots) return fail(FP4_ERR_ARG, "slots is null");
  if (!aligned(slots, 8)) return fail(FP4_ERR_ARG, "slots must be aligned to their elements");
  if (norm) {
    st = check_norm(norm, positions, tokens, d);
    if (!st) st = check_pair("q", q, "q_out", q_out, tokens, d);
    if (st) return st;
  } else if (q || q_out) {
    return fail(FP4_ERR_ARG, "q needs a norm");
  }
  if (tokens == 0) return ok();
  fp4lib::QkRowsArgs a{};
  a.in[0] = heads_args(q);
  a.in[1] = heads_args(k);
  a.in[2] = heads_args(v);
  a.out[0] = heads_args(q_out);
  a.norm = norm_args(norm, positions);
  a.cache = cache_args(cache);
  a.cached = 1;
  a.slots = slots;
  a.tokens = tokens;
  a.head_dim = static_cast<int>(d);
  return device_status(fp4lib::launch_qk_rows(a, static_cast<hipStream_t>(stream)), "fp4_kv_cache_write launch");
}

FP4_EXPORT fp4_status fp4_kv_cache_read(const fp4_kv_cache* cache, const int64_t* slots, int64_t n, void* k,
                                        void* v, int out_fp32, void* stream) {
  fp4_status st = check_tokens("n", n);
  if (!st) st = check_cache(cache);
  if (st) return st;
  if (n == 0) return ok();
  if (!slots) return fail(FP4_ERR_ARG, "slots is null");
  if (!aligned(slots, 8)) return fail(FP4_ERR_ARG, "slots must be aligned to their elements");
  if (!k && !v) return fail(FP4_ERR_ARG, "k and v are null");
  if (!aligned16(k) || !aligned16(v)) return fail(FP4_ERR_ARG, "outputs must be 16-byte aligned");
  fp4lib::KvReadArgs a{};
  a.cache = cache_args(cache);
  a.slots = slots;
  a.n = n;
  a.out[0] = k;
  a.out[1] = v;
  a.out_f32 = out_fp32;
  return device_status(fp4lib::launch_kv_read(a, static_cast<hipStream_t>(stream)), "fp4_kv_cache_read launch");
}

namespace {

fp4_status check_attention(const fp4_kv_cache* cache, int64_t q_heads, int64_t requests, int64_t width) {
  fp4_status st = check_tokens("requests", requests);
  if (!st) st = check_cache(cache);
  if (st) return st;
  if (q_heads < 1 || q_heads > kMaxHeads || q_heads % cache->heads)
    return fail(FP4_ERR_SHAPE, "%lld query heads: a multiple of the cache's %d, up to %lld, is needed",
                (long long)q_heads, cache->heads, (long long)kMaxHeads);
  if (width < 0 || width > kMaxTokens || width * cache->page_size >= kMaxTokens / 2)
    return fail(FP4_ERR_SHAPE, "table_width=%lld: contexts are shorter than 2^30", (long long)width);
  // rows of the output, which the kernel that joins parts has a workgroup each for
  if (requests * q_heads >= kMaxTokens)
    return fail(FP4_ERR_SHAPE, "requests * heads must be below 2^31");
  return FP4_OK;
}

fp4lib::AttnArgs attention_args(const fp4_kv_cache* cache, int64_t q_heads, int64_t requests, int64_t width) {
  fp4lib::AttnArgs a{};
  a.cache = cache_args(cache);
  a.q.heads = static_cast<int>(q_heads);
  a.table_width = static_cast<int>(width);
  a.requests = static_cast<int>(requests);
  return a;
}

}  // namespace

FP4_EXPORT int64_t fp4_attention_workspace(const fp4_kv_cache* cache, int64_t q_heads, int64_t requests,
                                           int64_t table_width) {
  if (check_attention(cache, q_heads, requests, table_width) || requests == 0) return 0;
  return fp4lib::attention_workspace(attention_args(cache, q_heads, requests, table_width));
}

FP4_EXPORT fp4_status fp4_attention_decode(const fp4_kv_cache* cache, const fp4_heads* q, const int32_t* page_table,
                                           int64_t table_stride, int64_t table_width, const int32_t* lens,
                                           int64_t requests, float scale, void* out, fp4_out_type out_type,
                                           float* lse, void* workspace, int64_t workspace_bytes, void* stream) {
  if (!q) return fail(FP4_ERR_ARG, "q is null");
  fp4_status st = check_attention(cache, q->heads, requests, table_width);
  if (!st) st = check_heads("q", q, requests, cache->head_dim, false);
  if (st) return st;
  if (out_type != FP4_OUT_F32 && out_type != FP4_OUT_BF16) return fail(FP4_ERR_ARG, "bad out_type %d", (int)out_type);
  if (!std::isfinite(scale)) return fail(FP4_ERR_ARG, "scale must be finite");
  if (table_stride < 0) return fail(FP4_ERR_ARG, "table_stride=%lld is negative", (long long)table_stride);
  if (requests == 0) return ok();
  if (table_width > 0 && !page_table) return fail(FP4_ERR_ARG, "page_table is null");
  if (!lens) return fail(FP4_ERR_ARG, "lens is null");
  if (!aligned(page_table, 4) || !aligned(lens, 4) || !aligned(lse, 4))
    return fail(FP4_ERR_ARG, "page_table, lens and lse must be aligned to their elements");
  if (!out || !aligned16(out)) return fail(FP4_ERR_ARG, "out must be non-null and 16-byte aligned");
  if (workspace_bytes < 0 || (workspace && !aligned16(workspace)))
    return fail(FP4_ERR_ARG, "the workspace must be 16-byte aligned and its size not negative");
  fp4lib::AttnArgs a = attention_args(cache, q->heads, requests, table_width);
  a.q = heads_args(q);
  a.table = page_table;
  a.table_stride = table_stride;
  a.lens = lens;
  a.scale = scale;
  a.out = out;
  a.out_f32 = out_type == FP4_OUT_F32;
  a.lse = lse;
  a.part = static_cast<float*>(workspace);
  a.part_bytes = workspace ? workspace_bytes : 0;
  return device_status(fp4lib::launch_attention(a, static_cast<hipStream_t>(stream)),
                       "fp4_attention_decode launch");
}

FP4_EXPORT fp4_status fp4_selftest_set_attention_splits(int splits) {
  if (splits < 0 || splits > 512) return fail(FP4_ERR_ARG, "splits=%d must be 0 .. 512", splits);
  fp4lib::set_attention_splits(splits);
  return ok();
}
