// The C ABI's FP8 (block-128) calls (include/fp4.h): the FP8 halves of the
// entry points shared with the FP4 formats, and the entry points of the 8-bit
// checkpoints.  Host-side argument checks, then launches; no check touches a
// HIP API, so rejected calls work without a GPU.
#include "api_common.hpp"
#include "fp4_internal.hpp"

using namespace fp4api;

namespace {

constexpr int64_t kMaxDim = int64_t(1) << 31;

fp4_status check_size(int64_t rows, int64_t cols) {
  if (rows < 0 || cols < 0)
    return fail(FP4_ERR_SHAPE, "negative size rows=%lld cols=%lld", (long long)rows, (long long)cols);
  if (rows >= kMaxDim || cols >= kMaxDim)
    return fail(FP4_ERR_SHAPE, "rows=%lld and cols=%lld must be below 2^31", (long long)rows,
                (long long)cols);
  return FP4_OK;
}

// A bf16 matrix in the library's manner: 16-byte aligned, ld a multiple of 8.
fp4_status check_bf16(const char* name, const uint16_t* x, int64_t cols, int64_t ld) {
  if (!x) return fail(FP4_ERR_ARG, "%s is null", name);
  if (!aligned16(x)) return fail(FP4_ERR_ARG, "%s must be 16-byte aligned", name);
  if (ld < cols) return fail(FP4_ERR_ARG, "%s: ld=%lld < cols=%lld", name, (long long)ld, (long long)cols);
  if (ld % 8) return fail(FP4_ERR_ARG, "%s: ld=%lld must be a multiple of 8", name, (long long)ld);
  return FP4_OK;
}

fp4_status check_codes(const char* name, const void* codes, const void* scales) {
  if (!codes || !scales) return fail(FP4_ERR_ARG, "%s: codes/scales are null", name);
  if (!aligned16(codes) || !aligned16(scales))
    return fail(FP4_ERR_ARG, "%s: codes and scales must be 16-byte aligned", name);
  return FP4_OK;
}

// A pair of outputs that may be left out: both null or both there.
fp4_status check_codes_opt(const char* name, const void* codes, const void* scales) {
  if (!codes && !scales) return FP4_OK;
  return check_codes(name, codes, scales);
}

fp4_status check_desc(const fp4_quant_desc* d, const char* side) {
  if (!is_fp8(d->format)) return fail(FP4_ERR_UNSUPPORTED, "%s: the two formats differ", side);
  if (d->block == FP4_BLOCK_2D16)
    return fail(FP4_ERR_UNSUPPORTED, "%s: 2D16 blocks need NVFP4 or UE5M3 (FP8: 2D128)", side);
  if (d->block != FP4_BLOCK_1D && d->block != FP4_BLOCK_2D128)
    return fail(FP4_ERR_ARG, "%s: bad block %d", side, (int)d->block);
  if (d->orient != FP4_ROWWISE && d->orient != FP4_COLWISE)
    return fail(FP4_ERR_ARG, "%s: bad orient %d", side, (int)d->orient);
  if (d->round != FP4_RNE && d->round != FP4_SR)
    return fail(FP4_ERR_ARG, "%s: bad round %d", side, (int)d->round);
  if (d->round != FP4_RNE) return fail(FP4_ERR_UNSUPPORTED, "%s: FP8 rounds to nearest even", side);
  if (d->scale_layout != FP4_SCALES_KMAJOR)
    return fail(FP4_ERR_UNSUPPORTED, "%s: FP8 scales are KMAJOR (scale_layout %d)", side,
                (int)d->scale_layout);
  if (d->rht) return fail(FP4_ERR_UNSUPPORTED, "%s: RHT needs NVFP4 or UE5M3", side);
  if (d->amax_given) return fail(FP4_ERR_UNSUPPORTED, "%s: FP8 has no tensor amax", side);
  if (d->emit_transpose)
    return fail(FP4_ERR_UNSUPPORTED, "%s: emit_transpose needs 2D16 (FP8: fp4_quantize_dual)", side);
  if (d->scale_round != FP4_SCALE_RNE && d->scale_round != FP4_SCALE_UP)
    return fail(FP4_ERR_ARG, "%s: bad scale_round %d", side, (int)d->scale_round);
  if (d->global_scope != FP4_GLOBAL_TENSOR && d->global_scope != FP4_GLOBAL_ROW)
    return fail(FP4_ERR_ARG, "%s: bad global_scope %d", side, (int)d->global_scope);
  if (d->global_scope != FP4_GLOBAL_TENSOR)
    return fail(FP4_ERR_UNSUPPORTED, "%s: FP8 has no global scale", side);
  if (d->count_level != FP4_COUNT_ALL && d->count_level != FP4_COUNT_SCALES)
    return fail(FP4_ERR_ARG, "%s: bad count_level %d", side, (int)d->count_level);
  return FP4_OK;
}

}  // namespace

namespace fp4api {

fp4_status quantize_fp8(const fp4_quant_desc* d, const uint16_t* x, int64_t rows, int64_t cols,
                        int64_t ld, uint8_t* codes, uint8_t* scales, uint8_t* codes_t,
                        fp4_counters* counters, void* stream) {
  fp4_status st = check_desc(d, "desc");
  if (!st) st = check_size(rows, cols);
  if (st) return st;
  if (codes_t) return fail(FP4_ERR_UNSUPPORTED, "FP8 codes_t: use fp4_quantize_dual");
  if (rows == 0 || cols == 0) return ok();
  st = check_bf16("x", x, cols, ld);
  if (!st) st = check_codes("output", codes, scales);
  if (st) return st;
  fp4lib::Fp8QuantArgs a{};
  a.x = x;
  a.rows = rows;
  a.cols = cols;
  a.ld = ld;
  a.e5m2 = d->format == FP4_FP8_E5M2;
  a.block2d = d->block == FP4_BLOCK_2D128;
  (d->orient == FP4_COLWISE ? a.codes_t : a.codes) = codes;
  (d->orient == FP4_COLWISE ? a.scales_t : a.scales) = scales;
  a.counters = d->count_level == FP4_COUNT_ALL ? counters : nullptr;
  return device_status(fp4lib::launch_quant_fp8(a, static_cast<hipStream_t>(stream)),
                       "fp4_quantize launch");
}

fp4_status quantize_dual_fp8(const fp4_quant_desc* rd, const fp4_quant_desc* cd, const uint16_t* x,
                             int64_t rows, int64_t cols, int64_t ld, uint8_t* codes,
                             uint8_t* scales, uint8_t* codes_t, uint8_t* scales_t,
                             fp4_counters* counters, void* stream) {
  fp4_status st = check_desc(rd, "rowwise");
  if (!st) st = check_desc(cd, "colwise");
  if (st) return st;
  if (rd->format != cd->format) return fail(FP4_ERR_UNSUPPORTED, "the two formats differ");
  if (rd->block != cd->block) return fail(FP4_ERR_UNSUPPORTED, "the two blocks differ");
  if (rd->count_level != cd->count_level)
    return fail(FP4_ERR_UNSUPPORTED, "the two descs count different events");
  if (rd->orient != FP4_ROWWISE || cd->orient != FP4_COLWISE)
    return fail(FP4_ERR_UNSUPPORTED, "descs must be ROWWISE then COLWISE");
  st = check_size(rows, cols);
  if (st) return st;
  if (rows == 0 || cols == 0) return ok();
  st = check_bf16("x", x, cols, ld);
  if (!st) st = check_codes("rowwise output", codes, scales);
  if (!st) st = check_codes("colwise output", codes_t, scales_t);
  if (st) return st;
  fp4lib::Fp8QuantArgs a{};
  a.x = x;
  a.rows = rows;
  a.cols = cols;
  a.ld = ld;
  a.e5m2 = rd->format == FP4_FP8_E5M2;
  a.block2d = rd->block == FP4_BLOCK_2D128;
  a.codes = codes;
  a.scales = scales;
  a.codes_t = codes_t;
  a.scales_t = scales_t;
  a.counters = rd->count_level == FP4_COUNT_ALL ? counters : nullptr;
  return device_status(fp4lib::launch_quant_fp8(a, static_cast<hipStream_t>(stream)),
                       "fp4_quantize_dual launch");
}

fp4_status dequantize_fp8(fp4_format format, fp4_block block, fp4_scale_layout layout,
                          const uint8_t* codes, const uint8_t* scales, fp4_global_scope scope,
                          int64_t rows, int64_t cols, void* out, int out_fp32, void* stream) {
  if (block != FP4_BLOCK_1D && block != FP4_BLOCK_2D128)
    return fail(FP4_ERR_UNSUPPORTED, "FP8 blocks are 1D or 2D128 (block %d)", (int)block);
  if (layout != FP4_SCALES_KMAJOR)
    return fail(FP4_ERR_UNSUPPORTED, "FP8 scales are KMAJOR (scale_layout %d)", (int)layout);
  if (scope != FP4_GLOBAL_TENSOR) return fail(FP4_ERR_UNSUPPORTED, "FP8 has no global scale");
  fp4_status st = check_size(rows, cols);
  if (st) return st;
  if (rows == 0 || cols == 0) return ok();
  st = check_codes("input", codes, scales);
  if (st) return st;
  if (!out || !aligned16(out)) return fail(FP4_ERR_ARG, "out must be non-null and 16-byte aligned");
  return device_status(fp4lib::launch_dequant_fp8(format == FP4_FP8_E5M2, codes, scales, rows, cols,
                                                  out, out_fp32, static_cast<hipStream_t>(stream)),
                       "fp4_dequantize launch");
}

namespace {

fp4lib::Fp8GemmArgs gemm_args(const fp4_operand* const (&ops)[2], int64_t M, int64_t N, int64_t nkb,
                              fp4_out_type d_type) {
  fp4lib::Fp8GemmArgs g{};
  for (int i = 0; i < 2; ++i) {
    g.codes[i] = ops[i]->codes;
    g.ld[i] = ops[i]->ld_codes;
    g.scales[i] = ops[i]->scales;
    g.s_kblk[i] = ops[i]->scale_stride_kblk;
  }
  g.M = M;
  g.N = N;
  g.nkb = nkb;
  g.d_bf16 = d_type == FP4_OUT_BF16;
  g.a_e5m2 = ops[0]->format == FP4_FP8_E5M2;
  g.splits = 1;
  return g;
}

}  // namespace

fp4_status gemm_fp8(const fp4_operand* A, const fp4_operand* B, int64_t M, int64_t N, int64_t K,
                    void* D, fp4_out_type d_type, int64_t ldd, int accumulate, void* workspace,
                    int64_t workspace_bytes, void* stream) {
  if (!is_fp8(A->format) || !is_fp8(B->format))
    return fail(FP4_ERR_UNSUPPORTED, "A and B formats differ");
  if (B->format != FP4_FP8_E4M3)
    return fail(FP4_ERR_UNSUPPORTED, "operand B must be FP8_E4M3 (E5M2 gradients are operand A)");
  if (M < 0 || N < 0 || K < 0) return fail(FP4_ERR_SHAPE, "negative size");
  if (M >= kMaxDim || N >= kMaxDim || K >= kMaxDim)
    return fail(FP4_ERR_SHAPE, "M, N and K must be below 2^31");
  if (ldd < N) return fail(FP4_ERR_ARG, "ldd=%lld < N=%lld", (long long)ldd, (long long)N);
  if (d_type != FP4_OUT_F32 && d_type != FP4_OUT_BF16)
    return fail(FP4_ERR_ARG, "bad d_type %d", (int)d_type);
  const int64_t kp = (K + 127) / 128 * 128;
  const fp4_operand* ops[2] = {A, B};
  const int64_t rows[2] = {M, N};
  for (int i = 0; i < 2; ++i) {
    const fp4_operand* o = ops[i];
    if (o->scale_layout != FP4_SCALES_KMAJOR)
      return fail(FP4_ERR_UNSUPPORTED, "operand %c: FP8 scales are KMAJOR", "AB"[i]);
    if (o->scale_row_group != 1)
      return fail(FP4_ERR_UNSUPPORTED, "operand %c: KMAJOR scales need scale_row_group 1", "AB"[i]);
    if (o->s_dec_scope != FP4_GLOBAL_TENSOR)
      return fail(FP4_ERR_UNSUPPORTED, "operand %c: FP8 has no global scale", "AB"[i]);
    if (M > 0 && N > 0 && K > 0) {
      fp4_status st = check_codes(i ? "operand B" : "operand A", o->codes, o->scales);
      if (st) return st;
      if (o->ld_codes < kp || o->ld_codes % 16)
        return fail(FP4_ERR_ARG, "operand %c: ld_codes=%lld must be a multiple of 16 and at least %lld",
                    "AB"[i], (long long)o->ld_codes, (long long)kp);
      if (o->scale_stride_kblk % 16 || o->scale_stride_kblk < rows[i])
        return fail(FP4_ERR_ARG, "operand %c: scale_stride_kblk=%lld must be a multiple of 16 and at "
                    "least the operand's rows", "AB"[i], (long long)o->scale_stride_kblk);
    }
  }
  if (M == 0 || N == 0) return ok();
  if (!D) return fail(FP4_ERR_ARG, "D is null");
  const int es = d_type == FP4_OUT_BF16 ? 2 : 4;
  if (reinterpret_cast<uintptr_t>(D) % es) return fail(FP4_ERR_ARG, "D must be aligned to its elements");
  if (workspace_bytes < 0 || (workspace && !aligned16(workspace)))
    return fail(FP4_ERR_ARG, "the workspace must be 16-byte aligned and its size not negative");
  fp4lib::Fp8GemmArgs g = gemm_args(ops, M, N, kp / 128, d_type);
  g.D = D;
  g.ldd = ldd;
  g.accumulate = accumulate != 0;
  g.part = static_cast<float*>(workspace);
  g.part_bytes = workspace ? workspace_bytes : 0;
  return device_status(fp4lib::launch_gemm_fp8(g, static_cast<hipStream_t>(stream)),
                       "fp4_gemm launch");
}

}  // namespace fp4api

FP4_EXPORT int64_t fp4_gemm_workspace(const fp4_operand* A, const fp4_operand* B, int64_t M, int64_t N,
                                      int64_t K, fp4_out_type d_type) {
  if (!A || !B || !is_fp8(A->format) || !is_fp8(B->format) || M <= 0 || N <= 0 || K <= 0 ||
      M >= kMaxDim || N >= kMaxDim || K >= kMaxDim)
    return 0;
  const fp4_operand* ops[2] = {A, B};
  return fp4lib::gemm_fp8_workspace(gemm_args(ops, M, N, (K + 127) / 128, d_type));
}

FP4_EXPORT fp4_status fp4_requantize_t(fp4_format format, const uint8_t* codes,
                                       const uint8_t* scales, int64_t rows, int64_t cols,
                                       uint8_t* codes_t, uint8_t* scales_t, void* stream) {
  if (!is_fp8(format))
    return fail(FP4_ERR_UNSUPPORTED, "format %d: only FP8 codes are re-encoded", (int)format);
  fp4_status st = check_size(rows, cols);
  if (st) return st;
  if (rows == 0 || cols == 0) return ok();
  st = check_codes("input", codes, scales);
  if (!st) st = check_codes("output", codes_t, scales_t);
  if (st) return st;
  return device_status(fp4lib::launch_requant_t_fp8(format == FP4_FP8_E5M2, codes, scales, rows, cols,
                                                    codes_t, scales_t,
                                                    static_cast<hipStream_t>(stream)),
                       "fp4_requantize_t launch");
}

namespace {

fp4_status check_act(fp4_act act, int64_t rows, int64_t cols) {
  if (act != FP4_ACT_SWIGLU && act != FP4_ACT_RELU2) return fail(FP4_ERR_ARG, "bad act %d", (int)act);
  fp4_status st = check_size(rows, cols);
  if (st) return st;
  if (act == FP4_ACT_SWIGLU && cols % 8)
    return fail(FP4_ERR_SHAPE, "SWIGLU: cols=%lld must be a multiple of 8", (long long)cols);
  if (act == FP4_ACT_SWIGLU && cols >= kMaxDim / 2 - 128)
    return fail(FP4_ERR_SHAPE, "SWIGLU: 2 * cols must be below 2^31");
  return FP4_OK;
}

}  // namespace

FP4_EXPORT fp4_status fp4_act_quantize(fp4_act act, const uint16_t* h, int64_t rows, int64_t cols,
                                       int64_t ld, uint8_t* a_codes, uint8_t* a_scales,
                                       uint16_t* a, int64_t ld_a, uint8_t* h_codes,
                                       uint8_t* h_scales, void* stream) {
  fp4_status st = check_act(act, rows, cols);
  if (st) return st;
  if (rows == 0 || cols == 0) return ok();
  const int64_t width = act == FP4_ACT_SWIGLU ? 2 * cols : cols;
  st = check_bf16("h", h, width, ld);
  if (!st) st = check_codes_opt("a", a_codes, a_scales);
  if (!st) st = check_codes_opt("h", h_codes, h_scales);
  if (!st && a) st = check_bf16("a", a, cols, ld_a);
  if (st) return st;
  if (!a_codes && !a && !h_codes) return fail(FP4_ERR_ARG, "every output is null");
  fp4lib::Fp8ActArgs g{};
  g.act = act;
  g.h = h;
  g.rows = rows;
  g.cols = cols;
  g.ld = ld;
  g.a_codes = a_codes;
  g.a_scales = a_scales;
  g.a = a;
  g.ld_a = ld_a;
  g.h_codes = h_codes;
  g.h_scales = h_scales;
  return device_status(fp4lib::launch_act_quant_fp8(g, static_cast<hipStream_t>(stream)),
                       "fp4_act_quantize launch");
}

FP4_EXPORT fp4_status fp4_act_backward(fp4_act act, const uint8_t* h_codes, const uint8_t* h_scales,
                                       const uint16_t* da, int64_t rows, int64_t cols, int64_t ld,
                                       fp4_format format, uint8_t* dh_codes, uint8_t* dh_scales,
                                       uint8_t* dh_t_codes, uint8_t* dh_t_scales,
                                       uint8_t* a_t_codes, uint8_t* a_t_scales, uint16_t* dh,
                                       int64_t ld_dh, uint16_t* a, int64_t ld_a, void* stream) {
  fp4_status st = check_act(act, rows, cols);
  if (st) return st;
  if (!is_fp8(format)) return fail(FP4_ERR_UNSUPPORTED, "format %d: gradients are FP8", (int)format);
  if (rows == 0 || cols == 0) return ok();
  st = check_codes("checkpoint", h_codes, h_scales);
  if (!st) st = check_bf16("da", da, cols, ld);
  if (!st) st = check_codes_opt("dh", dh_codes, dh_scales);
  if (!st) st = check_codes_opt("dh_t", dh_t_codes, dh_t_scales);
  if (!st) st = check_codes_opt("a_t", a_t_codes, a_t_scales);
  if (!st && dh) st = check_bf16("dh", dh, act == FP4_ACT_SWIGLU ? 2 * cols : cols, ld_dh);
  if (!st && a) st = check_bf16("a", a, cols, ld_a);
  if (st) return st;
  if (!dh_codes && !dh_t_codes && !a_t_codes && !dh && !a)
    return fail(FP4_ERR_ARG, "every output is null");
  fp4lib::Fp8ActGradArgs g{};
  g.act = act;
  g.e5m2 = format == FP4_FP8_E5M2;
  g.h_codes = h_codes;
  g.h_scales = h_scales;
  g.da = da;
  g.rows = rows;
  g.cols = cols;
  g.ld = ld;
  g.dh_codes = dh_codes;
  g.dh_scales = dh_scales;
  g.dh_t_codes = dh_t_codes;
  g.dh_t_scales = dh_t_scales;
  g.a_t_codes = a_t_codes;
  g.a_t_scales = a_t_scales;
  g.dh = dh;
  g.ld_dh = ld_dh;
  g.a = a;
  g.ld_a = ld_a;
  return device_status(fp4lib::launch_act_grad_fp8(g, static_cast<hipStream_t>(stream)),
                       "fp4_act_backward launch");
}
