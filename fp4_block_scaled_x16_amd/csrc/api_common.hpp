// Shared by the C ABI's translation units (fp4_api.cpp, fp8_api.cpp): how a
// call fails, and the FP8 halves of the entry points that take every format.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/fp4.h"

#define FP4_EXPORT extern "C" __attribute__((visibility("default")))

namespace fp4api {

// Record the detail that fp4_last_error returns and pass the status on.
fp4_status fail(fp4_status st, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
fp4_status ok();

inline fp4_status device_status(hipError_t e, const char* what) {
  if (e != hipSuccess) return fail(FP4_ERR_DEVICE, "%s: %s", what, hipGetErrorString(e));
  return ok();
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline bool is_fp8(int f) { return f == FP4_FP8_E4M3 || f == FP4_FP8_E5M2; }

// fp8_api.cpp: the entry points' calls with an FP8 format, checks included.
fp4_status quantize_fp8(const fp4_quant_desc* d, const uint16_t* x, int64_t rows, int64_t cols,
                        int64_t ld, uint8_t* codes, uint8_t* scales, uint8_t* codes_t,
                        fp4_counters* counters, void* stream);
fp4_status quantize_dual_fp8(const fp4_quant_desc* rd, const fp4_quant_desc* cd, const uint16_t* x,
                             int64_t rows, int64_t cols, int64_t ld, uint8_t* codes,
                             uint8_t* scales, uint8_t* codes_t, uint8_t* scales_t,
                             fp4_counters* counters, void* stream);
fp4_status dequantize_fp8(fp4_format format, fp4_block block, fp4_scale_layout layout,
                          const uint8_t* codes, const uint8_t* scales, fp4_global_scope scope,
                          int64_t rows, int64_t cols, void* out, int out_fp32, void* stream);
fp4_status gemm_fp8(const fp4_operand* A, const fp4_operand* B, int64_t M, int64_t N, int64_t K,
                    void* D, fp4_out_type d_type, int64_t ldd, int accumulate, void* workspace,
                    int64_t workspace_bytes, void* stream);

}  // namespace fp4api
