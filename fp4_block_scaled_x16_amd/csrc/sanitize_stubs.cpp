// Host-only stand-ins for the kernel launchers, linked with fp4_api.cpp, fp8_api.cpp and kv_api.cpp
// into the AddressSanitizer / UndefinedBehaviorSanitizer build of the C ABI's
// validation code (build.py build_sanitized).  That build runs the
// argument-checking tests, which never reach a device: any call that passes
// validation reports "no device" here instead of launching.
#include <hip/hip_runtime.h>

#include "fp4_internal.hpp"
#include "kv_internal.hpp"

namespace fp4lib {

int device_cu_count() { return 256; }
int64_t grid_cap(int per_cu) { return 256 * static_cast<int64_t>(per_cu); }
int gemm_tile_rows_forced() { return 0; }
void set_launch_geometry(int, int) {}

hipError_t launch_amax(const uint16_t*, int64_t, int64_t, int64_t, int, int, const uint32_t (&)[4],
                       float*, hipStream_t, float*, bool) {
  return hipErrorNoDevice;
}
hipError_t launch_quant_row(const QuantArgs&, hipStream_t) { return hipErrorNoDevice; }
hipError_t launch_quant_row_scoped(const QuantArgs&, hipStream_t) { return hipErrorNoDevice; }
hipError_t launch_quant_col(const QuantArgs&, hipStream_t) { return hipErrorNoDevice; }
hipError_t launch_quant_2d(const QuantArgs&, hipStream_t) { return hipErrorNoDevice; }
hipError_t launch_quant_mx8(const QuantArgs&, bool, hipStream_t) { return hipErrorNoDevice; }
hipError_t launch_dequant_mx8(int, const uint8_t*, const uint8_t*, int64_t, int64_t, void*, int,
                              hipStream_t) {
  return hipErrorNoDevice;
}
hipError_t launch_quant_dual(const QuantArgs&, const QuantArgs&, hipStream_t) {
  return hipErrorNoDevice;
}
hipError_t launch_dequant(int, int, int, const uint8_t*, const uint8_t*, const float*, bool, int64_t,
                          int64_t, void*, int, hipStream_t) {
  return hipErrorNoDevice;
}
hipError_t launch_rht(const uint16_t*, int64_t, int64_t, int64_t, int, const uint32_t (&)[4], bool,
                      float*, hipStream_t) {
  return hipErrorNoDevice;
}
hipError_t launch_gemm(int, const GemmOperand&, const GemmOperand&, int64_t, int64_t, int64_t, void*,
                       int, int64_t, int, hipStream_t) {
  return hipErrorNoDevice;
}
hipError_t launch_quant_fp8(const Fp8QuantArgs&, hipStream_t) { return hipErrorNoDevice; }
hipError_t launch_dequant_fp8(int, const uint8_t*, const uint8_t*, int64_t, int64_t, void*, int,
                              hipStream_t) {
  return hipErrorNoDevice;
}
hipError_t launch_requant_t_fp8(int, const uint8_t*, const uint8_t*, int64_t, int64_t, uint8_t*,
                                uint8_t*, hipStream_t) {
  return hipErrorNoDevice;
}
hipError_t launch_act_quant_fp8(const Fp8ActArgs&, hipStream_t) { return hipErrorNoDevice; }
hipError_t launch_act_grad_fp8(const Fp8ActGradArgs&, hipStream_t) { return hipErrorNoDevice; }
hipError_t launch_gemm_fp8(const Fp8GemmArgs&, hipStream_t) { return hipErrorNoDevice; }
int64_t gemm_fp8_workspace(const Fp8GemmArgs&) { return 0; }
void set_fp8_plan(int, int) {}
hipError_t launch_selftest_sweep(int, const uint32_t*, int, uint64_t*, hipStream_t) {
  return hipErrorNoDevice;
}
hipError_t launch_selftest_gemm_decode(int, uint16_t*, hipStream_t) { return hipErrorNoDevice; }
hipError_t launch_qk_rows(const QkRowsArgs&, hipStream_t) { return hipErrorNoDevice; }
hipError_t launch_qk_grad(const QkGradArgs&, hipStream_t) { return hipErrorNoDevice; }
int64_t qk_grad_workspace(int head_dim) { return 4096 * static_cast<int64_t>(head_dim); }
hipError_t launch_kv_read(const KvReadArgs&, hipStream_t) { return hipErrorNoDevice; }
hipError_t launch_attention(const AttnArgs&, hipStream_t) { return hipErrorNoDevice; }
int64_t attention_workspace(const AttnArgs&) { return 0; }
void set_attention_splits(int) {}

}  // namespace fp4lib
