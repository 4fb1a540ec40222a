// Host-side launch interface of the row operators and of the weight gradient
// (tsgemm_rows_tu.hip, tsgemm_wgrad_tu.hip) for the C ABI (tsgemm_ops.hip).
// dt, wdt and odt are TSGEMM_FP16, TSGEMM_BF16 or TSGEMM_FP32.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace tsg {

struct LnArgs;
struct LnGradArgs;
struct WgradArgs;

void launch_layer_norm(int dt, const LnArgs& a, hipStream_t s);

// Workgroups of a layer norm gradient: the count of partial sums per column.
uint32_t layer_norm_grad_groups(int dt, int64_t rows, uint32_t width);
bool layer_norm_grad_small(int64_t rows, uint32_t width);  // then no partial sums are left
void launch_layer_norm_grad(int dt, const LnGradArgs& a, hipStream_t s);
void launch_layer_norm_grad_sum(int wdt, const float* part, uint32_t groups, uint32_t pitch, uint32_t width, void* dgamma,
                                void* dbeta, hipStream_t s);

void launch_mx_quantize(int dt, const void* x, int64_t ld, int64_t rows, uint32_t width, uint8_t* codes, uint8_t* scales,
                        hipStream_t s);
void launch_mx_dequantize(int dt, const uint8_t* codes, const uint8_t* scales, int64_t rows, uint32_t width, void* out,
                          int64_t ld, hipStream_t s);

// Bytes of fp32 partial products that a weight gradient of this shape needs (0: none).
int64_t wgrad_workspace(int64_t rows, int64_t out, int64_t width);
void launch_wgrad(int dt, int odt, const WgradArgs& a, hipStream_t s);

}  // namespace tsg
