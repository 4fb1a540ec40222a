// Host-side launch interface of the gated projection and of the linear head's cross
// entropy (tsgemm_linear_tu.hip, one unit per type) for the C ABI (tsgemm_linear.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace tsg {

struct LinArgs;
struct GatedGradArgs;
struct LossArgs;
struct LossGradArgs;
struct LinSumArgs;

enum LinKind { LIN_KIND_GATED, LIN_KIND_LSE, LIN_KIND_DLOGITS, LIN_KIND_DX, LIN_KIND_DW };

// The kernels of one 16-bit type.
template <int DT>
struct LinearOf {
    static void product(LinKind kind, int tile, const LinArgs& a, hipStream_t s);
    static void few(LinKind kind, const LinArgs& a, hipStream_t s);  // LIN_KIND_GATED, LIN_KIND_LSE where takes_few
    static void sum(const LinSumArgs& a, hipStream_t s);
    static void gated_slope(const GatedGradArgs& a, hipStream_t s);
    static void loss_rows(const LossGradArgs& a, hipStream_t s);
};
void launch_loss_join(const LossArgs& a, hipStream_t s);
void launch_linear_zero(uint16_t* out, int64_t ld, int64_t rows, uint32_t width, hipStream_t s);

}  // namespace tsg
