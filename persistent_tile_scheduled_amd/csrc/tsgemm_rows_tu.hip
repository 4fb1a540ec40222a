// The row operators' kernels and the rules that choose among them.
#include "tsgemm_rows_kernel.h"
#include "tsgemm_ops_launch.h"

namespace tsg {

namespace {

constexpr uint32_t kCus = 256;  // MI355X

// Which kernel a row of `width` values takes.  Up to 512 * kWaveChunks values a
// row belongs to a part of a wave (or a whole one): its sums need no barrier.
// Wider rows take a workgroup with two chunks per thread (the gradient, which
// also holds its columns' sums, one while it can), or (forward only) four;
// still wider ones are read in several rounds.
enum RowClass { ROW_WAVE1, ROW_WAVE2, ROW_BLOCK1, ROW_BLOCK2, ROW_BLOCK4, ROW_WIDE };

struct RowShape {
    RowClass cls;
    uint32_t threads;  // of a workgroup
    uint32_t lpr;      // lanes per row of the wave classes
};

RowShape row_shape(uint32_t width, bool grad) {
    const uint32_t chunks = (width + 7u) / 8u;
    if (chunks <= 64u) {
        uint32_t lpr = 4;
        while (lpr < chunks) lpr *= 2;
        return {ROW_WAVE1, 256, lpr};
    }
    if (chunks <= 128u) return {ROW_WAVE2, 256, 64};
    if (grad && chunks <= 1024u) return {ROW_BLOCK1, (chunks + 63u) / 64u * 64u, 64};
    if (chunks <= 2048u) return {ROW_BLOCK2, (chunks + 127u) / 128u * 64u, 64};
    if (chunks <= 4096u && !grad) return {ROW_BLOCK4, 1024, 64};
    return {ROW_WIDE, 1024, 64};
}

uint32_t at_most(int64_t n, uint32_t most) { return n < (int64_t)most ? (uint32_t)n : most; }

// Workgroups that stay: as many as find room on the chip at once.
uint32_t row_groups(const RowShape& r, int64_t rows) {
    const int64_t per = r.cls <= ROW_WAVE2 ? 256 / r.lpr : 1;
    return at_most((rows + per - 1) / per, kCus * (2048u / r.threads));
}

template <int DT, bool CODES>
void layer_norm_of(const LnArgs& a, const RowShape& r, hipStream_t s) {
    const dim3 grid(row_groups(r, a.rows)), block(r.threads);
    switch (r.cls) {
        case ROW_WAVE1: hipLaunchKernelGGL((layer_norm_kernel<DT, 1, CODES, true>), grid, block, 0, s, a); break;
        case ROW_WAVE2: hipLaunchKernelGGL((layer_norm_kernel<DT, 2, CODES, true>), grid, block, 0, s, a); break;
        case ROW_BLOCK2: hipLaunchKernelGGL((layer_norm_kernel<DT, 2, CODES, false>), grid, block, 0, s, a); break;
        case ROW_BLOCK4: hipLaunchKernelGGL((layer_norm_kernel<DT, 4, CODES, false>), grid, block, 0, s, a); break;
        default: hipLaunchKernelGGL((layer_norm_wide_kernel<DT, CODES>), grid, block, 0, s, a); break;
    }
}

template <int DT>
void layer_norm_grad_of(const LnGradArgs& a, const RowShape& r, hipStream_t s) {
    const dim3 grid(layer_norm_grad_groups(a.rows, a.width)), block(r.threads);
    switch (r.cls) {
        case ROW_WAVE1: hipLaunchKernelGGL((layer_norm_grad_kernel<DT, 1, true>), grid, block, 0, s, a); break;
        case ROW_WAVE2: hipLaunchKernelGGL((layer_norm_grad_kernel<DT, 2, true>), grid, block, 0, s, a); break;
        case ROW_BLOCK1: hipLaunchKernelGGL((layer_norm_grad_kernel<DT, 1, false>), grid, block, 0, s, a); break;
        case ROW_BLOCK2: hipLaunchKernelGGL((layer_norm_grad_kernel<DT, 2, false>), grid, block, 0, s, a); break;
        default: hipLaunchKernelGGL((layer_norm_grad_wide_kernel<DT>), grid, block, 0, s, a); break;
    }
}

uint32_t chunk_groups(int64_t rows, uint32_t width) { return at_most((rows * (width / 8u) + 255) / 256, kCus * 32u); }

}  // namespace

void launch_layer_norm(int dt, const LnArgs& args, hipStream_t s) {
    LnArgs a = args;
    const RowShape r = row_shape(a.width, false);
    a.lpr = r.lpr;
    const bool codes = a.codes != nullptr;
    if (dt == DT_FP16) codes ? layer_norm_of<DT_FP16, true>(a, r, s) : layer_norm_of<DT_FP16, false>(a, r, s);
    else if (dt == DT_BF16) codes ? layer_norm_of<DT_BF16, true>(a, r, s) : layer_norm_of<DT_BF16, false>(a, r, s);
    else codes ? layer_norm_of<DT_FP32, true>(a, r, s) : layer_norm_of<DT_FP32, false>(a, r, s);
}

uint32_t layer_norm_grad_groups(int64_t rows, uint32_t width) {
    const RowShape r = row_shape(width, true);
    const int64_t per = r.cls <= ROW_WAVE2 ? 256 / r.lpr : 1;
    return at_most((rows + per - 1) / per, kCus * (r.threads > 512u ? 1u : 2u));
}

void launch_layer_norm_grad(int dt, const LnGradArgs& args, hipStream_t s) {
    LnGradArgs a = args;
    const RowShape r = row_shape(a.width, true);
    a.lpr = r.lpr;
    if (dt == DT_FP16) layer_norm_grad_of<DT_FP16>(a, r, s);
    else if (dt == DT_BF16) layer_norm_grad_of<DT_BF16>(a, r, s);
    else layer_norm_grad_of<DT_FP32>(a, r, s);
}

void launch_layer_norm_grad_sum(int wdt, const float* part, uint32_t groups, uint32_t pitch, uint32_t width, void* dgamma,
                                void* dbeta, hipStream_t s) {
    const dim3 grid((width + 63u) / 64u), block(1024);
    if (wdt == DT_FP16)
        hipLaunchKernelGGL((layer_norm_grad_sum_kernel<DT_FP16>), grid, block, 0, s, part, groups, pitch, width, dgamma, dbeta);
    else if (wdt == DT_BF16)
        hipLaunchKernelGGL((layer_norm_grad_sum_kernel<DT_BF16>), grid, block, 0, s, part, groups, pitch, width, dgamma, dbeta);
    else
        hipLaunchKernelGGL((layer_norm_grad_sum_kernel<DT_FP32>), grid, block, 0, s, part, groups, pitch, width, dgamma, dbeta);
}

void launch_mx_quantize(int dt, const void* x, int64_t ld, int64_t rows, uint32_t width, uint8_t* codes, uint8_t* scales,
                        hipStream_t s) {
    const uint64_t chunks = (uint64_t)rows * (width / 8u);
    const dim3 grid(chunk_groups(rows, width)), block(256);
    if (dt == DT_FP16)
        hipLaunchKernelGGL((mx_quantize_kernel<DT_FP16>), grid, block, 0, s, x, ld, chunks, width, codes, scales);
    else if (dt == DT_BF16)
        hipLaunchKernelGGL((mx_quantize_kernel<DT_BF16>), grid, block, 0, s, x, ld, chunks, width, codes, scales);
    else
        hipLaunchKernelGGL((mx_quantize_kernel<DT_FP32>), grid, block, 0, s, x, ld, chunks, width, codes, scales);
}

void launch_mx_dequantize(int dt, const uint8_t* codes, const uint8_t* scales, int64_t rows, uint32_t width, void* out,
                          int64_t ld, hipStream_t s) {
    const uint64_t chunks = (uint64_t)rows * (width / 8u);
    const dim3 grid(chunk_groups(rows, width)), block(256);
    if (dt == DT_FP16)
        hipLaunchKernelGGL((mx_dequantize_kernel<DT_FP16>), grid, block, 0, s, codes, scales, chunks, width, out, ld);
    else if (dt == DT_BF16)
        hipLaunchKernelGGL((mx_dequantize_kernel<DT_BF16>), grid, block, 0, s, codes, scales, chunks, width, out, ld);
    else
        hipLaunchKernelGGL((mx_dequantize_kernel<DT_FP32>), grid, block, 0, s, codes, scales, chunks, width, out, ld);
}

}  // namespace tsg
