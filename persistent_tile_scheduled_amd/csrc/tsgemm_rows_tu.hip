// The row operators' kernels and the rules that choose among them.
#include <cmath>

#include "tsgemm_rows_kernel.h"
#include "tsgemm_ops_launch.h"

namespace tsg {

namespace {

constexpr uint32_t kCus = 256;  // MI355X

// Which kernel a row of `width` values takes.  Up to 512 values per wave and
// chunk a row belongs to a part of a wave (or a whole one): its sums need no
// barrier.  Wider rows take a workgroup with two chunks per thread (the
// gradient, which also holds its columns' sums, one while it can); still wider
// ones are read in several rounds.
enum RowClass { ROW_WAVE1, ROW_WAVE2, ROW_BLOCK1, ROW_BLOCK2, ROW_WIDE };

struct RowShape {
    RowClass cls;
    uint32_t threads;  // of a workgroup
    uint32_t lpr;      // lanes per row of the wave classes
    uint32_t rows;     // of a workgroup at a time
};

RowShape row_shape(uint32_t width, bool grad) {
    const uint32_t chunks = (width + 7u) / 8u;
    if (chunks <= 64u) {
        uint32_t lpr = 4;
        while (lpr < chunks) lpr *= 2;
        return {ROW_WAVE1, 256, lpr, 256u / lpr};
    }
    if (chunks <= 128u) return {ROW_WAVE2, 256, 64, 4};
    if (grad && chunks <= 1024u) return {ROW_BLOCK1, (chunks + 63u) / 64u * 64u, 64, 1};
    if (chunks <= 2048u) return {ROW_BLOCK2, (chunks + 127u) / 128u * 64u, 64, 1};
    return {ROW_WIDE, 1024, 64, 1};
}

uint32_t at_most(int64_t n, uint32_t most) { return n < (int64_t)most ? (uint32_t)n : most; }

// Workgroups that stay, per compute unit: as many as hold 32 KiB of rows at a
// time (with as much again on its way), at most what finds room at once.  Fewer
// leave memory idle, more make it jump between more rows: layer norm 8192 x 8192
// bf16 with 1, 2, 4 and 8 workgroups 62, 51, 52 and 55 us, 60000 x 1024 with 2, 4, 8 and
// 16 52, 48, 53 and 51 us.
uint32_t groups_per_cu(const RowShape& r, uint32_t width, int element, uint32_t matrices, uint32_t most) {
    const uint64_t held = (uint64_t)r.rows * width * (uint32_t)element * matrices;
    const uint64_t n = (32768u + held / 2u) / held, room = 2048u / r.threads < most ? 2048u / r.threads : most;
    return n < 1u ? 1u : n < room ? (uint32_t)n : (uint32_t)room;
}

uint32_t row_groups(const RowShape& r, int64_t rows, uint32_t per_cu) {
    return at_most((rows + r.rows - 1) / r.rows, kCus * per_cu);
}

template <int DT, bool CODES>
void layer_norm_of(const LnArgs& a, const RowShape& r, hipStream_t s) {
    const dim3 grid(row_groups(r, a.rows, groups_per_cu(r, a.width, ElemBytes<DT>::v, 1u, 8u))), block(r.threads);
    if (a.width < 8u) {
        if constexpr (!CODES) hipLaunchKernelGGL((layer_norm_kernel<DT, 1, false, true, false>), grid, block, 0, s, a);
        return;
    }
    switch (r.cls) {
        case ROW_WAVE1: hipLaunchKernelGGL((layer_norm_kernel<DT, 1, CODES, true, true>), grid, block, 0, s, a); break;
        case ROW_WAVE2: hipLaunchKernelGGL((layer_norm_kernel<DT, 2, CODES, true, true>), grid, block, 0, s, a); break;
        case ROW_BLOCK2: hipLaunchKernelGGL((layer_norm_kernel<DT, 2, CODES, false, true>), grid, block, 0, s, a); break;
        default: hipLaunchKernelGGL((layer_norm_wide_kernel<DT, CODES>), grid, block, 0, s, a); break;
    }
}

template <int DT>
void layer_norm_to(const LnArgs& a, const RowShape& r, hipStream_t s) {
    a.codes != nullptr ? layer_norm_of<DT, true>(a, r, s) : layer_norm_of<DT, false>(a, r, s);
}

// The gradient reads two matrices, and each workgroup leaves sums of its own:
// at most three workgroups per compute unit (65536 x 256 bf16 with 2, 3 and 4:
// 28.4, 27.5 and 29.7 us).
uint32_t grad_per_cu(const RowShape& r, uint32_t width, int element) { return groups_per_cu(r, width, element, 2u, 3u); }

template <int DT>
void layer_norm_grad_of(const LnGradArgs& a, const RowShape& r, hipStream_t s) {
    const uint32_t per_cu = grad_per_cu(r, a.width, ElemBytes<DT>::v);
    const uint32_t columns = a.dgamma || a.dbeta ? (a.width + 7u) / 8u : 0u;
    const dim3 grid(a.row_groups + columns), block(r.threads);
    if (a.width < 8u) {
        hipLaunchKernelGGL((layer_norm_grad_kernel<DT, 1, true, false, 1>), grid, block, 0, s, a);
        return;
    }
    switch (r.cls) {
        case ROW_WAVE1: hipLaunchKernelGGL((layer_norm_grad_kernel<DT, 1, true, true, 1>), grid, block, 0, s, a); break;
        case ROW_WAVE2: hipLaunchKernelGGL((layer_norm_grad_kernel<DT, 2, true, true, 1>), grid, block, 0, s, a); break;
        case ROW_BLOCK1:
            // a workgroup alone on its compute unit asks for two rows ahead:
            // 8192 x 8192 bf16 87.2 -> 84.0 us; with two or more there is
            // nothing to gain (16000 x 4000 fp16 77.3 -> 79.7)
            if (per_cu == 1u) hipLaunchKernelGGL((layer_norm_grad_kernel<DT, 1, false, true, 2>), grid, block, 0, s, a);
            else hipLaunchKernelGGL((layer_norm_grad_kernel<DT, 1, false, true, 1>), grid, block, 0, s, a);
            break;
        case ROW_BLOCK2: hipLaunchKernelGGL((layer_norm_grad_kernel<DT, 2, false, true, 1>), grid, block, 0, s, a); break;
        default: hipLaunchKernelGGL((layer_norm_grad_wide_kernel<DT>), grid, block, 0, s, a); break;
    }
}

uint32_t chunk_groups(int64_t rows, uint32_t width) { return at_most((rows * (width / 8u) + 255) / 256, kCus * 32u); }

}  // namespace

void launch_layer_norm(int dt, const LnArgs& args, hipStream_t s) {
    LnArgs a = args;
    const RowShape r = row_shape(a.width, false);
    a.lpr = r.lpr;
    if (dt == DT_FP16) layer_norm_to<DT_FP16>(a, r, s);
    else if (dt == DT_BF16) layer_norm_to<DT_BF16>(a, r, s);
    else layer_norm_to<DT_FP32>(a, r, s);
}

// A workgroup more spares the others a row (0.55 us up to 4096 values, then in
// proportion) and costs its sums' way through memory (16 bytes per column at
// 3.2 TB/s) and a step of the sums' loop (0.45 us for 128 workgroups): where
// there are few rows the two meet at the root below.  512 x 4096 bf16 with 1, 3,
// 4 and 8 rows per workgroup: 16.9, 11.1, 11.1 and 12.4 us; 2000 x 512 with 1, 2
// and 4 rounds: 10.3, 8.3 and 9.0; 8 x 16384 with 1 and 2: 9.2 and 11.4.
uint32_t layer_norm_grad_groups(int dt, int64_t rows, uint32_t width) {
    const RowShape r = row_shape(width, true);
    const uint32_t most = row_groups(r, rows, grad_per_cu(r, width, dt == DT_FP32 ? 4 : 2));
    const int64_t all = (rows + r.rows - 1) / r.rows;
    const double sums = 5e-6 * width + 0.0035, row = 0.55 * (width > 4096u ? width / 4096.0 : 1.0);
    const int64_t rounds = (int64_t)(std::sqrt((double)all * sums / row) + 0.5);
    return rounds <= 1 ? most : at_most((all + rounds - 1) / rounds, most);
}

// Whether dgamma and dbeta come from workgroups of the same launch that read the
// matrices again: 512 x 512 bf16 7.0 -> 3.6 us, 1000 x 1000 10.8 -> 8.5,
// 1000 x 64 6.0 -> 4.6, and one launch less for the host.  Not for more rows
// (4000 x 64 6.4 -> 7.3), more values (1000 x 2048 11.2 -> 14.1) or wider ones,
// whose workgroups have more threads than there are rows (100 x 8000 11 -> 13).
bool layer_norm_grad_small(int64_t rows, uint32_t width) {
    return rows <= 1024 && width <= 4096u && rows * (int64_t)width <= 1 << 20;
}

void launch_layer_norm_grad(int dt, const LnGradArgs& args, hipStream_t s) {
    LnGradArgs a = args;
    const RowShape r = row_shape(a.width, true);
    a.lpr = r.lpr;
    a.row_groups = layer_norm_grad_groups(dt, a.rows, a.width);
    if (dt == DT_FP16) layer_norm_grad_of<DT_FP16>(a, r, s);
    else if (dt == DT_BF16) layer_norm_grad_of<DT_BF16>(a, r, s);
    else layer_norm_grad_of<DT_FP32>(a, r, s);
}

void launch_layer_norm_grad_sum(int wdt, const float* part, uint32_t groups, uint32_t pitch, uint32_t width, void* dgamma,
                                void* dbeta, hipStream_t s) {
    const dim3 grid((width + 31u) / 32u), block(1024);
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
