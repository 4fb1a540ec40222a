// The launches of one type's kernels (-DTSG_LIN_DT=1: fp16, 2: bf16).
#include "tsgemm_linear_few.h"
#include "tsgemm_linear_kernel.h"
#include "tsgemm_linear_launch.h"
#include "tsgemm_linear_rows.h"
#include "tsgemm_linear_shape.h"

namespace tsg {

namespace {

constexpr int DT = TSG_LIN_DT;
constexpr uint32_t kCus = 256;  // MI355X

// Workgroups of a kernel that goes on to further work by the grid's size: 2^32 threads
// or more are not launched whole (the runtime counts them in 32 bits, without an error).
int64_t at_most(int64_t groups, int64_t most) { return groups < most ? groups : most; }

template <int AL, int BL, int EPI>
void product_of(int tile, const LinArgs& a, hipStream_t s) {
    const uint32_t units = a.m_blocks * a.n_blocks * a.splits, room = tile == 256 ? kCus : 2u * kCus;
    const dim3 grid(units < room ? units : room), block(256);
    if (tile == 256) hipLaunchKernelGGL((linear_kernel<DT, AL, BL, EPI, 256>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((linear_kernel<DT, AL, BL, EPI, 128>), grid, block, 0, s, a);
}

}  // namespace

template <>
void LinearOf<DT>::product(LinKind kind, int tile, const LinArgs& a, hipStream_t s) {
    switch (kind) {
        case LIN_KIND_GATED: return product_of<LIN_ALONG, LIN_ALONG, LIN_GATED>(tile, a, s);
        case LIN_KIND_LSE: return product_of<LIN_ALONG, LIN_ALONG, LIN_LSE>(tile, a, s);
        case LIN_KIND_DLOGITS: return product_of<LIN_ALONG, LIN_ALONG, LIN_DLOGITS>(tile, a, s);
        case LIN_KIND_DX: return product_of<LIN_ALONG, LIN_ACROSS, LIN_OUT>(tile, a, s);
        case LIN_KIND_DW: return product_of<LIN_ACROSS, LIN_ACROSS, LIN_OUT>(tile, a, s);
    }
}

template <>
void LinearOf<DT>::few(LinKind kind, const LinArgs& a, hipStream_t s) {
    const dim3 grid((unsigned)few_groups(a.N)), block(256);
    if (kind == LIN_KIND_GATED) {
        if (a.M <= 16u) hipLaunchKernelGGL((linear_few_kernel<DT, LIN_GATED, 1>), grid, block, 0, s, a);
        else hipLaunchKernelGGL((linear_few_kernel<DT, LIN_GATED, 2>), grid, block, 0, s, a);
    } else {
        if (a.M <= 16u) hipLaunchKernelGGL((linear_few_kernel<DT, LIN_LSE, 1>), grid, block, 0, s, a);
        else hipLaunchKernelGGL((linear_few_kernel<DT, LIN_LSE, 2>), grid, block, 0, s, a);
    }
}

template <>
void LinearOf<DT>::sum(const LinSumArgs& a, hipStream_t s) {
    const int64_t count = (int64_t)a.M * a.N / 8;
    hipLaunchKernelGGL(linear_sum_kernel<DT>, dim3((unsigned)at_most((count + 255) / 256, 1 << 20)), dim3(256), 0, s, a);
}

template <>
void LinearOf<DT>::gated_slope(const GatedGradArgs& a, hipStream_t s) {
    const int64_t groups = a.rows * (int64_t)((a.filled / 8u + 255u) / 256u);
    const dim3 grid((unsigned)at_most(groups, 4096)), block(256);
    if (a.act == kActBell) hipLaunchKernelGGL((gated_slope_kernel<DT, true>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((gated_slope_kernel<DT, false>), grid, block, 0, s, a);
}

template <>
void LinearOf<DT>::loss_rows(const LossGradArgs& a, hipStream_t s) {
    hipLaunchKernelGGL(loss_rows_kernel<DT>, dim3((unsigned)at_most(a.rows, 1024)), dim3(256), 0, s, a);
}

#if TSG_LIN_DT == 1  // what no type goes by
// 16 rows a workgroup, 64 threads a row: sum of exp(t) s over the parts, each thread's
// over every 64th part, eight requested at a time, then over the threads in order.
__global__ __launch_bounds__(1024) void loss_join_kernel(LossArgs a) {
    __shared__ float tops[64][16], sums[64][16];
    const uint32_t i = threadIdx.x & 15u, j = threadIdx.x >> 4;
    const auto zero_if_none = [](float e) { return e == -__builtin_inff() ? 0.0f : e; };
    for (int64_t first = (int64_t)blockIdx.x * 16; first < a.rows; first += (int64_t)gridDim.x * 16) {
        const int64_t r = first + i;
        float top = -__builtin_inff(), sum = 0.0f;
        if (r < a.rows) {
            for (uint32_t p = j; p < a.parts; p += 512u) {
                float2 v[8];
                float t = top;
#pragma unroll
                for (uint32_t k = 0; k < 8; ++k)
                    v[k] = p + 64u * k < a.parts ? a.part[(size_t)(p + 64u * k) * a.rows + r] : make_float2(-__builtin_inff(), 0.0f);
#pragma unroll
                for (int k = 0; k < 8; ++k) t = fmaxf(t, v[k].x);
                const float from = zero_if_none(t);
                sum *= exp_past(top, from);
#pragma unroll
                for (int k = 0; k < 8; ++k) sum += v[k].y * exp_past(v[k].x, from);
                top = t;
            }
        }
        __syncthreads();  // the rows before have been read
        tops[j][i] = top;
        sums[j][i] = sum;
        __syncthreads();
        if (j != 0u || r >= a.rows) continue;
        for (int k = 1; k < 64; ++k) top = fmaxf(top, tops[k][i]);
        const float from = zero_if_none(top);
        sum = 0.0f;
        for (int k = 0; k < 64; ++k) sum += sums[k][i] * exp_past(tops[k][i], from);
        // in fp64: the loss is the difference of two numbers that may be close
        const double lse = (double)from + log((double)sum);
        a.lse[r] = (float)lse;
        const int64_t t = a.target[r];
        a.loss[r] = t == a.ignore ? 0.0f : t >= 0 && t < (int64_t)a.vocab ? (float)(lse - (double)a.hit[r]) : __builtin_nanf("");
    }
}

// dweight = 0 of a call without rows
__global__ __launch_bounds__(256) void linear_zero_kernel(uint16_t* out, int64_t ld, int64_t rows, uint32_t width) {
    for (int64_t r = blockIdx.x; r < rows; r += gridDim.x)
        for (uint32_t n = threadIdx.x * 8u; n < width; n += 2048u) *(u32x4*)(out + r * ld + n) = u32x4{0, 0, 0, 0};
}

void launch_loss_join(const LossArgs& a, hipStream_t s) {
    hipLaunchKernelGGL(loss_join_kernel, dim3((unsigned)at_most((a.rows + 15) / 16, 1 << 16)), dim3(1024), 0, s, a);
}

void launch_linear_zero(uint16_t* out, int64_t ld, int64_t rows, uint32_t width, hipStream_t s) {
    hipLaunchKernelGGL(linear_zero_kernel, dim3((unsigned)at_most(rows, 4096)), dim3(256), 0, s, out, ld, rows, width);
}
#endif

}  // namespace tsg
