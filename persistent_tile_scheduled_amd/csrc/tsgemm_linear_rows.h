// The small kernels around the tile kernel of tsgemm_linear_kernel.h: what joins a
// loss, prepares a gradient and adds up split products.  All are bound by memory
// or by their launch.
#pragma once

#include "tsgemm_linear_kernel.h"

namespace tsg {

template <int DT>
__device__ __forceinline__ float unpack1(uint16_t v) {
    if constexpr (DT == DT_FP16) return (float)__builtin_bit_cast(_Float16, v);
    else return __builtin_bit_cast(float, (uint32_t)v << 16);
}

// ---------------------------------------------------------------------------
// gated projection: dg = dy * u * act'(g), du = dy * act(g), in fp32 and rounded once to
// the 16 bits that the matrix core takes.  Of the outputs' error, 1.7e-3 in bf16 and 2.1e-4
// in fp16 by their own rounding, that makes 2.3e-3 and 2.9e-4; a second operand for what is
// rounded off would double the products.
// ---------------------------------------------------------------------------
struct GatedGradArgs {
    const uint16_t* dy;
    const uint16_t* gate;
    const uint16_t* up;
    uint16_t* d;     // [rows][ld]: dg, then du from column `pitch` on
    int64_t lddy, ldgate, ldup, ld;
    int64_t rows;
    uint32_t hidden, filled, pitch;  // columns [hidden, filled) are zero
    int act;
};

// act(g) = g p(g) and its derivative p + g p'.  Where p or the bell has run out of fp32
// they are what they tend to, 0 and g, 0 and 1: not 0 * inf, of a gate that was kept as an
// infinity (fp16: any from 65520 on).
template <bool BELL>
__device__ __forceinline__ void act_slope(const Act& k, float g, float& value, float& slope) {
    float bell;
    const float p = act_share<BELL>(k, g, bell);
    value = p == 0.0f ? 0.0f : g * p;
    if constexpr (BELL) {
        slope = bell == 0.0f ? p : __builtin_fmaf(g * 0.39894228f, bell, p);
    } else {
        // p (1 - p) z'
        const float rise = p * (1.0f - p) * __builtin_fmaf(3.0f * k.k, act_square(g), k.c) * (1.0f / kLog2e);
        slope = p == 0.0f || p == 1.0f ? p : __builtin_fmaf(g, rise, p);
    }
}

template <int DT, bool BELL>
__global__ __launch_bounds__(256) void gated_slope_kernel(GatedGradArgs a) {
    const Act act(a.act);
    const uint32_t chunks = a.filled / 8u;
    const uint32_t per_row = (chunks + 255u) / 256u;
    for (uint64_t w = blockIdx.x; w < (uint64_t)a.rows * per_row; w += gridDim.x) {
        const int64_t r = (int64_t)(w / per_row);
        const uint32_t n = ((uint32_t)(w % per_row) * 256u + threadIdx.x) * 8u;
        if (n >= a.filled) continue;
        const uint16_t* dy = a.dy + r * a.lddy + n;
        const uint16_t* g = a.gate + r * a.ldgate + n;
        const uint16_t* u = a.up + r * a.ldup + n;
        u32x4 wd = {0, 0, 0, 0}, wg = wd, wu = wd;
        if (n + 8u <= a.hidden) {
            wd = *(const u32x4_at2*)dy;
            wg = *(const u32x4_at2*)g;
            wu = *(const u32x4_at2*)u;
        } else {
#pragma unroll
            for (uint32_t e = 0; e < 7u; ++e)
                if (n + e < a.hidden) {
                    wd[e / 2] |= (uint32_t)dy[e] << (16 * (e % 2));
                    wg[e / 2] |= (uint32_t)g[e] << (16 * (e % 2));
                    wu[e / 2] |= (uint32_t)u[e] << (16 * (e % 2));
                }
        }
        float dg[8], du[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float d = unpack1<DT>((uint16_t)(wd[e / 2] >> (16 * (e % 2))));
            const float up = unpack1<DT>((uint16_t)(wu[e / 2] >> (16 * (e % 2))));
            float value, slope;
            act_slope<BELL>(act, unpack1<DT>((uint16_t)(wg[e / 2] >> (16 * (e % 2)))), value, slope);
            dg[e] = d * up * slope;
            du[e] = d * value;
            if (n + e >= a.hidden) dg[e] = du[e] = 0.0f;
        }
        uint16_t* to = a.d + r * a.ld + n;
        store8<DT>(to, dg, 8u);
        store8<DT>(to + a.pitch, du, 8u);
    }
}

// ---------------------------------------------------------------------------
// cross entropy
// ---------------------------------------------------------------------------
struct LossArgs {
    const float2* part;  // [parts][rows]: t and s
    const float* hit;
    const int64_t* target;
    float* loss;
    float* lse;
    int64_t ignore;
    int64_t rows;
    uint32_t parts, vocab;
};

struct LossGradArgs {
    const float* dloss;
    const float* lse;
    const int64_t* target;
    const uint16_t* x;
    uint16_t* counted_x;  // [rows][ldcx]: x, zero in rows that do not count; NULL: not wanted
    LossRow* row;
    float* unscale;       // what dl is to be multiplied with
    int64_t ignore, rows, ldx, ldcx;
    uint32_t width, vocab;
};

// What the gradient needs of every row.  dl is held over the largest finite |dloss| of
// the rows that count (an infinite one is its own row's matter), so that of a loss's mean
// over the rows, all of whose dloss are alike, no rounding of dloss itself enters; fp16,
// which has few exponents, holds 2^13 times that, and its least normal value stands for
// 2^-27 of the largest.  Every workgroup finds that largest value for itself.
template <int DT>
__global__ __launch_bounds__(256) void loss_rows_kernel(LossGradArgs a) {
    __shared__ float most[4];
    auto counts = [&](int64_t r) -> bool {
        const int64_t t = a.target[r];
        return t != a.ignore && t >= 0 && t < (int64_t)a.vocab;
    };
    constexpr float kMore = DT == DT_FP16 ? 8192.0f : 1.0f;
    float top = 0.0f;
    for (int64_t r = threadIdx.x; r < a.rows; r += 256)
        if (counts(r)) {
            const float d = fabsf(a.dloss[r]);
            top = d < __builtin_inff() ? fmaxf(top, d) : top;
        }
#pragma unroll
    for (int d = 1; d < 64; d *= 2) top = fmaxf(top, __shfl_xor(top, d));
    if ((threadIdx.x & 63u) == 0u) most[threadIdx.x >> 6] = top;
    __syncthreads();
    top = fmaxf(fmaxf(most[0], most[1]), fmaxf(most[2], most[3]));
    if (!(top >= 0x1p-110f)) top = 1.0f;  // no scale comes of it
    if (blockIdx.x == 0 && threadIdx.x == 0) *a.unscale = top / kMore;
    for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const bool is = counts(r);
        if (threadIdx.x == 0) {
            LossRow row = {0.0f, 0.0f, -1, 0};
            if (is) row = {a.lse[r], a.dloss[r] / top * kMore, (int32_t)a.target[r], 0};
            a.row[r] = row;
        }
        if (a.counted_x)
            for (uint32_t n = threadIdx.x * 8u; n < a.width; n += 2048u) {
                u32x4 v = {0, 0, 0, 0};
                if (is) v = *(const u32x4*)(a.x + r * a.ldx + n);
                *(u32x4*)(a.counted_x + r * a.ldcx + n) = v;
            }
    }
}

// ---------------------------------------------------------------------------
// out = the splits' sums added up in order, 8 values per thread
// ---------------------------------------------------------------------------
struct LinSumArgs {
    const float* sums;  // [splits][M][N]
    uint32_t splits, M, N;
    uint16_t* out;
    uint16_t* out2;
    int64_t ldo, ldo2;
    uint32_t half, out_rows;
    const float* unscale;
};
template <int DT>
__global__ __launch_bounds__(256) void linear_sum_kernel(LinSumArgs a) {
    const uint64_t count = (uint64_t)a.M * a.N;
    const float scale = a.unscale ? *a.unscale : 1.0f;
    for (uint64_t i = ((uint64_t)blockIdx.x * 256u + threadIdx.x) * 8u; i < count; i += (uint64_t)gridDim.x * 2048u) {
        const uint32_t m = (uint32_t)(i / a.N), n = (uint32_t)(i % a.N);
        const bool upper = m >= a.half;
        const uint32_t mo = upper ? m - a.half : m;
        if (mo >= a.out_rows) continue;
        f32x4 x = {0.f, 0.f, 0.f, 0.f}, y = x;
#pragma unroll 4
        for (uint32_t s = 0; s < a.splits; ++s) {
            x += *(const f32x4*)(a.sums + s * count + i);
            y += *(const f32x4*)(a.sums + s * count + i + 4);
        }
        float v[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            v[e] = x[e] * scale;
            v[4 + e] = y[e] * scale;
        }
        store8<DT>((upper ? a.out2 + (int64_t)mo * a.ldo2 : a.out + (int64_t)mo * a.ldo) + n, v, 8u);
    }
}

}  // namespace tsg
