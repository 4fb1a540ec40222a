// The gated projection and the cross entropy's sums for few rows (up to 32), for
// gfx950 (CDNA4): every weight is read once and used for all rows, so the weights'
// bytes are the time while there are few.
//
// A workgroup of 4 waves takes 16 weight rows (16 of each weight of the gated
// projection) at a time; the waves share the sum, 128 values of it each in turn, and
// add up in LDS.  A wave's fragments come straight from memory to registers, 16 bytes
// a lane and row, the next 128 values' loads on their way while these are multiplied
// (16x16x32 MFMA, x's rows past the last read as zeros).
//
// Measured bf16: one row, 4096 x 8192 (two weights, 134 MB) 26.5 us, 5.1 TB/s; 16 rows,
// 4096 x 131072 (1.07 GB) 239 us, 4.5 TB/s, of 1, 8 and 32 rows 174, 196 and 352 (takes_few of
// tsgemm_linear_shape.h says when the tile kernel, 240 there, is taken).  With two sets of
// the first one's weights in turn, half of them in the Infinity Cache, 24.0 and 239 us; in
// that set-up loads past the caches (nt) take 26.3 and 265, 256 values a turn 26.6 and 243,
// twice the workgroups 24.0 and 240.
#pragma once

#include "tsgemm_linear_kernel.h"

namespace tsg {

template <int DT>
__device__ __forceinline__ f32x4 mfma_seen(u32x4 a, u32x4 b, f32x4 c) {
    if constexpr (DT == DT_FP16)
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// EPI: LIN_GATED or LIN_LSE.  MB: blocks of 16 rows of x.
template <int DT, int EPI, int MB>
__global__ __launch_bounds__(256, EPI == LIN_GATED && MB == 2 ? 1 : 2) void linear_few_kernel(LinArgs args) {
    constexpr int NB = EPI == LIN_GATED ? 2 : 1;  // weights
    constexpr int U = 4, DEEP = 32 * U;           // MFMA steps and values of the sum of one turn
    __shared__ f32x4 part[2][4][MB * NB][64];     // of two tiles in turn: one barrier a tile
    const uint32_t lane = threadIdx.x & 63u, l16 = lane & 15u, lg = lane >> 4;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t K = args.Ka, N = args.N, M = args.M;
    const uint32_t tiles = (N + 15u) / 16u, turns = (K + 4u * DEEP - 1u) / (4u * DEEP);  // of every wave
    // a thread's place in the sums: row m of a block, column n
    const uint32_t m = threadIdx.x >> 4, n = threadIdx.x & 15u;
    // ... which lane 16 (n / 4) + m holds, as value n % 4
    const uint32_t from = 16u * (n >> 2) + m;
    const Act act(args.act);
    float top[MB], sum[MB];
    int64_t target[MB];
    if constexpr (EPI == LIN_LSE) {
#pragma unroll
        for (int b = 0; b < MB; ++b) {
            top[b] = -__builtin_inff();
            sum[b] = 0.0f;
            target[b] = m + 16u * b < M ? args.target[m + 16u * b] : -1;
        }
    }

    // ---- loads: turn by turn of a tile, tile by tile, one turn ahead of the MFMAs and
    // without a branch, so that the compiler counts what is on its way.  Past the sum's end,
    // in rows that do not exist and past the last tile no descriptor covers anything:
    // zeros, for which nothing is requested. ----
    u32x4 w[2][NB][U], x[2][MB][U];
    uint32_t ld_tile = blockIdx.x, ld_turn = 0;
    const uint32_t x_off = l16 * (uint32_t)args.lda * 2u + lg * 16u;
    auto load = [&](auto s_c) __attribute__((always_inline)) {
        constexpr int s = decltype(s_c)::value;
        const uint32_t k0 = (4u * ld_turn + wave) * DEEP;
        const bool live = ld_tile < tiles && k0 < K;
        const uint32_t n0 = live ? ld_tile * 16u : 0u, at = live ? k0 : 0u, rows = N - n0 < 16u ? N - n0 : 16u;
#pragma unroll
        for (int i = 0; i < NB; ++i) {
            const uint16_t* base = i == 0 ? args.b : args.b2;
            const int64_t ld = i == 0 ? args.ldb : args.ldb2;
            const __amdgpu_buffer_rsrc_t r = make_rsrc(base + (int64_t)n0 * ld + at, live ? ((rows - 1u) * (uint32_t)ld + K - at) * 2u : 0u);
            const uint32_t off = l16 * (uint32_t)ld * 2u + lg * 16u;
#pragma unroll
            for (int u = 0; u < U; ++u)
                w[s][i][u] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                    r, k0 + 32u * u + 8u * lg < K ? off + 64u * u : 0x80000000u, 0, 0));
        }
#pragma unroll
        for (int b = 0; b < MB; ++b) {
            const uint32_t have = M > 16u * b ? (M - 16u * b < 16u ? M - 16u * b : 16u) : 0u;
            const __amdgpu_buffer_rsrc_t r = make_rsrc(args.a + (int64_t)(have ? 16 * b : 0) * args.lda + at,
                                                       live && have ? ((have - 1u) * (uint32_t)args.lda + K - at) * 2u : 0u);
#pragma unroll
            for (int u = 0; u < U; ++u)
                x[s][b][u] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                    r, k0 + 32u * u + 8u * lg < K ? x_off + 64u * u : 0x80000000u, 0, 0));
        }
        if (++ld_turn == turns) {
            ld_turn = 0;
            ld_tile += gridDim.x;
        }
    };
    f32x4 acc[MB][NB];
    auto clear = [&]() __attribute__((always_inline)) {
#pragma unroll
        for (int b = 0; b < MB; ++b)
#pragma unroll
            for (int i = 0; i < NB; ++i) acc[b][i] = f32x4{0.f, 0.f, 0.f, 0.f};
    };
    uint32_t side = 0;
    auto finish = [&](uint32_t n0) __attribute__((always_inline)) {
#pragma unroll
        for (int b = 0; b < MB; ++b)
#pragma unroll
            for (int i = 0; i < NB; ++i) part[side][wave][b * NB + i][lane] = acc[b][i];
        lds_barrier();
        auto total = [&](int b, int i) __attribute__((always_inline)) -> float {
            float v = 0.0f;
#pragma unroll
            for (int k = 0; k < 4; ++k) v += reinterpret_cast<const float*>(&part[side][k][b * NB + i][from])[n & 3u];
            return v;
        };
#pragma unroll
        for (int b = 0; b < MB; ++b) {
            const uint32_t r = m + 16u * b, c = n0 + n;
            if constexpr (EPI == LIN_GATED) {
                const float g = total(b, 0), up = total(b, 1);
                float bell, p;
                if (args.act == kActBell) p = act_share<true>(act, g, bell);
                else p = act_share<false>(act, g, bell);
                if (r < M && c < N) {
                    args.y[(int64_t)r * args.ldy + c] = (uint16_t)pack2<DT>(g * p * up, 0.0f);
                    if (args.gate) args.gate[(int64_t)r * args.ldgate + c] = (uint16_t)pack2<DT>(g, 0.0f);
                    if (args.up) args.up[(int64_t)r * args.ldup + c] = (uint16_t)pack2<DT>(up, 0.0f);
                }
            } else {
                const float l = total(b, 0);
                if (r < M && c < N) {
                    if (target[b] == (int64_t)c) args.hit[r] = l;
                    // the sum is in units of exp(top)
                    const float now = fmaxf(top[b], l), base = now == -__builtin_inff() ? 0.0f : now;
                    sum[b] = sum[b] * exp_past(top[b], base) + exp_past(l, base);
                    top[b] = now;
                }
            }
        }
        side ^= 1u;  // the next tile's sums go elsewhere; by the one after it every wave has passed that one's barrier
    };
    uint32_t tile = blockIdx.x, turn = 0;
    auto multiply = [&](auto s_c) __attribute__((always_inline)) -> bool {
        constexpr int s = decltype(s_c)::value;
        load(std::integral_constant<int, 1 - s>{});
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int b = 0; b < MB; ++b)
#pragma unroll
                for (int i = 0; i < NB; ++i) acc[b][i] = mfma_seen<DT>(w[s][i][u], x[s][b][u], acc[b][i]);
        if (++turn != turns) return true;
        finish(tile * 16u);
        clear();
        turn = 0;
        tile += gridDim.x;
        return tile < tiles;
    };
    clear();
    load(std::integral_constant<int, 0>{});
    while (multiply(std::integral_constant<int, 0>{}) && multiply(std::integral_constant<int, 1>{})) {
    }
    if constexpr (EPI == LIN_LSE) {
#pragma unroll
        for (int b = 0; b < MB; ++b) {
            float all = top[b];
#pragma unroll
            for (int d = 1; d < 16; d *= 2) all = fmaxf(all, __shfl_xor(all, d));
            float s = sum[b] * exp_past(top[b], all == -__builtin_inff() ? 0.0f : all);
#pragma unroll
            for (int d = 1; d < 16; d *= 2) s += __shfl_xor(s, d);
            if (n == 0u && m + 16u * b < M) args.part[(size_t)blockIdx.x * M + m + 16u * b] = make_float2(all, s);
        }
    }
}

}  // namespace tsg
