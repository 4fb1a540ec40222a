// Row operators around the block-scaled product, for gfx950 (CDNA4): layer norm
// and its gradient, and the conversion of activations to and from MX (E4M3
// codes, one E8M0 scale per 32 values along the row).
//
// All of them move far more bytes than they compute: a row is read once, kept
// in registers in fp32 and written once.  Statistics, sums and gradients of the
// weights are fp32; a value is rounded once, when it is stored.
//
// Everything works on chunks of 8 consecutive values of a row (16 bytes of a
// 16-bit type): four neighbouring lanes hold an MX block of 32, whose largest
// magnitude is a matter of two cross-lane moves inside the quad.  Rows need
// only the alignment of their elements (gfx950 loads and stores 16 bytes at any
// address); a chunk that the row's end cuts is loaded and stored value by value.
#pragma once

#include "tsgemm_device.h"

namespace tsg {

enum { DT_FP32 = 4 };  // tsgemm.h: TSGEMM_FP32

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));  // 16 bytes at a 2-byte boundary
typedef short s16x2 __attribute__((ext_vector_type(2)));

struct LnArgs {
    const void* x;
    const void* gamma;  // NULL: ones
    const void* beta;   // NULL: zeros
    void* y;            // NULL: not wanted
    float* mean;        // NULL: not wanted
    float* rstd;
    uint8_t* codes;     // [rows][width]; the kernels with CODES
    uint8_t* scales;    // [rows][width / 32]
    int64_t rows, ldx, ldy;
    uint32_t width;
    int wdt;            // type of gamma and beta: the activation's or DT_FP32
    float eps, inv_n;   // inv_n = 1 / width
    uint32_t lpr;       // lanes per row (kernels with several rows per workgroup): 4 ... 64
};

struct LnGradArgs {
    const void* dy;
    const void* x;
    const void* gamma;  // NULL: ones
    const float* mean;
    const float* rstd;
    void* dx;
    float* part;        // [gridDim.x][2][pitch]: a workgroup's sums for dgamma and dbeta; NULL: not wanted
    int64_t rows, lddy, ldx, lddx;
    uint32_t width, pitch;
    int wdt;
    float inv_n;
    uint32_t lpr;
};

// ---------------------------------------------------------------------------
// chunks of 8 values
// ---------------------------------------------------------------------------
template <int DT> struct ElemBytes { static constexpr int v = DT == DT_FP32 ? 4 : 2; };

template <int DT> struct Chunk { u32x4 w[DT == DT_FP32 ? 2 : 1]; };  // 8 values as they lie in memory

// The first `cnt` values of the chunk at p, zeros after them.
template <int DT>
__device__ __forceinline__ Chunk<DT> load_chunk(const char* p, int cnt) {
    Chunk<DT> c;
    constexpr int W = DT == DT_FP32 ? 2 : 1;
    if (cnt == 8) {
#pragma unroll
        for (int i = 0; i < W; ++i) c.w[i] = *(const u32x4_any*)(p + 16 * i);
    } else {
#pragma unroll
        for (int i = 0; i < W; ++i) c.w[i] = u32x4{0u, 0u, 0u, 0u};
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e < cnt) {
                if constexpr (DT == DT_FP32)
                    c.w[e / 4][e % 4] = *(const uint32_t*)(p + 4 * e);
                else
                    c.w[0][e / 2] |= (uint32_t)*(const uint16_t*)(p + 2 * e) << (16 * (e % 2));
            }
    }
    return c;
}

template <int DT>
__device__ __forceinline__ void unpack(const Chunk<DT>& c, float* f) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        if constexpr (DT == DT_FP32)
            f[e] = __builtin_bit_cast(float, (uint32_t)c.w[e / 4][e % 4]);
        else if constexpr (DT == DT_BF16)
            f[e] = __builtin_bit_cast(float, e % 2 ? c.w[0][e / 2] & 0xFFFF0000u : c.w[0][e / 2] << 16);
        else
            f[e] = (float)__builtin_bit_cast(f16x2, (uint32_t)c.w[0][e / 2])[e % 2];
    }
}

// Two fp32 values -> a dword of two 16-bit ones, nearest even.
template <int DT>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    if constexpr (DT == DT_BF16)
        return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{a, b}), bf16x2));
    else
        return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{a, b}), f16x2));
}

template <int DT>
__device__ __forceinline__ void store_chunk(char* p, int cnt, const float* f) {
    u32x4 w[DT == DT_FP32 ? 2 : 1];
#pragma unroll
    for (int i = 0; i < (DT == DT_FP32 ? 8 : 4); ++i) {
        if constexpr (DT == DT_FP32)
            w[i / 4][i % 4] = __builtin_bit_cast(uint32_t, f[i]);
        else
            w[0][i] = pack2<DT>(f[2 * i], f[2 * i + 1]);
    }
    if (cnt == 8) {
#pragma unroll
        for (int i = 0; i < (DT == DT_FP32 ? 2 : 1); ++i) *(u32x4_any*)(p + 16 * i) = w[i];
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e < cnt) {
                if constexpr (DT == DT_FP32)
                    *(uint32_t*)(p + 4 * e) = w[e / 4][e % 4];
                else
                    *(uint16_t*)(p + 2 * e) = (uint16_t)(w[0][e / 2] >> (16 * (e % 2)));
            }
    }
}

// 8 weights from column `col`, of the activation's type or fp32; `fill` where there are none.
template <int DT>
__device__ __forceinline__ void load_weights(const void* w, int wdt, uint32_t col, int cnt, float fill, float* f) {
    if (w == nullptr || cnt <= 0) {
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = fill;
    } else if (DT == DT_FP32 || wdt == DT_FP32) {
        unpack<DT_FP32>(load_chunk<DT_FP32>((const char*)w + (size_t)col * 4u, cnt), f);
    } else {
        unpack<DT>(load_chunk<DT>((const char*)w + (size_t)col * 2u, cnt), f);
    }
}

// ---------------------------------------------------------------------------
// sums over lanes.  Every step adds a lane's value to its mirror image's, so
// all lanes of a group end with the same bits.
// ---------------------------------------------------------------------------
template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
    const int b = __builtin_bit_cast(int, v);
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(b, b, CTRL, 0xF, 0xF, true));
}
constexpr int kQuadXor1 = 0xB1, kQuadXor2 = 0x4E, kHalfMirror = 0x141, kRowMirror = 0x140;

__device__ __forceinline__ float add_rows16(float v) {
    const uint32_t b = __builtin_bit_cast(uint32_t, v);
    const auto s = __builtin_amdgcn_permlane16_swap(b, b, false, false);
    return __builtin_bit_cast(float, (uint32_t)s[0]) + __builtin_bit_cast(float, (uint32_t)s[1]);
}
__device__ __forceinline__ float add_rows32(float v) {
    const uint32_t b = __builtin_bit_cast(uint32_t, v);
    const auto s = __builtin_amdgcn_permlane32_swap(b, b, false, false);
    return __builtin_bit_cast(float, (uint32_t)s[0]) + __builtin_bit_cast(float, (uint32_t)s[1]);
}

// Sum over groups of `lanes` (4, 8, ... 64, wave-uniform) neighbouring lanes.
__device__ __forceinline__ float group_sum(float v, uint32_t lanes) {
    v += dpp<kQuadXor1>(v);
    v += dpp<kQuadXor2>(v);
    if (lanes > 4u) v += dpp<kHalfMirror>(v);
    if (lanes > 8u) v += dpp<kRowMirror>(v);
    if (lanes > 16u) v = add_rows16(v);
    if (lanes > 32u) v = add_rows32(v);
    return v;
}

// Sum over the workgroup's waves of K values each.  `slot`: 16 * K floats of
// LDS, another than the previous call's (one barrier per call then suffices: a
// wave reaches the next call's barrier only after it has read this call's slot).
template <int K>
__device__ __forceinline__ void block_sum(float (&v)[K], float* slot) {
    const uint32_t wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] = group_sum(v[k], 64u);
    if ((threadIdx.x & 63u) == 0u)
#pragma unroll
        for (int k = 0; k < K; ++k) slot[wave * K + k] = v[k];
    lds_barrier();
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] = 0.f;
    for (uint32_t w = 0; w < waves; ++w)
#pragma unroll
        for (int k = 0; k < K; ++k) v[k] += slot[w * K + k];
}

// ---------------------------------------------------------------------------
// MX conversion (OCP Microscaling Formats specification v1.0): of a block of 32
// the scale is 2^(floor(log2 max |v|) - 8), 8 being E4M3's largest exponent, its
// code that exponent + 127, at least 0 (also for a block of zeros); the codes
// are v / scale, nearest even, held at +-448.  A NaN or an infinity becomes a
// NaN code and the scale follows the block's finite values, so it stays where
// it was and spoils no neighbour.
//
// gfx950's conversion takes the scale by the exponent field of an fp32 operand,
// which is the E8M0 code itself (0 stands for 2^-127), and rounds once; what
// would round past 448 it makes a NaN, hence the clamp.
// ---------------------------------------------------------------------------
__device__ __forceinline__ float max_abs8(const float* v) {
    // NaN goes through (maximum, not maxnum): one test then finds every odd value
    float m = __builtin_elementwise_maximum(__builtin_fabsf(v[0]), __builtin_fabsf(v[1]));
#pragma unroll
    for (int e = 2; e < 8; e += 2)
        m = __builtin_elementwise_maximum(__builtin_elementwise_maximum(m, __builtin_fabsf(v[e])), __builtin_fabsf(v[e + 1]));
    return m;
}
__device__ __forceinline__ float quad_max(float m) {
    m = __builtin_elementwise_maximum(m, dpp<kQuadXor1>(m));
    return __builtin_elementwise_maximum(m, dpp<kQuadXor2>(m));
}

// v: a quarter of a block per lane, the quad's lanes in order -> 8 codes; returns the scale's code.
__device__ __forceinline__ uint32_t encode_chunk(float* v, u32x2& codes) {
    float top = quad_max(max_abs8(v));
    const float inf = __builtin_inff();
    const bool odd = __builtin_amdgcn_ballot_w64(!(top < inf)) != 0u;  // wave-uniform, rare
    if (odd) {
        float m = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) m = __builtin_fmaxf(m, __builtin_fabsf(v[e]) < inf ? __builtin_fabsf(v[e]) : 0.f);
        top = quad_max(m);
    }
    const uint32_t field = __builtin_bit_cast(uint32_t, top) >> 23;
    const uint32_t scale = field > 8u ? field - 8u : 0u;
    const float lim = __builtin_bit_cast(float, ((scale + 8u) << 23) | 0x600000u);  // 448 * 2^(scale - 127)
    if (odd) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (__builtin_fabsf(v[e]) < inf) v[e] = __builtin_amdgcn_fmed3f(v[e], -lim, lim);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = __builtin_amdgcn_fmed3f(v[e], -lim, lim);
    }
    const float s = __builtin_bit_cast(float, scale << 23);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        s16x2 r = {0, 0};
        r = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(r, v[4 * i], v[4 * i + 1], s, false);
        r = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(r, v[4 * i + 2], v[4 * i + 3], s, true);
        codes[i] = __builtin_bit_cast(uint32_t, r);
    }
    return scale;
}

// 8 codes and their scale's code -> 8 values, exact.
__device__ __forceinline__ void decode_chunk(u32x2 codes, uint32_t scale, float* v) {
    const float s = __builtin_bit_cast(float, scale << 23);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(codes[i], s, false);
        const f32x2 b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(codes[i], s, true);
        v[4 * i] = a[0];
        v[4 * i + 1] = a[1];
        v[4 * i + 2] = b[0];
        v[4 * i + 3] = b[1];
    }
}

// ---------------------------------------------------------------------------
// layer norm, forward
// ---------------------------------------------------------------------------
// The chunk's part of a row, normalised, scaled and stored.
template <int DT, bool CODES>
__device__ __forceinline__ void ln_store(const LnArgs& a, int64_t row, uint32_t col, int cnt, float* v, float rstd,
                                         const float* g, const float* b) {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = __builtin_fmaf(v[e] * rstd, g[e], b[e]);
    if (cnt > 0 && a.y != nullptr)
        store_chunk<DT>((char*)a.y + ((size_t)row * a.ldy + col) * ElemBytes<DT>::v, cnt, v);
    if constexpr (CODES) {
        u32x2 c;
        const uint32_t s = encode_chunk(v, c);  // all lanes of a quad hold a chunk, or none does
        if (cnt > 0) {
            *(u32x2*)(a.codes + (size_t)row * a.width + col) = c;
            if ((threadIdx.x & 3u) == 0u) a.scales[(size_t)row * (a.width >> 5) + (col >> 5)] = (uint8_t)s;
        }
    }
}

// One row per workgroup at a time, at most NC chunks per thread.  The row after
// is requested before this one's sums, so that its latency passes behind them.
// WAVES: several rows per workgroup of 256 threads, args.lpr lanes each.
template <int DT, int NC, bool CODES, bool WAVES>
__global__ __launch_bounds__(WAVES ? 256 : 1024) void layer_norm_kernel(LnArgs a) {
    __shared__ float slots[2][16];
    constexpr int EB = ElemBytes<DT>::v;
    const uint32_t T = WAVES ? a.lpr : blockDim.x;          // threads of a row
    const uint32_t t = WAVES ? threadIdx.x & (T - 1u) : threadIdx.x;
    const uint32_t rows_wg = WAVES ? 256u / T : 1u;         // rows of a workgroup
    const int64_t step = (int64_t)gridDim.x * rows_wg;
    int64_t row = (int64_t)blockIdx.x * rows_wg + (WAVES ? threadIdx.x / T : 0u);

    uint32_t col[NC];
    int cnt[NC];
#pragma unroll
    for (int j = 0; j < NC; ++j) {
        col[j] = (t + j * T) * 8u;
        const int left = (int)a.width - (int)col[j];
        cnt[j] = left < 0 ? 0 : left > 8 ? 8 : left;
    }
    constexpr bool HOLD = NC <= 2;  // the weights stay in registers
    float g[HOLD ? NC : 1][8], b[HOLD ? NC : 1][8];
    if constexpr (HOLD) {
#pragma unroll
        for (int j = 0; j < NC; ++j) {
            load_weights<DT>(a.gamma, a.wdt, col[j], cnt[j], 1.f, g[j]);
            load_weights<DT>(a.beta, a.wdt, col[j], cnt[j], 0.f, b[j]);
        }
    }
    Chunk<DT> next[NC];
    auto fetch = [&](int64_t r) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < NC; ++j)
            next[j] = load_chunk<DT>((const char*)a.x + ((size_t)r * a.ldx + col[j]) * EB, r < a.rows ? cnt[j] : 0);
    };
    fetch(row);
    // the count of rounds is the workgroup's: lanes without a row go along
    for (int64_t base = (int64_t)blockIdx.x * rows_wg; base < a.rows; base += step, row += step) {
        float v[NC][8];
#pragma unroll
        for (int j = 0; j < NC; ++j) unpack<DT>(next[j], v[j]);
        fetch(row + step);

        float s[1] = {0.f};
#pragma unroll
        for (int j = 0; j < NC; ++j)
#pragma unroll
            for (int e = 0; e < 8; ++e) s[0] += v[j][e];
        if constexpr (WAVES) s[0] = group_sum(s[0], T);
        else block_sum<1>(s, slots[0]);
        const float mean = s[0] * a.inv_n;
        s[0] = 0.f;
#pragma unroll
        for (int j = 0; j < NC; ++j) {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[j][e] -= mean;
            if (cnt[j] < 8) {
#pragma unroll
                for (int e = 0; e < 8; ++e) v[j][e] = e < cnt[j] ? v[j][e] : 0.f;
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) s[0] = __builtin_fmaf(v[j][e], v[j][e], s[0]);
        }
        if constexpr (WAVES) s[0] = group_sum(s[0], T);
        else block_sum<1>(s, slots[1]);
        const float rstd = rsqrtf(__builtin_fmaf(s[0], a.inv_n, a.eps));

        const bool live = row < a.rows;
        if (t == 0u && live && a.mean != nullptr) {
            a.mean[row] = mean;
            a.rstd[row] = rstd;
        }
#pragma unroll
        for (int j = 0; j < NC; ++j) {
            if constexpr (HOLD) {
                ln_store<DT, CODES>(a, row, col[j], live ? cnt[j] : 0, v[j], rstd, g[j], b[j]);
            } else {
                load_weights<DT>(a.gamma, a.wdt, col[j], cnt[j], 1.f, g[0]);
                load_weights<DT>(a.beta, a.wdt, col[j], cnt[j], 0.f, b[0]);
                ln_store<DT, CODES>(a, row, col[j], live ? cnt[j] : 0, v[j], rstd, g[0], b[0]);
            }
        }
    }
}

// Rows of any width, one workgroup of 1024 threads each: the row is read three
// times (the second and third time mostly out of a cache).
template <int DT, bool CODES>
__global__ __launch_bounds__(1024) void layer_norm_wide_kernel(LnArgs a) {
    __shared__ float slots[2][16];
    constexpr int EB = ElemBytes<DT>::v;
    const uint32_t rounds = (a.width + 8191u) / 8192u;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const char* x = (const char*)a.x + (size_t)row * a.ldx * EB;
        float s[1] = {0.f}, mean = 0.f, v[8];
        for (uint32_t i = 0; i < 2u * rounds; ++i) {  // first the sum, then the squares about the mean
            if (i == rounds) {
                block_sum<1>(s, slots[0]);
                mean = s[0] * a.inv_n;
                s[0] = 0.f;
            }
            const uint32_t col = (threadIdx.x + 1024u * (i % rounds)) * 8u;
            const int cnt = col >= a.width ? 0 : a.width - col < 8u ? (int)(a.width - col) : 8;
            unpack<DT>(load_chunk<DT>(x + (size_t)col * EB, cnt), v);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float d = e < cnt ? v[e] - mean : 0.f;
                s[0] = i < rounds ? s[0] + d : __builtin_fmaf(d, d, s[0]);
            }
        }
        block_sum<1>(s, slots[1]);
        const float rstd = rsqrtf(__builtin_fmaf(s[0], a.inv_n, a.eps));
        if (threadIdx.x == 0u && a.mean != nullptr) {
            a.mean[row] = mean;
            a.rstd[row] = rstd;
        }
        for (uint32_t i = 0; i < rounds; ++i) {
            const uint32_t col = (threadIdx.x + 1024u * i) * 8u;
            const int cnt = col >= a.width ? 0 : a.width - col < 8u ? (int)(a.width - col) : 8;
            float g[8], b[8];
            unpack<DT>(load_chunk<DT>(x + (size_t)col * EB, cnt), v);
            load_weights<DT>(a.gamma, a.wdt, col, cnt, 1.f, g);
            load_weights<DT>(a.beta, a.wdt, col, cnt, 0.f, b);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = e < cnt ? v[e] - mean : 0.f;
            ln_store<DT, CODES>(a, row, col, cnt, v, rstd, g, b);
        }
    }
}

// ---------------------------------------------------------------------------
// layer norm, gradient: with h = (x - mean) rstd and g = dy gamma,
//   dx = rstd (g - mean(g) - h mean(g h)),  dgamma = sum_rows dy h,  dbeta = sum_rows dy.
// A thread keeps its columns' sums over the workgroup's rows in registers; the
// workgroups' sums meet in a second, small launch in a fixed order.
// ---------------------------------------------------------------------------
template <int DT, int NC, bool WAVES>
__global__ __launch_bounds__(WAVES ? 256 : 1024) void layer_norm_grad_kernel(LnGradArgs a) {
    __shared__ float slots[2][32];
    __shared__ float sums[WAVES ? 256 * 8 : 1];
    constexpr int EB = ElemBytes<DT>::v;
    const uint32_t T = WAVES ? a.lpr : blockDim.x;
    const uint32_t t = WAVES ? threadIdx.x & (T - 1u) : threadIdx.x;
    const uint32_t rows_wg = WAVES ? 256u / T : 1u;
    const int64_t step = (int64_t)gridDim.x * rows_wg;
    int64_t row = (int64_t)blockIdx.x * rows_wg + (WAVES ? threadIdx.x / T : 0u);

    uint32_t col[NC];
    int cnt[NC];
    float gam[NC][8], dg[NC][8], db[NC][8];
#pragma unroll
    for (int j = 0; j < NC; ++j) {
        col[j] = (t + j * T) * 8u;
        const int left = (int)a.width - (int)col[j];
        cnt[j] = left < 0 ? 0 : left > 8 ? 8 : left;
        load_weights<DT>(a.gamma, a.wdt, col[j], cnt[j], 1.f, gam[j]);
#pragma unroll
        for (int e = 0; e < 8; ++e) dg[j][e] = db[j][e] = 0.f;
    }
    Chunk<DT> nx[NC], nd[NC];
    float n_mean = 0.f, n_rstd = 0.f;
    auto fetch = [&](int64_t r) __attribute__((always_inline)) {
        const bool live = r < a.rows;
        n_mean = live ? a.mean[r] : 0.f;
        n_rstd = live ? a.rstd[r] : 0.f;
#pragma unroll
        for (int j = 0; j < NC; ++j) {
            nx[j] = load_chunk<DT>((const char*)a.x + ((size_t)r * a.ldx + col[j]) * EB, live ? cnt[j] : 0);
            nd[j] = load_chunk<DT>((const char*)a.dy + ((size_t)r * a.lddy + col[j]) * EB, live ? cnt[j] : 0);
        }
    };
    fetch(row);
    uint32_t slot = 0;
    for (int64_t base = (int64_t)blockIdx.x * rows_wg; base < a.rows; base += step, row += step, slot ^= 1u) {
        float h[NC][8], g[NC][8];
        const float mean = n_mean, rstd = n_rstd;
#pragma unroll
        for (int j = 0; j < NC; ++j) {
            unpack<DT>(nx[j], h[j]);
            unpack<DT>(nd[j], g[j]);
        }
        fetch(row + step);
        float s[2] = {0.f, 0.f};
#pragma unroll
        for (int j = 0; j < NC; ++j)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                // past the row's end dy is 0, and so are g, g h and dy h (mean and rstd
                // that are no numbers only reach columns that are not stored)
                const float d = g[j][e];
                h[j][e] = (h[j][e] - mean) * rstd;
                dg[j][e] = __builtin_fmaf(d, h[j][e], dg[j][e]);
                db[j][e] += d;
                g[j][e] = d * gam[j][e];
            }
#pragma unroll
        for (int j = 0; j < NC; ++j) {
            if (cnt[j] < 8) {
#pragma unroll
                for (int e = 0; e < 8; ++e) h[j][e] = e < cnt[j] ? h[j][e] : 0.f;
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                s[0] += g[j][e];
                s[1] = __builtin_fmaf(g[j][e], h[j][e], s[1]);
            }
        }
        if constexpr (WAVES) {
            s[0] = group_sum(s[0], T);
            s[1] = group_sum(s[1], T);
        } else {
            block_sum<2>(s, slots[slot]);
        }
        const float c1 = -rstd * (s[0] * a.inv_n), c2 = -rstd * (s[1] * a.inv_n);
        if (row < a.rows) {
#pragma unroll
            for (int j = 0; j < NC; ++j) {
                float o[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) o[e] = __builtin_fmaf(rstd, g[j][e], __builtin_fmaf(c2, h[j][e], c1));
                if (cnt[j] > 0) store_chunk<DT>((char*)a.dx + ((size_t)row * a.lddx + col[j]) * EB, cnt[j], o);
            }
        }
    }
    if (a.part == nullptr) return;
    // the workgroup's sums; with several rows per workgroup those of its row
    // groups are added up in order
    float* part = a.part + (size_t)blockIdx.x * 2u * a.pitch;
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int j = 0; j < NC; ++j) {
            float (&v)[8] = k == 0 ? dg[j] : db[j];
            if constexpr (WAVES) {
                lds_barrier();
#pragma unroll
                for (int e = 0; e < 8; ++e) sums[e * 256 + threadIdx.x] = v[e];
                lds_barrier();
                for (uint32_t o = threadIdx.x; o < 8u * T; o += 256u) {  // T columns times 8
                    const uint32_t e = o / T, lane = o & (T - 1u);
                    float s = 0.f;
                    for (uint32_t r = 0; r < rows_wg; ++r) s += sums[e * 256u + r * T + lane];
                    const uint32_t c = (lane + j * T) * 8u + e;
                    if (c < a.pitch) part[k * a.pitch + c] = s;
                }
            } else if (cnt[j] > 0) {  // the pitch is a multiple of 8
                *(f32x4*)(part + k * a.pitch + col[j]) = f32x4{v[0], v[1], v[2], v[3]};
                *(f32x4*)(part + k * a.pitch + col[j] + 4) = f32x4{v[4], v[5], v[6], v[7]};
            }
        }
}

// Rows of any width, one workgroup of 1024 threads each; the workgroup's sums
// for the weights gather in its own part of the workspace.
template <int DT>
__global__ __launch_bounds__(1024) void layer_norm_grad_wide_kernel(LnGradArgs a) {
    __shared__ float slots[2][32];
    constexpr int EB = ElemBytes<DT>::v;
    const uint32_t rounds = (a.width + 8191u) / 8192u;
    float* part = a.part ? a.part + (size_t)blockIdx.x * 2u * a.pitch : nullptr;
    bool first = true;
    uint32_t slot = 0;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, first = false, slot ^= 1u) {
        const char* x = (const char*)a.x + (size_t)row * a.ldx * EB;
        const char* dy = (const char*)a.dy + (size_t)row * a.lddy * EB;
        const float mean = a.mean[row], rstd = a.rstd[row];
        float s[2] = {0.f, 0.f}, c1 = 0.f, c2 = 0.f;
        for (uint32_t i = 0; i < 2u * rounds; ++i) {
            if (i == rounds) {
                block_sum<2>(s, slots[slot]);
                c1 = -rstd * (s[0] * a.inv_n);
                c2 = -rstd * (s[1] * a.inv_n);
            }
            const uint32_t col = (threadIdx.x + 1024u * (i % rounds)) * 8u;
            const int cnt = col >= a.width ? 0 : a.width - col < 8u ? (int)(a.width - col) : 8;
            if (cnt == 0) continue;
            float h[8], g[8], gam[8];
            unpack<DT>(load_chunk<DT>(x + (size_t)col * EB, cnt), h);
            unpack<DT>(load_chunk<DT>(dy + (size_t)col * EB, cnt), g);
            load_weights<DT>(a.gamma, a.wdt, col, cnt, 1.f, gam);
            float o[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                h[e] = e < cnt ? (h[e] - mean) * rstd : 0.f;
                if (i < rounds) {
                    if (part != nullptr && e < cnt) {
                        float* p = part + col + e;
                        p[0] = first ? g[e] * h[e] : __builtin_fmaf(g[e], h[e], p[0]);
                        p[a.pitch] = first ? g[e] : p[a.pitch] + g[e];
                    }
                    g[e] *= gam[e];
                    s[0] += g[e];
                    s[1] = __builtin_fmaf(g[e], h[e], s[1]);
                } else {
                    o[e] = __builtin_fmaf(rstd, g[e] * gam[e], __builtin_fmaf(c2, h[e], c1));
                }
            }
            if (i >= rounds) store_chunk<DT>((char*)a.dx + ((size_t)row * a.lddx + col) * EB, cnt, o);
        }
    }
}

// dgamma and dbeta from the workgroups' sums: 64 columns per workgroup, the
// sums split over its 16 waves, each adding its share in order.  `groups` may be
// 0 (no rows): the gradients are then 0.
template <int WDT>
__global__ __launch_bounds__(1024) void layer_norm_grad_sum_kernel(const float* part, uint32_t groups, uint32_t pitch,
                                                                   uint32_t width, void* dgamma, void* dbeta) {
    __shared__ float sums[2][16][64];
    const uint32_t lane = threadIdx.x & 63u, wave = threadIdx.x >> 6;
    const uint32_t c = blockIdx.x * 64u + lane;
    float s[2] = {0.f, 0.f};
    if (c < width) {
        const uint32_t each = (groups + 15u) / 16u;
        const uint32_t end = (wave + 1u) * each < groups ? (wave + 1u) * each : groups;
#pragma unroll 8
        for (uint32_t g = wave * each; g < end; ++g) {
            const float* p = part + (size_t)g * 2u * pitch + c;
            s[0] += p[0];
            s[1] += p[pitch];
        }
    }
    sums[0][wave][lane] = s[0];
    sums[1][wave][lane] = s[1];
    lds_barrier();
    if (wave < 2u && c < width) {
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < 16; ++w) v += sums[wave][w][lane];
        void* out = wave == 0u ? dgamma : dbeta;
        if (out != nullptr) {
            if constexpr (WDT == DT_FP32) ((float*)out)[c] = v;
            else if constexpr (WDT == DT_BF16) ((__bf16*)out)[c] = (__bf16)v;
            else ((_Float16*)out)[c] = (_Float16)v;
        }
    }
}

// ---------------------------------------------------------------------------
// activations to MX and back, 8 values per thread
// ---------------------------------------------------------------------------
// Chunk i of the matrix -> its row and column.  `cpr` chunks per row.
struct ChunkAt { int64_t row; uint32_t col; };
__device__ __forceinline__ ChunkAt chunk_at(uint64_t i, uint32_t cpr) {
    if (i >> 32 == 0u) {
        const uint32_t r = (uint32_t)i / cpr;
        return {(int64_t)r, ((uint32_t)i - r * cpr) * 8u};
    }
    const uint64_t r = i / cpr;
    return {(int64_t)r, (uint32_t)(i - r * cpr) * 8u};
}

// x's rows `ld` apart; a matrix without gaps comes as one with ld == width.
template <int DT>
__global__ __launch_bounds__(256) void mx_quantize_kernel(const void* x, int64_t ld, uint64_t chunks, uint32_t width,
                                                          uint8_t* codes, uint8_t* scales) {
    constexpr int EB = ElemBytes<DT>::v;
    const bool flat = ld == (int64_t)width;
    const uint64_t step = (uint64_t)gridDim.x * 256u;
    // chunks is a multiple of 4 and so is the step: a quad is all in or all out
    for (uint64_t i = (uint64_t)blockIdx.x * 256u + threadIdx.x; i < chunks; i += step) {
        size_t at = (size_t)i * 8u;
        if (!flat) {
            const ChunkAt c = chunk_at(i, width >> 3);
            at = (size_t)c.row * ld + c.col;
        }
        float v[8];
        unpack<DT>(load_chunk<DT>((const char*)x + at * EB, 8), v);
        u32x2 c;
        const uint32_t s = encode_chunk(v, c);
        *(u32x2*)(codes + (size_t)i * 8u) = c;
        if ((threadIdx.x & 3u) == 0u) scales[i >> 2] = (uint8_t)s;
    }
}

template <int DT>
__global__ __launch_bounds__(256) void mx_dequantize_kernel(const uint8_t* codes, const uint8_t* scales, uint64_t chunks,
                                                            uint32_t width, void* out, int64_t ld) {
    constexpr int EB = ElemBytes<DT>::v;
    const bool flat = ld == (int64_t)width;
    const uint64_t step = (uint64_t)gridDim.x * 256u;
    for (uint64_t i = (uint64_t)blockIdx.x * 256u + threadIdx.x; i < chunks; i += step) {
        float v[8];
        decode_chunk(*(const u32x2*)(codes + (size_t)i * 8u), scales[i >> 2], v);
        size_t at = (size_t)i * 8u;
        if (!flat) {
            const ChunkAt c = chunk_at(i, width >> 3);
            at = (size_t)c.row * ld + c.col;
        }
        store_chunk<DT>((char*)out + at * EB, 8, v);
    }
}

}  // namespace tsg
