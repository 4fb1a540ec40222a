// Row operators around the block-scaled product, for gfx950 (CDNA4): layer norm
// and its gradient, and the conversion of activations to and from MX (E4M3
// codes, one E8M0 scale per 32 values along the row).
//
// All of them move far more bytes than they compute: a row is read once, kept
// in registers in fp32 and written once.  Statistics, sums and gradients of the
// weights are fp32; a value is rounded once, when it is stored.
//
// Measured on the MI355X against a copy's 5.35 TB/s (inputs and outputs changing
// from pass to pass): layer norm 16000 x 4000 fp16 48.6 us, 5.27 TB/s; 8192 x 8192
// bf16 to codes 44 us, 4.6 TB/s, of which its vector instructions alone take 29;
// gradient 8192 x 8192 bf16 81 us, 4.97 TB/s (17 MB of partial sums come on top);
// quantize 16384 x 4096 bf16 36.9 us and dequantize 8192 x 8192 36.5 us, 5.5 TB/s.
//
// Everything works on chunks of 8 consecutive values of a row (16 bytes of a
// 16-bit type): four neighbouring lanes hold an MX block of 32, whose largest
// magnitude is a matter of two cross-lane moves inside the quad.  Rows need
// only the alignment of their elements (gfx950 loads and stores 16 bytes at any
// address).  A row that is not a multiple of 8 wide ends with a chunk that
// reaches back over the one before (Chunks below): both lanes compute and store
// the same values for the columns they share, and the sums count them once.
// Against loads and stores of the cut chunk in pieces of 4, 2 and 1 values:
// layer norm 20000 x 2501 bf16 67 -> 58 us.  Rows below 8 values have no other way.
#pragma once

#include "tsgemm_device.h"

namespace tsg {

enum { DT_FP32 = 4 };  // tsgemm.h: TSGEMM_FP32

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));  // 16 bytes at a 2-byte boundary
typedef uint32_t u32x2_any __attribute__((ext_vector_type(2), aligned(2)));
typedef uint32_t u32_any __attribute__((aligned(2)));
typedef float f32x4_any __attribute__((ext_vector_type(4), aligned(4)));
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
    float eps;
    double inv_n;       // 1 / width
    uint32_t lpr;       // lanes per row (kernels with several rows per workgroup): 4 ... 64
};

struct LnGradArgs {
    const void* dy;
    const void* x;
    const void* gamma;  // NULL: ones
    const float* mean;
    const float* rstd;
    void* dx;
    float* part;        // [row_groups][2][pitch]: a workgroup's sums for dgamma and dbeta; NULL: not wanted
    void* dgamma;       // of workgroups past row_groups; NULL: not wanted
    void* dbeta;
    uint32_t row_groups;
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

// The first `cnt` values of the chunk at p, zeros after them.  A chunk that the
// row's end cuts comes in pieces of 4, 2 and 1 values.  FULL: cnt is 8 or 0.
template <int DT, bool FULL = false>
__device__ __forceinline__ Chunk<DT> load_chunk(const char* p, int cnt) {
    Chunk<DT> c;
    constexpr int W = DT == DT_FP32 ? 2 : 1;
    if (cnt == 8) {
#pragma unroll
        for (int i = 0; i < W; ++i) c.w[i] = *(const u32x4_any*)(p + 16 * i);
    } else {
#pragma unroll
        for (int i = 0; i < W; ++i) c.w[i] = u32x4{0u, 0u, 0u, 0u};
        if (FULL || cnt <= 0) return c;
        if constexpr (DT == DT_FP32) {
            u32x2 two = {0u, 0u};
            uint32_t one = 0u;
            if (cnt & 4) c.w[0] = *(const u32x4_any*)p;
            if (cnt & 2) two = *(const u32x2_any*)(p + 4 * (cnt & 4));
            if (cnt & 1) one = *(const uint32_t*)(p + 4 * (cnt & 6));
            if (cnt & 4) c.w[1] = u32x4{cnt & 2 ? two.x : one, two.y, cnt & 2 ? one : 0u, 0u};
            else c.w[0] = u32x4{cnt & 2 ? two.x : one, two.y, cnt & 2 ? one : 0u, 0u};
        } else {
            uint32_t two = 0u, one = 0u;
            if (cnt & 4) {
                const u32x2 v = *(const u32x2_any*)p;
                c.w[0].x = v.x;
                c.w[0].y = v.y;
            }
            if (cnt & 2) two = *(const u32_any*)(p + 2 * (cnt & 4));
            if (cnt & 1) one = *(const uint16_t*)(p + 2 * (cnt & 6));
            const uint32_t first = cnt & 2 ? two : one, second = cnt & 2 ? one : 0u;
            if (cnt & 4) {
                c.w[0].z = first;
                c.w[0].w = second;
            } else {
                c.w[0].x = first;
                c.w[0].y = second;
            }
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

template <int DT, bool FULL = false>
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
    } else if (!FULL && cnt > 0) {
        if constexpr (DT == DT_FP32) {
            if (cnt & 4) *(u32x4_any*)p = w[0];
            const u32x4 r = cnt & 4 ? w[1] : w[0];
            if (cnt & 2) *(u32x2_any*)(p + 4 * (cnt & 4)) = u32x2{r.x, r.y};
            if (cnt & 1) *(uint32_t*)(p + 4 * (cnt & 6)) = cnt & 2 ? r.z : r.x;
        } else {
            if (cnt & 4) *(u32x2_any*)p = u32x2{w[0].x, w[0].y};
            const uint32_t first = cnt & 4 ? w[0].z : w[0].x, second = cnt & 4 ? w[0].w : w[0].y;
            if (cnt & 2) *(u32_any*)(p + 2 * (cnt & 4)) = first;
            if (cnt & 1) *(uint16_t*)(p + 2 * (cnt & 6)) = (uint16_t)(cnt & 2 ? second : first);
        }
    }
}

// 8 weights from column `col`, of the activation's type or fp32; `fill` where there are none.
template <int DT, bool FULL = false>
__device__ __forceinline__ void load_weights(const void* w, int wdt, uint32_t col, int cnt, float fill, float* f) {
    if (w == nullptr || cnt <= 0) {
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = fill;
    } else if (DT == DT_FP32 || wdt == DT_FP32) {
        unpack<DT_FP32>(load_chunk<DT_FP32, FULL>((const char*)w + (size_t)col * 4u, cnt), f);
    } else {
        unpack<DT>(load_chunk<DT, FULL>((const char*)w + (size_t)col * 2u, cnt), f);
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
constexpr int kQuadXor1 = 0xB1, kQuadXor2 = 0x4E, kHalfMirror = 0x141, kRowMirror = 0x140, kRowRotate8 = 0x128;

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

// The same in fp64, for the forward statistics of rows that lanes of one wave
// hold: a thread's own few values add up in fp32, what crosses lanes in fp64.
template <int CTRL>
__device__ __forceinline__ double dpp(double v) {
    const u32x2 b = __builtin_bit_cast(u32x2, v);
    const u32x2 r = {__builtin_bit_cast(uint32_t, dpp<CTRL>(__builtin_bit_cast(float, (uint32_t)b.x))),
                     __builtin_bit_cast(uint32_t, dpp<CTRL>(__builtin_bit_cast(float, (uint32_t)b.y)))};
    return __builtin_bit_cast(double, r);
}
__device__ __forceinline__ double group_sum(double v, uint32_t lanes) {
    v += dpp<kQuadXor1>(v);
    v += dpp<kQuadXor2>(v);
    if (lanes > 4u) v += dpp<kHalfMirror>(v);
    if (lanes > 8u) v += dpp<kRowMirror>(v);
    if (lanes > 16u) {
        const u32x2 b = __builtin_bit_cast(u32x2, v);
        const auto lo = __builtin_amdgcn_permlane16_swap(b.x, b.x, false, false);
        const auto hi = __builtin_amdgcn_permlane16_swap(b.y, b.y, false, false);
        v = __builtin_bit_cast(double, (u32x2{lo[0], hi[0]})) + __builtin_bit_cast(double, (u32x2{lo[1], hi[1]}));
    }
    if (lanes > 32u) {
        const u32x2 b = __builtin_bit_cast(u32x2, v);
        const auto lo = __builtin_amdgcn_permlane32_swap(b.x, b.x, false, false);
        const auto hi = __builtin_amdgcn_permlane32_swap(b.y, b.y, false, false);
        v = __builtin_bit_cast(double, (u32x2{lo[0], hi[0]})) + __builtin_bit_cast(double, (u32x2{lo[1], hi[1]}));
    }
    return v;
}

// Sum over the workgroup of K values each: over a wave in fp32, over the waves
// in F.  `slot`: 16 * K values of LDS, another than the previous call's (one
// barrier per call then suffices: a wave reaches the next call's barrier only
// after it has read this call's slot).
template <int K, class F>
__device__ __forceinline__ void block_sum(F (&v)[K], F* slot) {
    const uint32_t wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
    float w1[K];
#pragma unroll
    for (int k = 0; k < K; ++k) w1[k] = group_sum((float)v[k], 64u);
    if ((threadIdx.x & 63u) == 0u)
#pragma unroll
        for (int k = 0; k < K; ++k) slot[wave * K + k] = w1[k];
    lds_barrier();
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] = F(0);
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
__device__ __forceinline__ uint32_t encode_chunk(const float* v, u32x2& codes) {
    float top = quad_max(max_abs8(v));
    const float inf = __builtin_inff();
    const bool odd = __builtin_amdgcn_ballot_w64(!(top < inf)) != 0u;  // wave-uniform, rare
    if (odd) {
        float m = 0.f;
        asm volatile("" : "+v"(m));  // keeps this block a branch: computed for every chunk it would cost a third more
#pragma unroll
        for (int e = 0; e < 8; ++e) m = __builtin_fmaxf(m, __builtin_fabsf(v[e]) < inf ? __builtin_fabsf(v[e]) : 0.f);
        top = quad_max(m);
    }
    const uint32_t field = __builtin_bit_cast(uint32_t, top) >> 23;
    const uint32_t scale = field > 8u ? field - 8u : 0u;
    const float lim = __builtin_bit_cast(float, ((scale + 8u) << 23) | 0x600000u);  // 448 * 2^(scale - 127)
    const float s = __builtin_bit_cast(float, scale << 23);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        float c[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) c[e] = __builtin_amdgcn_fmed3f(v[4 * i + e], -lim, lim);
        s16x2 r = {0, 0};
        r = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(r, c[0], c[1], s, false);
        r = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(r, c[2], c[3], s, true);
        codes[i] = __builtin_bit_cast(uint32_t, r);
    }
    if (odd) {
        uint32_t nan = 0x7Fu;
        asm volatile("" : "+v"(nan));
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (!(__builtin_fabsf(v[e]) < inf)) codes[e / 4] |= nan << (8 * (e % 4));
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
template <int DT, bool CODES, bool FULL = false>
__device__ __forceinline__ void ln_store(const LnArgs& a, int64_t row, uint32_t col, int cnt, float* v, float rstd,
                                         const float* g, const float* b) {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = __builtin_fmaf(v[e] * rstd, g[e], b[e]);
    if (cnt > 0 && a.y != nullptr)
        store_chunk<DT, FULL>((char*)a.y + ((size_t)row * a.ldy + col) * ElemBytes<DT>::v, cnt, v);
    if constexpr (CODES) {
        u32x2 c;
        const uint32_t s = encode_chunk(v, c);  // all lanes of a quad hold a chunk, or none does
        if (cnt > 0) {
            *(u32x2*)(a.codes + (size_t)row * a.width + col) = c;
            if ((threadIdx.x & 3u) == 0u) a.scales[(size_t)row * (a.width >> 5) + (col >> 5)] = (uint8_t)s;
        }
    }
}

// (sum of squares about the mean) / width + eps -> (...)^(-1/2)
__device__ __forceinline__ float inverse_root(double v) { return (float)rsqrt(v); }

// The chunks of a row that a thread works on: every T-th from its own.  FULL:
// rows of 8 values or more; a chunk is there whole or not at all, and `skip` of
// its first values are another lane's too (8: it is not there).  Else (one chunk
// per row) cnt says how many values there are.
template <int NC, bool FULL>
struct Chunks {
    uint32_t col[NC];
    int cnt[NC], skip[NC];
    __device__ __forceinline__ Chunks(uint32_t width, uint32_t t, uint32_t T) {
#pragma unroll
        for (int j = 0; j < NC; ++j) {
            col[j] = (t + j * T) * 8u;
            const int left = (int)width - (int)col[j];
            cnt[j] = left <= 0 ? 0 : FULL || left > 8 ? 8 : left;
            skip[j] = FULL ? (left <= 0 ? 8 : left < 8 ? 8 - left : 0) : 0;
            if (FULL && skip[j] > 0 && skip[j] < 8) col[j] = width - 8u;
        }
    }
    // f's values that this lane counts, zeros for the others
    __device__ __forceinline__ float counted(int j, int e, float f) const { return FULL ? (e >= skip[j] ? f : 0.f) : (e < cnt[j] ? f : 0.f); }
    __device__ __forceinline__ bool cut(int j) const { return FULL ? skip[j] != 0 : cnt[j] != 8; }
};

// One row per workgroup at a time, at most NC chunks per thread.  The row after
// is requested before this one's sums, so that its latency passes behind them.
// WAVES: several rows per workgroup of 256 threads, args.lpr lanes each.
template <int DT, int NC, bool CODES, bool WAVES, bool FULL>
__global__ __launch_bounds__(WAVES ? 256 : 1024) void layer_norm_kernel(LnArgs a) {
    __shared__ double slots[2][16];
    constexpr int EB = ElemBytes<DT>::v;
    const uint32_t T = WAVES ? a.lpr : blockDim.x;          // threads of a row
    const uint32_t t = WAVES ? threadIdx.x & (T - 1u) : threadIdx.x;
    const uint32_t rows_wg = WAVES ? 256u / T : 1u;         // rows of a workgroup
    const int64_t step = (int64_t)gridDim.x * rows_wg;
    int64_t row = (int64_t)blockIdx.x * rows_wg + (WAVES ? threadIdx.x / T : 0u);

    const Chunks<NC, FULL> c(a.width, t, T);
    float g[NC][8], b[NC][8];
#pragma unroll
    for (int j = 0; j < NC; ++j) {
        load_weights<DT, FULL>(a.gamma, a.wdt, c.col[j], c.cnt[j], 1.f, g[j]);
        load_weights<DT, FULL>(a.beta, a.wdt, c.col[j], c.cnt[j], 0.f, b[j]);
    }
    Chunk<DT> next[NC];
    auto fetch = [&](int64_t r) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < NC; ++j)
            next[j] = load_chunk<DT, FULL>((const char*)a.x + ((size_t)r * a.ldx + c.col[j]) * EB, r < a.rows ? c.cnt[j] : 0);
    };
    fetch(row);
    // the count of rounds is the workgroup's: lanes without a row go along
    for (int64_t base = (int64_t)blockIdx.x * rows_wg; base < a.rows; base += step, row += step) {
        float v[NC][8];
#pragma unroll
        for (int j = 0; j < NC; ++j) unpack<DT>(next[j], v[j]);
        fetch(row + step);

        double s[1];
        float part = 0.f;
#pragma unroll
        for (int j = 0; j < NC; ++j) {
            float p = ((v[j][0] + v[j][1]) + (v[j][2] + v[j][3])) + ((v[j][4] + v[j][5]) + (v[j][6] + v[j][7]));
            if (c.cut(j)) {
                p = 0.f;
#pragma unroll
                for (int e = 0; e < 8; ++e) p += c.counted(j, e, v[j][e]);
            }
            part += p;
        }
        s[0] = part;
        if constexpr (WAVES) s[0] = group_sum(s[0], T);
        else block_sum<1>(s, slots[0]);
        const float mean = (float)(s[0] * a.inv_n);
        part = 0.f;
#pragma unroll
        for (int j = 0; j < NC; ++j) {
            float q = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                v[j][e] -= mean;
                q = __builtin_fmaf(v[j][e], v[j][e], q);
            }
            if (c.cut(j)) {
                q = 0.f;
#pragma unroll
                for (int e = 0; e < 8; ++e) q = __builtin_fmaf(c.counted(j, e, v[j][e]), v[j][e], q);
            }
            part += q;
        }
        s[0] = part;
        if constexpr (WAVES) s[0] = group_sum(s[0], T);
        else block_sum<1>(s, slots[1]);
        const float rstd = inverse_root(s[0] * a.inv_n + (double)a.eps);

        const bool live = row < a.rows;
        if (t == 0u && live && a.mean != nullptr) {
            a.mean[row] = mean;
            a.rstd[row] = rstd;
        }
#pragma unroll
        for (int j = 0; j < NC; ++j)
            ln_store<DT, CODES, FULL>(a, row, c.col[j], live ? c.cnt[j] : 0, v[j], rstd, g[j], b[j]);
    }
}

// Rows of any width, one workgroup of 1024 threads each: the row is read three
// times (the second and third time mostly out of a cache).  Only past 16384
// values, which no longer fit the registers: 2000 x 30016 bf16 95 us, 2.5 TB/s.
template <int DT, bool CODES>
__global__ __launch_bounds__(1024) void layer_norm_wide_kernel(LnArgs a) {
    __shared__ double slots[2][16];
    constexpr int EB = ElemBytes<DT>::v;
    const uint32_t rounds = (a.width + 8191u) / 8192u;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const char* x = (const char*)a.x + (size_t)row * a.ldx * EB;
        double s[1] = {0.0};
        float mean = 0.f, v[8];
        for (uint32_t i = 0; i < 2u * rounds; ++i) {  // first the sum, then the squares about the mean
            if (i == rounds) {
                block_sum<1>(s, slots[0]);
                mean = (float)(s[0] * a.inv_n);
                s[0] = 0.0;
            }
            const uint32_t col = (threadIdx.x + 1024u * (i % rounds)) * 8u;
            const int cnt = col >= a.width ? 0 : a.width - col < 8u ? (int)(a.width - col) : 8;
            unpack<DT>(load_chunk<DT>(x + (size_t)col * EB, cnt), v);
            float part = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float d = e < cnt ? v[e] - mean : 0.f;
                part = i < rounds ? part + d : __builtin_fmaf(d, d, part);
            }
            s[0] += part;
        }
        block_sum<1>(s, slots[1]);
        const float rstd = inverse_root(s[0] * a.inv_n + (double)a.eps);
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
// workgroups' sums meet in a second, small launch in a fixed order.  Small
// matrices are read a second time instead, column by column, by workgroups of
// the same launch.
// ---------------------------------------------------------------------------
template <int WDT>
__device__ __forceinline__ void store_weight(void* out, uint32_t at, float v) {
    if (out == nullptr) return;
    if constexpr (WDT == DT_FP32) ((float*)out)[at] = v;
    else if constexpr (WDT == DT_BF16) ((__bf16*)out)[at] = (__bf16)v;
    else ((_Float16*)out)[at] = (_Float16)v;
}

// dgamma and dbeta of the 8 columns from 8 * block, over all rows; the last ones
// of a row that is not a multiple of 8 wide reach back as in Chunks.
template <int DT, bool FULL>
__device__ __forceinline__ void column_sums(const LnGradArgs& a, uint32_t block) {
    __shared__ float waves_sums[16][16];
    constexpr int EB = ElemBytes<DT>::v;
    const Chunks<1, FULL> c(a.width, block, 1u);
    float s[16] = {};
#pragma unroll 2
    for (int64_t r = threadIdx.x; r < a.rows; r += blockDim.x) {
        const float mean = a.mean[r], rstd = a.rstd[r];
        float x[8], d[8];
        unpack<DT>(load_chunk<DT, FULL>((const char*)a.x + ((size_t)r * a.ldx + c.col[0]) * EB, c.cnt[0]), x);
        unpack<DT>(load_chunk<DT, FULL>((const char*)a.dy + ((size_t)r * a.lddy + c.col[0]) * EB, c.cnt[0]), d);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            s[e] = __builtin_fmaf(d[e], (x[e] - mean) * rstd, s[e]);
            s[8 + e] += d[e];
        }
    }
#pragma unroll
    for (int k = 0; k < 16; ++k) s[k] = group_sum(s[k], 64u);
    if ((threadIdx.x & 63u) == 0u)
#pragma unroll
        for (int k = 0; k < 16; ++k) waves_sums[threadIdx.x >> 6][k] = s[k];
    lds_barrier();
    if (threadIdx.x < 16u && (int)(threadIdx.x & 7u) < c.cnt[0]) {
        float v = 0.f;
        for (uint32_t w = 0; w < blockDim.x >> 6; ++w) v += waves_sums[w][threadIdx.x];
        void* out = threadIdx.x < 8u ? a.dgamma : a.dbeta;
        const uint32_t at = c.col[0] + (threadIdx.x & 7u);
        if (a.wdt == DT_FP32) store_weight<DT_FP32>(out, at, v);
        else store_weight<DT>(out, at, v);
    }
}

// AHEAD rows are on their way while one is worked on.  With two chunks per
// thread and row (RAW) a row is kept as it was read and unpacked twice.
template <int DT, int NC, bool WAVES, bool FULL, int AHEAD>
__global__ __launch_bounds__(WAVES ? 256 : 1024) void layer_norm_grad_kernel(LnGradArgs a) {
    __shared__ float slots[2][32];
    __shared__ float sums[WAVES ? 256 * 8 : 1];
    if (blockIdx.x >= a.row_groups) return column_sums<DT, FULL>(a, blockIdx.x - a.row_groups);
    constexpr int EB = ElemBytes<DT>::v;
    constexpr bool RAW = !WAVES && NC > 1;
    const uint32_t T = WAVES ? a.lpr : blockDim.x;
    const uint32_t t = WAVES ? threadIdx.x & (T - 1u) : threadIdx.x;
    const uint32_t rows_wg = WAVES ? 256u / T : 1u;
    const int64_t step = (int64_t)a.row_groups * rows_wg;
    int64_t row = (int64_t)blockIdx.x * rows_wg + (WAVES ? threadIdx.x / T : 0u);

    const Chunks<NC, FULL> c(a.width, t, T);
    float gam[RAW ? 1 : NC][8], dg[NC][8], db[NC][8];
#pragma unroll
    for (int j = 0; j < NC; ++j) {
        if constexpr (!RAW) load_weights<DT, FULL>(a.gamma, a.wdt, c.col[j], c.cnt[j], 1.f, gam[j]);
#pragma unroll
        for (int e = 0; e < 8; ++e) dg[j][e] = db[j][e] = 0.f;
    }
    struct Row {
        Chunk<DT> x[NC], dy[NC];
        float mean, rstd;
    };
    auto fetch = [&](Row& n, int64_t r) __attribute__((always_inline)) {
        const bool live = r < a.rows;
        n.mean = live ? a.mean[r] : 0.f;
        n.rstd = live ? a.rstd[r] : 0.f;
#pragma unroll
        for (int j = 0; j < NC; ++j) {
            n.x[j] = load_chunk<DT, FULL>((const char*)a.x + ((size_t)r * a.ldx + c.col[j]) * EB, live ? c.cnt[j] : 0);
            n.dy[j] = load_chunk<DT, FULL>((const char*)a.dy + ((size_t)r * a.lddy + c.col[j]) * EB, live ? c.cnt[j] : 0);
        }
    };
    uint32_t slot = 0;
    // where no chunk is, dy is 0, and so are g, g h and dy h (mean and rstd that
    // are no numbers only reach columns that are not stored)
    auto open = [&](const Row& n, int j, float mean, float rstd, float* h, float* d) __attribute__((always_inline)) {
        unpack<DT>(n.x[j], h);
        unpack<DT>(n.dy[j], d);
#pragma unroll
        for (int e = 0; e < 8; ++e) h[e] = (h[e] - mean) * rstd;
    };
    auto work = [&](Row& n) __attribute__((always_inline)) {
        float h[RAW ? 1 : NC][8], g[RAW ? 1 : NC][8];
        const float mean = n.mean, rstd = n.rstd;
        float s[2] = {0.f, 0.f};
        Row kept;
        if constexpr (RAW) kept = n;
#pragma unroll
        for (int j = 0; j < NC; ++j) {
            const int k = RAW ? 0 : j;
            open(n, j, mean, rstd, h[k], g[k]);
            if constexpr (RAW) load_weights<DT, FULL>(a.gamma, a.wdt, c.col[j], c.cnt[j], 1.f, gam[0]);
            float p0 = 0.f, p1 = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float d = g[k][e];
                dg[j][e] = __builtin_fmaf(d, h[k][e], dg[j][e]);
                db[j][e] += d;
                g[k][e] = d * gam[k][e];
                p0 += g[k][e];
                p1 = __builtin_fmaf(g[k][e], h[k][e], p1);
            }
            if (c.cut(j)) {
                p0 = p1 = 0.f;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    p0 += c.counted(j, e, g[k][e]);
                    p1 += c.counted(j, e, g[k][e] * h[k][e]);
                }
            }
            s[0] += p0;
            s[1] += p1;
        }
        fetch(n, row + AHEAD * step);
        if constexpr (WAVES) {
            s[0] = group_sum(s[0], T);
            s[1] = group_sum(s[1], T);
        } else {
            block_sum<2>(s, slots[slot]);
            slot ^= 1u;
        }
        const float c1 = -rstd * (s[0] * a.inv_n), c2 = -rstd * (s[1] * a.inv_n);
        if (row < a.rows) {
#pragma unroll
            for (int j = 0; j < NC; ++j) {
                const int k = RAW ? 0 : j;
                if constexpr (RAW) {
                    open(kept, j, mean, rstd, h[0], g[0]);
                    load_weights<DT, FULL>(a.gamma, a.wdt, c.col[j], c.cnt[j], 1.f, gam[0]);
#pragma unroll
                    for (int e = 0; e < 8; ++e) g[0][e] *= gam[0][e];
                }
                float o[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) o[e] = __builtin_fmaf(rstd, g[k][e], __builtin_fmaf(c2, h[k][e], c1));
                if (c.cnt[j] > 0) store_chunk<DT, FULL>((char*)a.dx + ((size_t)row * a.lddx + c.col[j]) * EB, c.cnt[j], o);
            }
        }
        row += step;
    };
    Row n[AHEAD];
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) fetch(n[i], row + i * step);
    // the count of rounds is the workgroup's: lanes without a row go along
    int64_t base = (int64_t)blockIdx.x * rows_wg;
    while (base < a.rows) {
        work(n[0]);
        base += step;
        if constexpr (AHEAD > 1) {
            if (base >= a.rows) break;
            work(n[1]);
            base += step;
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
                    const Chunks<NC, FULL> of(a.width, lane, T);
                    if (of.cnt[j] > 0) part[k * a.pitch + of.col[j] + e] = s;
                }
            } else if (c.cnt[j] > 0) {
                *(f32x4_any*)(part + k * a.pitch + c.col[j]) = f32x4{v[0], v[1], v[2], v[3]};
                *(f32x4_any*)(part + k * a.pitch + c.col[j] + 4) = f32x4{v[4], v[5], v[6], v[7]};
            }
        }
}

// Rows of any width, one workgroup of 1024 threads each; the workgroup's sums
// for the weights gather in its own part of the workspace, 32 bytes of which move
// for every value: 2000 x 30016 bf16 306-322 us (value by value 553).
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
            for (int e = 0; e < 8; ++e) h[e] = e < cnt ? (h[e] - mean) * rstd : 0.f;
            if (part != nullptr && i < rounds) {  // the pitch is a multiple of 8: a cut chunk has room for 8
                f32x4* p = (f32x4*)(part + col);
                f32x4* q = (f32x4*)(part + a.pitch + col);
#pragma unroll
                for (int w = 0; w < 2; ++w) {
                    f32x4 sg = {0.f, 0.f, 0.f, 0.f}, sb = sg;
                    if (!first) {
                        sg = p[w];
                        sb = q[w];
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        sg[e] = __builtin_fmaf(g[4 * w + e], h[4 * w + e], sg[e]);
                        sb[e] += g[4 * w + e];
                    }
                    p[w] = sg;
                    q[w] = sb;
                }
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                if (i < rounds) {
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

// dgamma and dbeta from the workgroups' sums: 32 columns per workgroup from `first` on, 4 per
// lane, so that a wave reads 8 workgroups' sums at once; the lanes' and the 16
// waves' shares meet in a fixed order.  `groups` may be 0 (no rows): the
// gradients are then 0.
template <int WDT>
__global__ __launch_bounds__(1024) void layer_norm_grad_sum_kernel(const float* part, uint32_t groups, uint32_t pitch,
                                                                   uint32_t first, uint32_t width, void* dgamma, void* dbeta) {
    __shared__ float sums[2][16][32];
    const uint32_t lane = threadIdx.x & 63u, wave = threadIdx.x >> 6;
    const uint32_t c = first + blockIdx.x * 32u + (lane & 7u) * 4u;
    f32x4 s[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
    if (c < pitch) {
#pragma unroll 4
        for (uint32_t g = wave * 8u + (lane >> 3); g < groups; g += 128u) {
            const float* p = part + (size_t)g * 2u * pitch + c;
            s[0] += *(const f32x4*)p;
            s[1] += *(const f32x4*)(p + pitch);
        }
    }
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            float v = s[k][e];
            v += dpp<kRowRotate8>(v);
            v = add_rows32(add_rows16(v));
            if (lane < 8u) sums[k][wave][lane * 4u + e] = v;
        }
    lds_barrier();
    if (threadIdx.x < 64u) {
        const uint32_t k = threadIdx.x >> 5, at = first + blockIdx.x * 32u + (threadIdx.x & 31u);
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < 16; ++w) v += sums[k][w][threadIdx.x & 31u];
        if (at < width) store_weight<WDT>(k == 0u ? dgamma : dbeta, at, v);
    }
}

// ---------------------------------------------------------------------------
// activations to MX and back, 8 values per thread: bound by memory at any size
// that fills the chip, by the launch (2.1 us for 512 x 512) below
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
