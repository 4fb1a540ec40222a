// The matrix products of the gated projection, of the cross entropy of a linear
// head, and of their gradients, for gfx950 (CDNA4).  One tile kernel with three
// pairs of operand layouts and four epilogues:
//
//   x Wg^T and x Wu^T  (both operands lie along the sum)   y = act(g) * u
//   x W^T              (both along the sum)                a row's largest logit and sum of exponentials
//   x W^T              (both along the sum)                dl = d * (exp(l - lse) - onehot)
//   dl W               (dl along the sum, W across it)     dx
//   dl^T x             (both across it)                    dW
//
// A product's values stay in the accumulators until the epilogue has made of them
// what is written: the two projections and the logits never reach memory.
//
// One workgroup of 4 waves (2 x 2) forms one T x T tile (T = 256 or 128) over a
// range of 64-deep slabs.  Slabs go straight into LDS (buffer_load ... lds).  An
// operand along the sum lies there in rows of 64 and is read 16 bytes a lane
// (ds_read_b128), one across the sum in rows of T and is read through the
// transpose read ds_read_b64_tr_b16.  Either way chunks of 16 bytes change places
// inside a row (swz_a, swz_b), so that a read's lanes spread over the banks.  Rows
// and columns past a matrix's end, and the sum's last slab past its end, read
// zeros: a wave's descriptor ends with the matrix, and of rows along the sum the
// lanes past the end ask for an address that no descriptor covers.
#pragma once

#include "tile_scheduler.h"
#include "tsgemm_device.h"

namespace tsg {

typedef uint32_t u32x4_at2 __attribute__((ext_vector_type(4), aligned(2)));  // 16 bytes at a 2-byte boundary

constexpr float kLog2e = 1.44269504f;

enum { LIN_ALONG = 0, LIN_ACROSS = 1 };  // an operand's layout: the sum's index fastest, or slowest
enum { LIN_GATED = 0, LIN_LSE = 1, LIN_DLOGITS = 2, LIN_OUT = 3 };

// What the cross entropy's gradient needs of a row.
struct LossRow {
    float lse2;      // its logsumexp times log2 e
    float d;         // its share of the gradient, times the scale of dl
    int32_t target;  // -1: the row does not count
    int32_t unused;
};

struct LinArgs {
    const uint16_t* a;   // [M][K] or [K][M], rows lda apart
    const uint16_t* b;   // [N][K] or [K][N]
    const uint16_t* a2;  // the sum's second half: slabs from seg_slabs on (LIN_OUT)
    const uint16_t* b2;  // the same, or the up projection's weight (LIN_GATED)
    int64_t lda, ldb, ldb2;
    uint32_t M, N;       // rows and columns that exist; across the sum, columns of a and b in memory
    uint32_t Ka, Kb;     // the sum's length (of one half), as far as a and b hold values of it
    uint32_t m_blocks, n_blocks, splits, slabs, seg_slabs, slabs_per_split;
    // LIN_GATED
    uint16_t* y;
    uint16_t* gate;      // NULL: not kept
    uint16_t* up;
    int64_t ldy, ldgate, ldup;
    int act;
    // LIN_LSE
    const int64_t* target;
    float2* part;        // [2 * n_blocks][M]: of half a tile's columns e and s with sum of exp(l) = 2^e s
    float* hit;          // [M]: the target's logit
    // LIN_DLOGITS
    const LossRow* row;
    uint16_t* dl;        // [M][lddl], whole tiles wide
    int64_t lddl;
    uint32_t first;      // the vocabulary's index of column 0
    // LIN_OUT: rows [0, half) of the product go to out, rows [half, 2 half) to out2,
    // each as far as out_rows; or every value to `sums`, a stretch of M * N per split
    uint16_t* out;
    uint16_t* out2;
    int64_t ldo, ldo2;
    uint32_t half, out_rows;
    float* sums;         // NULL: to out
    int add;             // to what sums holds
    const float* unscale;  // NULL: 1
};

template <int AL, int BL, int T>
struct LinTraits {
    static constexpr int BK = 64;
    static constexpr int WT = T / 2, F = WT / 16;     // a wave's share of either side, in values and in 16-wide blocks
    static constexpr int STAGE = T * BK * 2;          // bytes of one operand's slab
    static constexpr int ND = STAGE / 4096;           // DMAs of a wave per operand and slab
};

__device__ __forceinline__ float act_of(int act, float g) {
    if (act == 1) return g / (1.0f + __expf(-g));
    if (act == 2) return 0.5f * g * erfcf(-0.70710678f * g);
    const float z = 0.79788456f * (g + 0.044715f * g * g * g);
    return g / (1.0f + __expf(-2.0f * z));  // (1 + tanh z) / 2 is the logistic function of 2 z
}

// Two values -> one dword of two 16-bit values (low half = a), round to nearest even.
template <int DT>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    if constexpr (DT == DT_FP16) {
        typedef _Float16 h2 __attribute__((ext_vector_type(2)));
        return __builtin_bit_cast(uint32_t, h2{(_Float16)a, (_Float16)b});
    } else {
        typedef __bf16 b2 __attribute__((ext_vector_type(2)));
        return __builtin_bit_cast(uint32_t, b2{(__bf16)a, (__bf16)b});
    }
}

// 8 consecutive values of a row as 16-bit ones, as far as `count` of them exist.
template <int DT>
__device__ __forceinline__ void store8(uint16_t* to, const float* v, uint32_t count) {
    const u32x4 w = {pack2<DT>(v[0], v[1]), pack2<DT>(v[2], v[3]), pack2<DT>(v[4], v[5]), pack2<DT>(v[6], v[7])};
    if (count >= 8u) {
        *(u32x4_at2*)to = w;
    } else {
#pragma unroll
        for (uint32_t e = 0; e < 7u; ++e)
            if (e < count) to[e] = (uint16_t)(w[e / 2] >> (16 * (e % 2)));
    }
}

// Tile and range of slabs of one unit of work.
struct LinUnit {
    uint32_t split, m_idx, n_idx, slab0, slabs;
};
__device__ __forceinline__ LinUnit lin_unit(const LinArgs& args, uint32_t unit) {
    const uint32_t tiles = args.m_blocks * args.n_blocks;
    TileScheduler s;
    s.setup(tiles, args.m_blocks, args.n_blocks, 8u);
    LinUnit u;
    u.split = unit / tiles;
    s.coord(unit - u.split * tiles, u.m_idx, u.n_idx);
    u.slab0 = u.split * args.slabs_per_split;
    const uint32_t left = u.slab0 < args.slabs ? args.slabs - u.slab0 : 0u;
    u.slabs = left < args.slabs_per_split ? left : args.slabs_per_split;
    return u;
}

template <int DT, int AL, int BL, int EPI, int T>
__global__ __launch_bounds__(256, T == 256 ? 1 : 2) void linear_kernel(LinArgs args) {
    using TR = LinTraits<AL, BL, T>;
    constexpr int F = TR::F, ND = TR::ND, WT = TR::WT, BK = TR::BK;
    __shared__ __attribute__((aligned(1024))) uint8_t smem[2 * TR::STAGE];
    typedef __attribute__((address_space(3))) uint8_t lds_u8;
    typedef __attribute__((address_space(3))) u32x4 lds_u32x4;
    const uint32_t lds_base = (uint32_t)reinterpret_cast<uintptr_t>((lds_u8*)smem);
    const uint32_t lane = threadIdx.x & 63u, l16 = lane & 15u, lg = lane >> 4;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t wr = wave >> 1, wc = wave & 1u;

    const uint32_t units = args.m_blocks * args.n_blocks * args.splits;
    const LinUnit u = lin_unit(args, worker_of_workgroup(blockIdx.x, units, 8u, units));
    const uint32_t m0 = u.m_idx * T, n0 = u.n_idx * (EPI == LIN_GATED ? WT : T);  // a gated tile holds T/2 columns of each projection

    // ---- sources.  A wave fetches a quarter of a slab's rows: T/4 rows along the
    // sum, or 16 across it.  Its descriptor starts there and ends with the matrix.
    // Along the sum a lane fetches chunk (lane & 7) ^ (lane >> 3) of rows lane/8,
    // lane/8 + 8, ...; of B's rows, those that bring 8 consecutive columns of the
    // product to one lane: place 16 b + i of 32 holds row 8 (i / 4) + 4 b + i % 4.
    // A gated tile's rows alternate between the weights by waves. ----
    const uint32_t k_chunk = (lane & 7u) ^ (lane >> 3);
    const int64_t ldb = EPI == LIN_GATED && (wave & 1u) ? args.ldb2 : args.ldb;
    uint32_t voff_a[ND], voff_b[ND];
#pragma unroll
    for (int q = 0; q < ND; ++q) {
        if constexpr (AL == LIN_ALONG) {
            voff_a[q] = (8u * q + lane / 8u) * (uint32_t)args.lda * 2u + k_chunk * 16u;
        } else {
            const uint32_t p = (wave * ND + q) * 64u + lane, r = p / (T / 8);
            voff_a[q] = (r & 15u) * (uint32_t)args.lda * 2u + ((p % (T / 8)) ^ swz_b(r)) * 16u;
        }
        if constexpr (BL == LIN_ALONG) {
            const uint32_t p = 8u * q + lane / 8u;
            voff_b[q] = ((p & ~31u) + 8u * ((p >> 2) & 3u) + 4u * ((p >> 4) & 1u) + (p & 3u)) * (uint32_t)ldb * 2u + k_chunk * 16u;
        } else {
            const uint32_t p = (wave * ND + q) * 64u + lane, r = p / (T / 8);
            voff_b[q] = (r & 15u) * (uint32_t)ldb * 2u + ((p % (T / 8)) ^ swz_b(r)) * 16u;
        }
    }
    // one operand's descriptor for a slab that starts at k0: `first` row or column of the tile
    auto source = [&](auto along_c, const uint16_t* base, int64_t ld, uint32_t first, uint32_t end, uint32_t K, uint32_t k0) __attribute__((always_inline)) -> i32x4 {
        if constexpr (decltype(along_c)::value) {
            const uint32_t left = first < end ? end - first : 0u, rows = left < T / 4 ? left : T / 4;
            const uint32_t bytes = rows == 0u ? 0u : ((rows - 1u) * (uint32_t)ld + (K - k0)) * 2u;
            return rsrc_words_u64(reinterpret_cast<uint64_t>(base) + ((uint64_t)first * (uint64_t)ld + k0) * 2u, bytes);
        } else {
            const uint32_t k = k0 + wave * 16u, left = k < K ? K - k : 0u, rows = left < 16u ? left : 16u;
            const uint32_t bytes = rows == 0u ? 0u : ((rows - 1u) * (uint32_t)ld + (end - first)) * 2u;
            return rsrc_words_u64(reinterpret_cast<uint64_t>(base) + ((uint64_t)k * (uint64_t)ld + first) * 2u, bytes);
        }
    };
    using TRUE_ = std::integral_constant<bool, true>;
    using FALSE_ = std::integral_constant<bool, false>;
    auto fetch = [&](uint32_t slab) __attribute__((always_inline)) {
        const bool second = slab >= args.seg_slabs;
        const uint32_t k0 = (slab - (second ? args.seg_slabs : 0u)) * BK;
        i32x4 ra, rb;
        const uint16_t* a = EPI == LIN_OUT && second ? args.a2 : args.a;
        if constexpr (AL == LIN_ALONG) ra = source(TRUE_{}, a, args.lda, m0 + wave * (T / 4), args.M, args.Ka, k0);
        else ra = source(FALSE_{}, a, args.lda, m0, args.M, args.Ka, k0);
        if constexpr (EPI == LIN_GATED)
            rb = source(TRUE_{}, (wave & 1u) ? args.b2 : args.b, ldb, n0 + (wave >> 1) * (T / 4), args.N, args.Kb, k0);
        else if constexpr (BL == LIN_ALONG) rb = source(TRUE_{}, args.b, ldb, n0 + wave * (T / 4), args.N, args.Kb, k0);
        else rb = source(FALSE_{}, second ? args.b2 : args.b, second ? args.ldb2 : args.ldb, n0, args.N, args.Kb, k0);
        const uint32_t past = k0 + k_chunk * 8u >= args.Ka ? 0x80000000u : 0u;
        asm volatile("s_nop 4" ::: "memory");  // a vector write of a descriptor -> its use
        static_for<0, ND>([&](auto q_c) __attribute__((always_inline)) {
            constexpr int q = decltype(q_c)::value;
            dma16_at<q * 1024u>(lds_base + wave * ND * 1024u, AL == LIN_ALONG ? voff_a[q] | past : voff_a[q], ra);
        });
        static_for<0, ND>([&](auto q_c) __attribute__((always_inline)) {
            constexpr int q = decltype(q_c)::value;
            dma16_at<TR::STAGE + q * 1024u>(lds_base + wave * ND * 1024u, BL == LIN_ALONG ? voff_b[q] | past : voff_b[q], rb);
        });
    };

    // ---- fragments.  Across the sum the columns of two 16-wide blocks are
    // interleaved: block b's lane group g holds 8 g + 4 (b ^ (g & 1)) + 0..3 of 32,
    // so that one read's 16 lanes spread over the banks. ----
    i16x8 fa[F][2], fb[F][2];
    auto read = [&](auto along_c, uint32_t base, uint32_t side, int f, int k) __attribute__((always_inline)) -> i16x8 {
        if constexpr (decltype(along_c)::value) {
            const uint32_t at = base + (side * WT + 16u * f + l16) * 128u + (((uint32_t)k * 4u + lg) ^ (l16 & 7u)) * 16u;
            return __builtin_bit_cast(i16x8, *(const lds_u32x4*)(lds_u8*)(uintptr_t)at);
        } else {
            const uint32_t r = 8u * lg + (l16 >> 2);
            const uint32_t chunk = (side * WT + 32u * (f / 2)) / 8u + (l16 & 3u);
            const uint32_t at = base + r * (T * 2) + (chunk ^ swz_b(r)) * 16u + 8u * ((f & 1u) ^ (l16 & 1u)) + k * 32u * (T * 2);
            const i16x4 x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)(lds_u8*)(uintptr_t)at);
            const i16x4 y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)(lds_u8*)(uintptr_t)(at + 4u * (T * 2)));
            return __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7);
        }
    };

    f32x4 acc[F][F];
#pragma unroll
    for (int fm = 0; fm < F; ++fm)
#pragma unroll
        for (int fn = 0; fn < F; ++fn) {
            acc[fm][fn] = f32x4{0.f, 0.f, 0.f, 0.f};
            asm volatile("" : "+a"(acc[fm][fn]));
        }
    asm volatile("s_nop 1" ::: "memory");  // a vector write of a register -> an MFMA that reads it

    for (uint32_t s = 0; s < u.slabs; ++s) {
        lds_barrier();
        fetch(u.slab0 + s);
        wait_vm<0>();
        lds_barrier();
        static_for<0, 2>([&](auto k_c) __attribute__((always_inline)) {
            constexpr int k = decltype(k_c)::value;
#pragma unroll
            for (int f = 0; f < F; ++f) {
                fa[f][k] = read(std::integral_constant<bool, AL == LIN_ALONG>{}, lds_base, wr, f, k);
                fb[f][k] = read(std::integral_constant<bool, BL == LIN_ALONG>{}, lds_base + TR::STAGE, wc, f, k);
            }
            asm volatile("s_nop 1" ::: "memory");
#pragma unroll
            for (int fm = 0; fm < F; ++fm)
#pragma unroll
                for (int fn = 0; fn < F; ++fn) mfma16x16x32<DT>(acc[fm][fn], fb[fn][k], fa[fm][k]);
        });
    }
    gap_nops();
    wait_vm<0>();
#pragma unroll
    for (int fm = 0; fm < F; ++fm)
#pragma unroll
        for (int fn = 0; fn < F; ++fn) asm volatile("" : "+a"(acc[fm][fn]));  // not read before the gap above

    // ---- where a lane's values belong: of block fm one row, of the pair t of
    // column blocks 8 consecutive columns ----
    auto row_of = [&](int fm) __attribute__((always_inline)) -> uint32_t {
        if constexpr (AL == LIN_ALONG) return m0 + wr * WT + 16u * fm + l16;
        const uint32_t p = l16 >> 2;
        return m0 + wr * WT + 32u * (fm / 2) + 8u * p + 4u * ((fm & 1u) ^ (p & 1u)) + (l16 & 3u);
    };
    const bool swap = BL == LIN_ACROSS && (lg & 1u) != 0u;
    auto eight = [&](int fm, int t, float* v) __attribute__((always_inline)) {
        const f32x4 x = acc[fm][2 * t], y = acc[fm][2 * t + 1];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            v[e] = swap ? y[e] : x[e];
            v[4 + e] = swap ? x[e] : y[e];
        }
    };
    auto left = [](uint32_t at, uint32_t end) __attribute__((always_inline)) -> uint32_t { return at < end ? end - at : 0u; };

    if constexpr (EPI == LIN_GATED) {
#pragma unroll
        for (int fm = 0; fm < F; ++fm) {
            const uint32_t m = row_of(fm);
#pragma unroll
            for (int t = 0; t < F / 4; ++t) {
                float g[8], up[8], y[8];
                eight(fm, t, g);
                eight(fm, t + F / 4, up);
#pragma unroll
                for (int e = 0; e < 8; ++e) y[e] = act_of(args.act, g[e]) * up[e];
                const uint32_t n = n0 + wc * (WT / 2) + 32u * t + 8u * lg;
                const uint32_t count = m < args.M ? left(n, args.N) : 0u;
                if (count == 0u) continue;
                store8<DT>(args.y + (int64_t)m * args.ldy + n, y, count);
                if (args.gate) store8<DT>(args.gate + (int64_t)m * args.ldgate + n, g, count);
                if (args.up) store8<DT>(args.up + (int64_t)m * args.ldup + n, up, count);
            }
        }
    } else if constexpr (EPI == LIN_LSE) {
#pragma unroll
        for (int fm = 0; fm < F; ++fm) {
            const uint32_t m = row_of(fm);
            const int64_t target = m < args.M ? args.target[m] : -1;
            float v[F / 2][8], top = -__builtin_inff();
#pragma unroll
            for (int t = 0; t < F / 2; ++t) {
                eight(fm, t, v[t]);
                const uint32_t n = n0 + wc * WT + 32u * t + 8u * lg;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    if (n + e >= args.N) v[t][e] = -__builtin_inff();
                    else if (target == (int64_t)(n + e)) args.hit[m] = v[t][e];
                    top = fmaxf(top, v[t][e]);
                }
            }
            top = fmaxf(top, __shfl_xor(top, 16));
            top = fmaxf(top, __shfl_xor(top, 32));
            const float from = top == -__builtin_inff() ? 0.0f : top * kLog2e;  // the sum is in units of 2^from
            float sum = 0.0f;
#pragma unroll
            for (int t = 0; t < F / 2; ++t)
#pragma unroll
                for (int e = 0; e < 8; ++e) sum += __builtin_amdgcn_exp2f(__builtin_fmaf(v[t][e], kLog2e, -from));
            sum += __shfl_xor(sum, 16);
            sum += __shfl_xor(sum, 32);
            if (lg == 0u && m < args.M) args.part[(size_t)(u.n_idx * 2u + wc) * args.M + m] = make_float2(top == -__builtin_inff() ? top : from, sum);
        }
    } else if constexpr (EPI == LIN_DLOGITS) {
#pragma unroll
        for (int fm = 0; fm < F; ++fm) {
            const uint32_t m = row_of(fm);
            if (m >= args.M) continue;
            const LossRow r = args.row[m];
#pragma unroll
            for (int t = 0; t < F / 2; ++t) {
                float v[8];
                eight(fm, t, v);
                const uint32_t n = n0 + wc * WT + 32u * t + 8u * lg;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float p = __builtin_amdgcn_exp2f(__builtin_fmaf(v[e], kLog2e, -r.lse2));
                    const bool is = r.target == (int32_t)(args.first + n + e);
                    v[e] = r.target < 0 || n + e >= args.N ? 0.0f : r.d * (is ? p - 1.0f : p);
                }
                store8<DT>(args.dl + (int64_t)m * args.lddl + n, v, 8u);
            }
        }
    } else {
        const float scale = args.unscale ? *args.unscale : 1.0f;
#pragma unroll
        for (int fm = 0; fm < F; ++fm) {
            const uint32_t m = row_of(fm);
            const bool upper = m >= args.half;
            const uint32_t mo = upper ? m - args.half : m;
            if (m >= args.M || mo >= args.out_rows) continue;
#pragma unroll
            for (int t = 0; t < F / 2; ++t) {
                float v[8];
                eight(fm, t, v);
                const uint32_t n = n0 + wc * WT + 32u * t + 8u * lg;
                if (n >= args.N) continue;  // N is a multiple of 8
                if (args.sums) {
                    float* to = args.sums + ((size_t)u.split * args.M + m) * args.N + n;
                    f32x4 x = {v[0], v[1], v[2], v[3]}, y = {v[4], v[5], v[6], v[7]};
                    if (args.add) {
                        x += *(const f32x4*)to;
                        y += *(const f32x4*)(to + 4);
                    }
                    *(f32x4*)to = x;
                    *(f32x4*)(to + 4) = y;
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[e] *= scale;
                    store8<DT>((upper ? args.out2 + (int64_t)mo * args.ldo2 : args.out + (int64_t)mo * args.ldo) + n, v, 8u);
                }
            }
        }
    }
}

}  // namespace tsg
