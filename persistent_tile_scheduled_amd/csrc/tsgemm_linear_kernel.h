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
//
// Workgroups are persistent: the loader runs two slabs ahead and on into the next
// tile, so that its first slabs arrive during the epilogue.  Measured bf16, T = 256, in
// cycles a slab (its 128 MFMAs take 2048) and of the epilogue: logsumexp 2200 and 12680,
// gated 2220 and 10010 (three outputs 2240 and 21000), dx 2220 and 8320, dW 2490 to 2690 and
// 8570.  8192 x 4096 x 131072, over several cards: loss 5.54 to 5.98 ms, 1588 to 1470 TFLOP/s,
// gradient 17.9 to 19.1 ms, 1478 to 1380; gated 8192 x 4096 x 16384 with both projections
// kept 1.53 to 1.57 ms, 1436 to 1403, gradient 3.30 to 3.37 ms, 1332 to 1304 (the library's
// plain product of 8192^3 1635, 1393 with b across the sum, 1217 with both): bound by the
// board's power.
#pragma once

#include "tile_scheduler.h"
#include "tsgemm_device.h"

namespace tsg {

typedef uint32_t u32x4_at2 __attribute__((ext_vector_type(4), aligned(2)));  // 16 bytes at a 2-byte boundary

constexpr float kLog2e = 1.44269504f;

// exp(v - from).  The difference comes first: v log2 e - from log2 e in one fma, an
// instruction less, carries the rounding of the second term, which past logits of 3e9 is
// more than an exponential has room for (8192 x 4096 x 131072 bf16 loss 5953 us, so 5984).
__device__ __forceinline__ float exp_past(float v, float from) { return __builtin_amdgcn_exp2f((v - from) * kLog2e); }

enum { LIN_ALONG = 0, LIN_ACROSS = 1 };  // an operand's layout: the sum's index fastest, or slowest
enum { LIN_GATED = 0, LIN_LSE = 1, LIN_DLOGITS = 2, LIN_OUT = 3 };

// What the cross entropy's gradient needs of a row.
struct LossRow {
    float lse;       // its logsumexp
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
    int aligned;         // rows of y, gate and up begin at multiples of 16 bytes
    // LIN_LSE
    const int64_t* target;
    float2* part;        // [2 * n_blocks][M]: of half a tile's columns t and s with sum of exp(l) = exp(t) s
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

template <int T>
struct LinTraits {
    static constexpr int BK = 64;
    static constexpr int WT = T / 2, F = WT / 16;     // a wave's share of either side, in values and in 16-wide blocks
    static constexpr int STAGE = T * BK * 2;          // bytes of one operand's slab
    static constexpr int ND = STAGE / 4096;           // DMAs of a wave per operand and slab
};

// Race-detection build (TSG_STRESS): a pause of 0 to ~2048 cycles of which every
// wave draws its own sequence; one asm block, since code that the compiler sees
// would take the registers that the accumulators need.  The count only falls, so
// the loop ends.
__device__ __forceinline__ uint32_t pause_seed(uint32_t wave) { return (blockIdx.x * 4u + wave + 1u) * 0x9E3779B1u; }
__device__ __forceinline__ void lin_pause(uint32_t& state) {
#if TSG_STRESS
    uint32_t count;  // 0, 0, 0, 1, 2, 4, 8 or 16 times 128 cycles
    asm volatile(
        "s_mul_i32 %0, %0, 0x19660d\n\ts_add_u32 %0, %0, 0x3c6ef35f\n\t"
        "s_lshr_b32 %1, %0, 29\n\ts_lshl_b32 %1, 1, %1\n\ts_lshr_b32 %1, %1, 3\n"
        ".Lpause%=:\n\ts_cmp_eq_u32 %1, 0\n\ts_cbranch_scc1 .Lon%=\n\ts_sleep 2\n\ts_sub_u32 %1, %1, 1\n\t"
        "s_branch .Lpause%=\n.Lon%=:"
        : "+s"(state), "=&s"(count)::"scc", "memory");
#else
    (void)state;
#endif
}

// The activations are g p(g), with p the logistic function of z = g (c + k g^2)
// (silu: c = 1, k = 0; gelu by tanh: (1 + tanh(z / 2)) / 2 is the logistic function of
// z) or, BELL, the normal distribution function (gelu).  Both without a branch: an
// accumulator that lives across one is copied.  g^2 ends at 1e30, where z has long
// run past every exponential: past fp32's end it would make silu's k g^2 0 * inf.
struct Act {
    float c, k;  // times log2 e
    __device__ __forceinline__ explicit Act(int act)
        : c(act == 1 ? kLog2e : 1.5957691f * kLog2e), k(act == 1 ? 0.0f : 1.5957691f * 0.044715f * kLog2e) {}
};
constexpr int kActBell = 2;  // TSGEMM_GELU

// The normal distribution function below -a, over exp(-a^2 / 2), a >= 0: a polynomial
// in 1 / (1 + 0.3 a) fitted by least squares to the relative error, which is below
// 4.3e-7 in fp32 for a up to 14, where exp(-a^2 / 2) ends.
__device__ __forceinline__ float tail_over_bell(float a) {
    const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.3f, a, 1.0f));
    float h = 0.03622337058186531f;
    h = __builtin_fmaf(h, t, -0.1593545526266098f);
    h = __builtin_fmaf(h, t, 0.20981964468955994f);
    h = __builtin_fmaf(h, t, -0.05664501339197159f);
    h = __builtin_fmaf(h, t, 0.13000500202178955f);
    h = __builtin_fmaf(h, t, 0.09951350837945938f);
    h = __builtin_fmaf(h, t, 0.12081217765808105f);
    h = __builtin_fmaf(h, t, 0.11962586641311646f);
    return h * t;
}
__device__ __forceinline__ float act_square(float g) { return fminf(g * g, 1e30f); }
// p(g); `bell` receives exp(-g^2 / 2) (BELL)
template <bool BELL>
__device__ __forceinline__ float act_share(const Act& k, float g, float& bell) {
    if constexpr (BELL) {
        bell = __builtin_amdgcn_exp2f(g * g * (-0.5f * kLog2e));
        const float tail = bell * tail_over_bell(fabsf(g));
        return g < 0.0f ? tail : 1.0f - tail;
    } else {
        return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-g * __builtin_fmaf(k.k, act_square(g), k.c)));
    }
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

// 8 consecutive values of a row as 16-bit ones: all of them, or as far as `count` of
// them exist.
template <int DT>
__device__ __forceinline__ u32x4 pack8(const float* v) {
    return u32x4{pack2<DT>(v[0], v[1]), pack2<DT>(v[2], v[3]), pack2<DT>(v[4], v[5]), pack2<DT>(v[6], v[7])};
}
__device__ __forceinline__ void store_some(uint16_t* to, u32x4 w, uint32_t count) {
    if (count >= 8u) {
        *(u32x4_at2*)to = w;
    } else {
#pragma unroll
        for (uint32_t e = 0; e < 7u; ++e)
            if (e < count) to[e] = (uint16_t)(w[e / 2] >> (16 * (e % 2)));
    }
}
template <int DT>
__device__ __forceinline__ void store8(uint16_t* to, const float* v, uint32_t count) {
    store_some(to, pack8<DT>(v), count);
}

// The largest value and the sum over the four lanes that hold a row's columns.
__device__ __forceinline__ float max_over_groups(float x) {
    const float y = fmaxf(x, __shfl_xor(x, 16));
    return fmaxf(y, __shfl_xor(y, 32));
}
__device__ __forceinline__ float sum_over_groups(float x) {
    const float y = x + __shfl_xor(x, 16);
    return y + __shfl_xor(y, 32);
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

// The reads of a phase by gaps: gap s holds reads first[s] ... first[s + 1] - 1.
template <int STEPS>
struct LinReads {
    int first[STEPS + 1];
};
// `per` reads a gap, `lead` reads of the operand that is needed first from gap `start` on,
// then `rest` of the other: `space` gaps apart (0: as they come), or, `row_reads` != 0, each
// `row_reads` of them once their row of `row_steps` MFMAs is used up.
template <int STEPS>
constexpr LinReads<STEPS> lin_reads(int per, int lead, int rest, int start, int space, int row_reads, int row_steps) {
    LinReads<STEPS> t = {};
    int gap = start, count = 0, at = 0;
    for (int i = 0; i < lead + rest; ++i) {
        int from = start;
        if (i >= lead && space != 0) from = start + (lead + per - 1) / per + (i - lead) * space / per;
        if (i >= lead && row_reads != 0) from = (i - lead) / row_reads * row_steps + row_steps - 1 + kGap;
        if (gap < from) {
            gap = from;
            count = 0;
        }
        if (count == per) {
            ++gap;
            count = 0;
        }
        if (gap >= STEPS) break;
        while (at <= gap) t.first[at++] = i;
        ++count;
        if (at <= STEPS) t.first[at] = i + 1;
    }
    const int all = t.first[at <= STEPS ? at : STEPS];
    while (at <= STEPS) t.first[at++] = all;
    return t;
}

// acc = a * b, in the registers that acc is in: with an output of its own the
// accumulator of a tile's first slab could be another register than that of the
// others, and the copies between them would lie right beside MFMAs that the compiler
// does not see.
template <int DT>
__device__ __forceinline__ void mfma_first(f32x4& acc, i16x8 a, i16x8 b) {
    if constexpr (DT == DT_FP16)
        asm volatile("v_mfma_f32_16x16x32_f16 %0, %1, %2, 0" : "+a"(acc) : "v"(a), "v"(b));
    else
        asm volatile("v_mfma_f32_16x16x32_bf16 %0, %1, %2, 0" : "+a"(acc) : "v"(a), "v"(b));
}

template <int DT, int AL, int BL, int EPI, int T>
__global__ __launch_bounds__(256, T == 256 ? 1 : 2) void linear_kernel(LinArgs args) {
    using TR = LinTraits<T>;
    constexpr int F = TR::F, ND = TR::ND, NL = 2 * ND, WT = TR::WT, BK = TR::BK, STAGE = TR::STAGE;
    constexpr bool A_ALONG = AL == LIN_ALONG, B_ALONG = BL == LIN_ALONG;
    __shared__ __attribute__((aligned(1024))) uint8_t smem[4 * STAGE];  // stage 0: A, B; stage 1: A, B
    typedef __attribute__((address_space(3))) uint8_t lds_u8;
    typedef __attribute__((address_space(3))) u32x4 lds_u32x4;
    const uint32_t lds_base = (uint32_t)reinterpret_cast<uintptr_t>((lds_u8*)smem);
    const uint32_t lane = threadIdx.x & 63u, l16 = lane & 15u, lg = lane >> 4;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t wr = wave >> 1, wc = wave & 1u;
    uint32_t pauses = pause_seed(wave);  // race-detection build only
    auto pause = [&]() __attribute__((always_inline)) { lin_pause(pauses); };

    // ---- sources.  A wave fetches a quarter of a slab's rows: T/4 rows along the
    // sum, or 16 across it.  Its descriptor starts there and ends with the matrix.
    // Along the sum a lane fetches chunk (lane & 7) ^ (lane >> 3) of rows lane/8,
    // lane/8 + 8, ...; of B's rows, those that bring 8 consecutive columns of the
    // product to one lane: place 16 b + i of 32 holds row 8 (i / 4) + 4 b + i % 4.
    // A gated tile's rows alternate between the weights by waves. ----
    const uint32_t k_chunk = (lane & 7u) ^ (lane >> 3);
    const uint32_t lda = (uint32_t)args.lda, ldb = (uint32_t)(EPI == LIN_GATED && (wave & 1u) ? args.ldb2 : args.ldb);
    uint32_t voff[NL];
#pragma unroll
    for (int q = 0; q < ND; ++q) {
        const uint32_t along = 8u * q + lane / 8u;
        const uint32_t at = (wave * ND + q) * 64u + lane, across = at / (T / 8), chunk = (at % (T / 8)) ^ swz_b(across);
        voff[q] = A_ALONG ? along * lda * 2u + k_chunk * 16u : (across & 15u) * lda * 2u + chunk * 16u;
        voff[ND + q] = B_ALONG ? ((along & ~31u) + 8u * ((along >> 2) & 3u) + 4u * ((along >> 4) & 1u) + (along & 3u)) * ldb * 2u + k_chunk * 16u
                               : (across & 15u) * ldb * 2u + chunk * 16u;
    }
    // one operand's descriptor for a slab that starts at k0; `first`: the tile's row or column
    auto source = [&](auto along_c, const uint16_t* base, int64_t ld, uint32_t first, uint32_t end, uint32_t K, uint32_t k0,
                      uint32_t& dec) __attribute__((always_inline)) -> i32x4 {
        if constexpr (decltype(along_c)::value) {
            const uint32_t left = first < end ? end - first : 0u, rows = left < T / 4 ? left : T / 4;
            const uint32_t bytes = rows == 0u ? 0u : ((rows - 1u) * (uint32_t)ld + (K - k0)) * 2u;
            dec = rows == 0u ? 0u : BK * 2u;
            return rsrc_words_u64(reinterpret_cast<uint64_t>(base) + ((uint64_t)first * (uint64_t)ld + k0) * 2u, bytes);
        } else {
            const uint32_t k = k0 + wave * 16u, left = k < K ? K - k : 0u, rows = left < 16u ? left : 16u;
            const uint32_t bytes = rows == 0u ? 0u : ((rows - 1u) * (uint32_t)ld + (end - first)) * 2u;
            dec = 0u;
            return rsrc_words_u64(reinterpret_cast<uint64_t>(base) + ((uint64_t)k * (uint64_t)ld + first) * 2u, bytes);
        }
    };

    // ---- loader: its own walk over the workgroup's units, two slabs ahead of the
    // MFMAs and on to the next unit's.  From slab to slab it steps the descriptors;
    // at an event (the sum's second half, its last slab when that is not whole, the
    // next unit) it forms them anew.  Past the last unit nothing is covered: the DMAs
    // then write zeros that nobody reads, so that every slab issues the same. ----
    const uint32_t units = args.m_blocks * args.n_blocks * args.splits, workers = gridDim.x;
    const uint32_t first_unit = worker_of_workgroup(blockIdx.x, workers, 8u, workers);
    uint32_t ld_unit = first_unit, ld_slab = 0, ld_end = 0, ld_event = 0, ld_m = 0, ld_n = 0;
    uint32_t a_dec = 0, b_dec = 0;
    const uint64_t a_step = A_ALONG ? BK * 2u : (uint64_t)BK * lda * 2u;
    uint64_t b_step = B_ALONG ? BK * 2u : (uint64_t)BK * ldb * 2u;
    i32x4 ra, rb;
    auto seek = [&]() __attribute__((always_inline)) {
        if (ld_slab == ld_end && ld_unit < units) {
            const LinUnit u = lin_unit(args, ld_unit);
            ld_unit += workers;
            ld_slab = u.slab0;
            ld_end = u.slab0 + u.slabs;
            ld_m = u.m_idx * T;
            ld_n = u.n_idx * (EPI == LIN_GATED ? WT : T);
        }
        const bool live = ld_slab != ld_end, second = EPI == LIN_OUT && ld_slab >= args.seg_slabs;
        const uint32_t seg = second ? args.seg_slabs : 0u, k0 = (ld_slab - seg) * BK;
        ra = source(std::integral_constant<bool, A_ALONG>{}, second ? args.a2 : args.a, args.lda, A_ALONG ? ld_m + wave * (T / 4) : ld_m,
                    args.M, args.Ka, k0, a_dec);
        if constexpr (EPI == LIN_GATED)
            rb = source(std::integral_constant<bool, true>{}, (wave & 1u) ? args.b2 : args.b, ldb, ld_n + (wave >> 1) * (T / 4), args.N, args.Kb, k0, b_dec);
        else
            rb = source(std::integral_constant<bool, B_ALONG>{}, second ? args.b2 : args.b, second ? args.ldb2 : args.ldb,
                        B_ALONG ? ld_n + wave * (T / 4) : ld_n, args.N, args.Kb, k0, b_dec);
        const uint32_t K = args.Ka < args.Kb ? args.Ka : args.Kb;
        const uint32_t whole = K / BK, run = seg + (k0 / BK < whole ? whole : k0 / BK + 1u);
        ld_event = run < ld_end ? run : ld_end;
        if (!live) {
            ra.z = rb.z = 0;
            a_dec = b_dec = 0u;
            ld_event = 0xFFFFFFFFu;
        }
        if constexpr (EPI == LIN_OUT && A_ALONG) {  // the halves' weights may lie differently
            const uint32_t ld = second ? (uint32_t)args.ldb2 : (uint32_t)args.ldb;
            b_step = (uint64_t)BK * ld * 2u;
#pragma unroll
            for (int q = 0; q < ND; ++q) {
                const uint32_t at = (wave * ND + q) * 64u + lane, across = at / (T / 8);
                voff[ND + q] = (across & 15u) * ld * 2u + ((at % (T / 8)) ^ swz_b(across)) * 16u;
            }
        }
        if constexpr (A_ALONG || B_ALONG) {
            const uint32_t past = k0 + k_chunk * 8u >= K ? 0x80000000u : 0u;
#pragma unroll
            for (int q = 0; q < NL; ++q)
                if (q < ND ? A_ALONG : B_ALONG) voff[q] = (voff[q] & 0x7FFFFFFFu) | past;
        }
        asm volatile("s_nop 4" : "+s"(ra), "+s"(rb)::"memory");  // a vector write of a descriptor -> its use
    };
    const uint32_t dma_first = lds_base + wave * ND * 1024u;
    uint32_t dma_lds = dma_first;
    auto add64 = [](i32x4& r, uint64_t d) __attribute__((always_inline)) {
        const uint64_t a = (((uint64_t)(uint32_t)r.y) << 32 | (uint32_t)r.x) + d;  // stride bits are 0
        r.x = (int)(uint32_t)a;
        r.y = (int)(uint32_t)(a >> 32);
    };
    // One step in four pieces, for four gaps between MFMAs; each is pinned there by
    // the empty asm around it.
    constexpr int PIECES = 4;
    auto step = [&](auto p_c) __attribute__((always_inline)) {
        constexpr int p = decltype(p_c)::value;
        if constexpr (p == 0) {
            asm volatile("" : "+s"(ra));
            add64(ra, a_step);
            if constexpr (A_ALONG) ra.z -= (int)a_dec;
            asm volatile("" : "+s"(ra));
        } else if constexpr (p == 1) {
            asm volatile("" : "+s"(rb));
            add64(rb, b_step);
            if constexpr (B_ALONG) rb.z -= (int)b_dec;
            asm volatile("" : "+s"(rb));
        } else if constexpr (p == 2) {
            asm volatile("" : "+s"(dma_lds));
            dma_lds = dma_lds == dma_first ? dma_first + 2 * STAGE : dma_first;
            asm volatile("" : "+s"(dma_lds));
        } else {
            asm volatile("" : "+s"(ld_slab));
            if (__builtin_expect(++ld_slab == ld_event, 0)) seek();
            asm volatile("" : "+s"(ld_slab), "+s"(ra), "+s"(rb));
        }
    };
    // M0 for a DMA is written a gap before it
    auto m0_op = [&](auto q_c) __attribute__((always_inline)) {
        constexpr int q = decltype(q_c)::value;
        set_m0<q < ND ? q * 1024u : (uint32_t)STAGE + (q - ND) * 1024u>(dma_lds);
    };
    auto dma_op = [&](auto q_c) __attribute__((always_inline)) {
        constexpr int q = decltype(q_c)::value;
        pause();
        if constexpr (q < ND) dma16_m0(voff[q], ra);
        else dma16_m0(voff[q], rb);
    };
    auto dma_now = [&](auto q_c) __attribute__((always_inline)) {
        constexpr int q = decltype(q_c)::value;
        if constexpr (q < ND) dma16_at<q * 1024u>(dma_lds, voff[q], ra);
        else dma16_at<(uint32_t)STAGE + (q - ND) * 1024u>(dma_lds, voff[q], rb);
    };

    // ---- fragments.  Across the sum the columns of two 16-wide blocks are
    // interleaved: block b's lane group g holds 8 g + 4 (b ^ (g & 1)) + 0..3 of 32,
    // so that one read's 16 lanes spread over the banks. ----
    constexpr int AA = A_ALONG ? 2 : F, AB = B_ALONG ? 2 : F;  // address registers: per k-step, or per block
    uint32_t a_off[AA], b_off[AB], a_at[AA], b_at[AB];
    auto offset = [&](bool along, uint32_t side, uint32_t i) __attribute__((always_inline)) -> uint32_t {
        if (along) return (side * WT + l16) * 128u + ((i * 4u + lg) ^ (l16 & 7u)) * 16u;
        const uint32_t r = 8u * lg + (l16 >> 2), chunk = (side * WT + 32u * (i / 2)) / 8u + (l16 & 3u);
        return r * (T * 2) + (chunk ^ swz_b(r)) * 16u + 8u * ((i & 1u) ^ (l16 & 1u));
    };
#pragma unroll
    for (int i = 0; i < AA; ++i) a_off[i] = lds_base + offset(A_ALONG, wr, i);
#pragma unroll
    for (int i = 0; i < AB; ++i) b_off[i] = lds_base + STAGE + offset(B_ALONG, wc, i);
    i16x4 fa[F][2][2], fb[F][2][2];  // [block][k-step][half]
    // LDS read i of those of half a side's blocks, both k-steps: 16 bytes a lane along
    // the sum, 8 across it
    constexpr int RA = A_ALONG ? F : 2 * F, RB = B_ALONG ? F : 2 * F;
    auto read = [&](auto along_c, i16x4 (&to)[F][2][2], const uint32_t* at, auto half_c, auto i_c) __attribute__((always_inline)) {
        constexpr bool ALONG = decltype(along_c)::value;
        constexpr int i = decltype(i_c)::value, f = decltype(half_c)::value * F / 2 + (ALONG ? i / 2 : i / 4), k = (ALONG ? i : i / 2) % 2;
        if constexpr (ALONG) {
            const i16x8 v = __builtin_bit_cast(i16x8, *(const lds_u32x4*)((lds_u8*)(uintptr_t)at[k] + f * 2048));
            to[f][k][0] = __builtin_shufflevector(v, v, 0, 1, 2, 3);
            to[f][k][1] = __builtin_shufflevector(v, v, 4, 5, 6, 7);
        } else {
            to[f][k][i % 2] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)((lds_u8*)(uintptr_t)at[f] + (k * 32 + i % 2 * 4) * (T * 2)));
        }
    };
    auto read_a = [&](auto half_c, auto i_c) __attribute__((always_inline)) { read(std::integral_constant<bool, A_ALONG>{}, fa, a_at, half_c, i_c); };
    auto read_b = [&](auto half_c, auto i_c) __attribute__((always_inline)) { read(std::integral_constant<bool, B_ALONG>{}, fb, b_at, half_c, i_c); };
    auto address = [&](auto i_c, uint32_t stage) __attribute__((always_inline)) {
        constexpr int i = decltype(i_c)::value;
        if constexpr (i < AB) b_at[i] = b_off[i] + stage;
        else a_at[i - AB] = a_off[i - AB] + stage;
    };

    // ---- a slab in two phases of F * F MFMAs.  Every pair of MFMAs adds the slab's two
    // k-steps to one accumulator, the second taking it from the matrix core's
    // forwarding path.  Phase 1 goes over the column blocks' first half, phase 2 over
    // the second, rows of blocks in order in both, so that the fragments of both
    // k-steps fit the registers:
    //   phase 1 reads this slab's second halves of A and B while it uses the first;
    //   phase 2 waits for the next slab and passes the workgroup's barrier, reads the
    //   next slab's first half of B, and of A each row of blocks once it is used up, and
    //   refills the stage that phase 1 read out (the last DMAs go out in phase 1).
    // No register is refilled within kGap MFMAs of its last use: an MFMA may still be
    // fetching it. ----
    f32x4 acc[F][F];
#pragma unroll
    for (int fm = 0; fm < F; ++fm)
#pragma unroll
        for (int fn = 0; fn < F; ++fn) asm volatile("" : "=a"(acc[fm][fn]));
    constexpr int STEPS = F * F, START = kGap > 2 ? kGap : 2;
    constexpr int SPACE = T == 256 ? 4 : 1;                                   // MFMAs between DMAs
    constexpr int DF = START + (NL - 1) * SPACE < STEPS ? NL : (STEPS - START + SPACE - 1) / SPACE;  // DMAs of phase 2
    constexpr int LATE = DF < NL ? START + (NL - 1 - DF) * SPACE + 1 : 0;     // phase 1: gap after its DMAs
    constexpr int STEP_AT = DF < NL ? LATE : START + (DF - 1) * SPACE + 1;    // the loader's step, in phase 1 or 2
    static_assert(STEP_AT + PIECES <= STEPS, "the loader's step needs gaps");
    // Which LDS reads of a phase go into which gap, in order: one a gap (T = 256; the four
    // waves' reads of 8 bytes a lane fill the LDS's time of one MFMA) or two, and none before
    // what it overwrites is used up.
    using Reads = LinReads<STEPS>;
    constexpr Reads reads1 = lin_reads<STEPS>(T == 256 ? 1 : 2, RA, RB, START, T == 256 ? 2 : 1, 0, 0);
    constexpr Reads reads2 = lin_reads<STEPS>(T == 256 ? 1 : 2, RB, RA, START, 0, 2 * RA / F, F);
    static_assert(reads1.first[STEPS] == RA + RB && reads2.first[STEPS] == RA + RB, "every read needs a gap");
    using I0 = std::integral_constant<int, 0>;
    using I1 = std::integral_constant<int, 1>;
    using TRUE_ = std::integral_constant<bool, true>;
    using FALSE_ = std::integral_constant<bool, false>;
    uint32_t stage = 0;  // of the slab at hand: 0 or 2 * STAGE
    auto phase = [&](auto second_c, auto clear_c) __attribute__((always_inline)) {
        constexpr bool SECOND = decltype(second_c)::value, CLEAR = decltype(clear_c)::value;
        static_for<0, STEPS>([&](auto s_c) __attribute__((always_inline)) {
            constexpr int s = decltype(s_c)::value, k = s % 2;
            constexpr int fm = s / F, j = (s % F) / 2, fn = (SECOND ? F / 2 : 0) + ((fm & 1) ? F / 2 - 1 - j : j);
            const i16x8 av = __builtin_shufflevector(fa[fm][k][0], fa[fm][k][1], 0, 1, 2, 3, 4, 5, 6, 7);
            const i16x8 bv = __builtin_shufflevector(fb[fn][k][0], fb[fn][k][1], 0, 1, 2, 3, 4, 5, 6, 7);
            if constexpr (CLEAR && k == 0) mfma_first<DT>(acc[fm][fn], bv, av);
            else mfma16x16x32<DT>(acc[fm][fn], bv, av);
            if constexpr (SECOND && s == 1) {
                pause();
                wait_vm<0>();   // the next slab has landed
                lds_barrier();  // ... for every wave, and this one is read out
                pause();
                stage = stage == 0u ? 2u * STAGE : 0u;
            }
            if constexpr (SECOND && s >= 2 && s < 4)  // the next slab's addresses
                static_for<(AA + AB) * (s - 2) / 2, (AA + AB) * (s - 1) / 2>([&](auto i_c) __attribute__((always_inline)) { address(i_c, stage); });
            if constexpr (s >= START) {
                constexpr int i = s - START;
                if constexpr (SECOND ? i % SPACE == 0 && i / SPACE < DF : i % SPACE == 0 && i / SPACE < NL - DF)
                    dma_op(std::integral_constant<int, (SECOND ? 0 : DF) + i / SPACE>{});
                static_for<SECOND ? reads2.first[s] : reads1.first[s], SECOND ? reads2.first[s + 1] : reads1.first[s + 1]>(
                    [&](auto r_c) __attribute__((always_inline)) {
                        constexpr int r = decltype(r_c)::value;
                        if constexpr (SECOND && r < RB) read_b(I0{}, r_c);
                        else if constexpr (SECOND) read_a(I0{}, std::integral_constant<int, r - RB>{});
                        else if constexpr (r < RA) read_a(I1{}, r_c);
                        else read_b(I1{}, std::integral_constant<int, r - RA>{});
                    });
            }
            if constexpr (SECOND == (DF == NL) && s >= STEP_AT && s < STEP_AT + PIECES) step(std::integral_constant<int, s - STEP_AT>{});
            if constexpr (s + 1 >= START) {
                constexpr int i = s + 1 - START;
                if constexpr (s + 1 < STEPS && i % SPACE == 0 && i / SPACE < (SECOND ? DF : NL - DF))
                    m0_op(std::integral_constant<int, (SECOND ? 0 : DF) + i / SPACE>{});
            }
            __builtin_amdgcn_sched_barrier(0);
        });
    };

    // two slabs on their way (of the second what phase 2 would have issued), the first one's first halves read
    auto advance = [&]() __attribute__((always_inline)) {
        static_for<0, PIECES>([&](auto p_c) __attribute__((always_inline)) { step(p_c); });
    };
    seek();
    static_for<0, NL>([&](auto q_c) __attribute__((always_inline)) { dma_now(q_c); });
    advance();
    static_for<0, DF>([&](auto q_c) __attribute__((always_inline)) { dma_now(q_c); });
    if constexpr (DF == NL) advance();
    pause();
    wait_vm<DF>();
    lds_barrier();
    pause();
    static_for<0, AA + AB>([&](auto i_c) __attribute__((always_inline)) { address(i_c, 0u); });
    static_for<0, RB>([&](auto i_c) __attribute__((always_inline)) { read_b(I0{}, i_c); });
    static_for<0, RA>([&](auto i_c) __attribute__((always_inline)) { read_a(I0{}, i_c); });

    for (uint32_t unit = first_unit; unit < units; unit += workers) {
    const LinUnit u = lin_unit(args, unit);
    const uint32_t m0 = u.m_idx * T, n0 = u.n_idx * (EPI == LIN_GATED ? WT : T);  // a gated tile holds T/2 columns of each projection
    // what the epilogue needs of the tile's rows is on its way while the products are formed
    int64_t row_target[EPI == LIN_LSE ? F : 1];
    LossRow row_info[EPI == LIN_DLOGITS ? F : 1];
    if constexpr (EPI == LIN_LSE || EPI == LIN_DLOGITS) {
#pragma unroll
        for (int fm = 0; fm < F; ++fm) {
            const uint32_t m = m0 + wr * WT + 16u * fm + l16, at = m < args.M ? m : args.M - 1u;
            if constexpr (EPI == LIN_LSE) row_target[fm] = args.target[at];
            else row_info[fm] = args.row[at];
        }
    }
    phase(FALSE_{}, TRUE_{});
    phase(TRUE_{}, TRUE_{});
    for (uint32_t s = 1; s < u.slabs; ++s) {
        phase(FALSE_{}, FALSE_{});
        phase(TRUE_{}, FALSE_{});
    }
    gap_nops();  // the last MFMAs have written their accumulators

    // ---- where a lane's values belong: of block fm one row, of the pair t of
    // column blocks 8 consecutive columns ----
    auto row_of = [&](int fm) __attribute__((always_inline)) -> uint32_t {
        if constexpr (AL == LIN_ALONG) return m0 + wr * WT + 16u * fm + l16;
        const uint32_t p = l16 >> 2;
        return m0 + wr * WT + 32u * (fm / 2) + 8u * p + 4u * ((fm & 1u) ^ (p & 1u)) + (l16 & 3u);
    };
    const bool swap = BL == LIN_ACROSS && (lg & 1u) != 0u;
    // Read in asm, where the values are used: read all at once, as the compiler would,
    // they do not fit the registers beside the fragments of the next tile.
    auto four = [&](const f32x4& from, float* v) __attribute__((always_inline)) {
#pragma unroll
        for (int e = 0; e < 4; ++e) asm volatile("v_accvgpr_read_b32 %0, %1" : "=v"(v[e]) : "a"(from[e]));
    };
    auto eight = [&](int fm, int t, float* v) __attribute__((always_inline)) {
        float x[4], y[4];
        four(acc[fm][2 * t], x);
        four(acc[fm][2 * t + 1], y);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            v[e] = swap ? y[e] : x[e];
            v[4 + e] = swap ? x[e] : y[e];
        }
    };
    auto left = [](uint32_t at, uint32_t end) __attribute__((always_inline)) -> uint32_t { return at < end ? end - at : 0u; };

    // Every epilogue comes in two copies: for a tile that lies inside the matrix, with
    // nothing to ask, and for one that does not.
    const bool inside = m0 + T <= args.M && n0 + (EPI == LIN_GATED ? WT : T) <= args.N && (EPI != LIN_GATED || args.aligned);

    if constexpr (EPI == LIN_GATED) {
        const Act act(args.act);
        auto gated = [&](auto bell_c, auto inside_c) __attribute__((always_inline)) {
            constexpr bool BELL = decltype(bell_c)::value, INSIDE = decltype(inside_c)::value;
#pragma unroll
            for (int fm = 0; fm < F; ++fm) {
                const uint32_t m = row_of(fm), n = n0 + wc * (WT / 2) + 8u * lg;
                uint16_t* const y_at = args.y + (int64_t)m * args.ldy + n;
                uint16_t* const gate_at = args.gate + (int64_t)m * args.ldgate + n;
                uint16_t* const up_at = args.up + (int64_t)m * args.ldup + n;
#pragma unroll
                for (int t = 0; t < F / 4; ++t) {
                    float g[8], up[8], y[8], bell;
                    eight(fm, t, g);
                    eight(fm, t + F / 4, up);
#pragma unroll
                    for (int e = 0; e < 8; ++e) y[e] = g[e] * act_share<BELL>(act, g[e], bell) * up[e];
                    const uint32_t count = INSIDE ? 8u : m < args.M ? left(n + 32u * t, args.N) : 0u;
                    if constexpr (INSIDE) {
                        // Past the caches (nt): y, gate and up, which nothing reads soon, would evict
                        // slabs that the XCD's other workgroups are still to read (all three kept at
                        // 8192 x 4096 x 8192 bf16: 2500 -> 2210 cycles a slab).
                        __builtin_nontemporal_store(pack8<DT>(y), (u32x4*)(y_at + 32 * t));
                        if (args.gate) __builtin_nontemporal_store(pack8<DT>(g), (u32x4*)(gate_at + 32 * t));
                        if (args.up) __builtin_nontemporal_store(pack8<DT>(up), (u32x4*)(up_at + 32 * t));
                    } else if (count != 0u) {
                        store8<DT>(y_at + 32 * t, y, count);
                        if (args.gate) store8<DT>(gate_at + 32 * t, g, count);
                        if (args.up) store8<DT>(up_at + 32 * t, up, count);
                    }
                }
            }
        };
        if (args.act == kActBell) inside ? gated(TRUE_{}, TRUE_{}) : gated(TRUE_{}, FALSE_{});
        else inside ? gated(FALSE_{}, TRUE_{}) : gated(FALSE_{}, FALSE_{});
    } else if constexpr (EPI == LIN_LSE) {
        // Every lane's sum is relative to its own largest logit; the four lanes of a row
        // meet afterwards, all rows at once.
        float top[F], sum[F];
        const uint32_t c0 = n0 + wc * WT;
        auto sums = [&](auto inside_c) __attribute__((always_inline)) {
            constexpr bool INSIDE = decltype(inside_c)::value;
            const uint32_t n = c0 + 8u * lg;
#pragma unroll
            for (int fm = 0; fm < F; ++fm) {
                float v[F / 2][8];
#pragma unroll
                for (int t = 0; t < F / 2; ++t) {
                    eight(fm, t, v[t]);
                    if constexpr (!INSIDE) {
#pragma unroll
                        for (uint32_t e = 0; e < 8; ++e)
                            if (n + 32u * t + e >= args.N) v[t][e] = -__builtin_inff();
                    }
                }
                float a = -__builtin_inff(), b = a;
#pragma unroll
                for (int t = 0; t < F / 2; ++t)
#pragma unroll
                    for (int e = 0; e < 8; e += 4) {
                        a = fmaxf(fmaxf(a, v[t][e]), v[t][e + 1]);
                        b = fmaxf(fmaxf(b, v[t][e + 2]), v[t][e + 3]);
                    }
                a = fmaxf(a, b);
                top[fm] = a;
                const float from = a == -__builtin_inff() ? 0.0f : a;  // the sum is in units of exp(from)
                float s0 = 0.0f, s1 = 0.0f;
#pragma unroll
                for (int t = 0; t < F / 2; ++t)
#pragma unroll
                    for (int e = 0; e < 8; e += 2) {
                        s0 += exp_past(v[t][e], from);
                        s1 += exp_past(v[t][e + 1], from);
                    }
                sum[fm] = s0 + s1;
                __builtin_amdgcn_sched_barrier(0);  // one row of blocks after the other: they do not fit the registers
            }
        };
        if (inside) sums(TRUE_{});
        else sums(FALSE_{});
        // the targets' logits, where they are among the wave's columns: seldom
#pragma unroll
        for (int fm = 0; fm < F; ++fm) {
            const uint32_t at = (uint32_t)row_target[fm] - c0, m = row_of(fm);
            const bool here = row_target[fm] >= (int64_t)c0 && row_target[fm] < (int64_t)c0 + WT && row_target[fm] < (int64_t)args.N &&
                              (at / 8u) % 4u == lg && m < args.M;
            if (__builtin_amdgcn_ballot_w64(here) == 0u) continue;
            float hit = 0.0f;
#pragma unroll
            for (uint32_t t = 0; t < F / 2; ++t) {
                float v[8];
                eight(fm, t, v);
#pragma unroll
                for (uint32_t e = 0; e < 8; ++e) hit = at == 32u * t + 8u * lg + e ? v[e] : hit;
            }
            if (here) args.hit[m] = hit;
        }
#pragma unroll
        for (int fm = 0; fm < F; ++fm) {
            const float all = max_over_groups(top[fm]);
            const float s = sum_over_groups(sum[fm] * exp_past(top[fm], all == -__builtin_inff() ? 0.0f : all));
            const uint32_t m = row_of(fm);
            if (lg == 0u && m < args.M) args.part[(size_t)(u.n_idx * 2u + wc) * args.M + m] = make_float2(all, s);
        }
    } else if constexpr (EPI == LIN_DLOGITS) {
        // dl is rounded once to the 16 bits that the matrix core takes: dx and dweight, 1.7e-3 off
        // in bf16 and 2.1e-4 in fp16 by their own rounding, become 1.8e-3 and 2.3e-4 off.
        const uint32_t c0 = n0 + wc * WT;
        auto gradient = [&](auto inside_c) __attribute__((always_inline)) {
            constexpr bool INSIDE = decltype(inside_c)::value;
            const uint32_t n = c0 + 8u * lg;
#pragma unroll
            for (int fm = 0; fm < F; ++fm) {
                const uint32_t m = row_of(fm);
                const LossRow r = row_info[fm];
                const uint32_t at = (uint32_t)r.target - args.first - c0;  // of the wave's columns, if below WT
                const bool some = __builtin_amdgcn_ballot_w64(r.target >= 0 && at < (uint32_t)WT) != 0u;
                uint16_t* const to = args.dl + (int64_t)m * args.lddl + n;
#pragma unroll
                for (int t = 0; t < F / 2; ++t) {
                    float v[8];
                    eight(fm, t, v);
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[e] = exp_past(v[e], r.lse);
                    if (some) {
#pragma unroll
                        for (uint32_t e = 0; e < 8; ++e) v[e] -= at == 32u * t + 8u * lg + e ? 1.0f : 0.0f;
                    }
#pragma unroll
                    for (uint32_t e = 0; e < 8; ++e) {
                        v[e] *= r.d;
                        if constexpr (!INSIDE) v[e] = n + 32u * t + e >= args.N ? 0.0f : v[e];
                    }
                    u32x4 w = pack8<DT>(v);
                    if (r.target < 0) w = u32x4{0u, 0u, 0u, 0u};  // whatever its logits are
                    if (INSIDE || m < args.M) *(u32x4*)(to + 32 * t) = w;
                }
            }
        };
        if (inside) gradient(TRUE_{});
        else gradient(FALSE_{});
    } else {
        // whole tiles belong to one half: `half` is a multiple of T or past the end
        const bool upper = m0 >= args.half;
        const uint32_t rows = upper ? args.half + args.out_rows : args.out_rows, end = rows < args.M ? rows : args.M;
        const bool whole = m0 + T <= end && n0 + T <= args.N;
        if (args.sums) {
            auto add_up = [&](auto whole_c, auto add_c) __attribute__((always_inline)) {
#pragma unroll
                for (int fm = 0; fm < F; ++fm) {
                    const uint32_t m = row_of(fm), n = n0 + wc * WT + 8u * lg;
                    float* const at = args.sums + ((size_t)u.split * args.M + m) * args.N + n;
#pragma unroll
                    for (int t = 0; t < F / 2; ++t) {
                        float v[8];
                        eight(fm, t, v);
                        if (!decltype(whole_c)::value && (m >= end || n + 32u * t >= args.N)) continue;  // N is a multiple of 8
                        f32x4 x = {v[0], v[1], v[2], v[3]}, y = {v[4], v[5], v[6], v[7]};
                        if constexpr (decltype(add_c)::value) {
                            x += *(const f32x4*)(at + 32 * t);
                            y += *(const f32x4*)(at + 32 * t + 4);
                        }
                        *(f32x4*)(at + 32 * t) = x;
                        *(f32x4*)(at + 32 * t + 4) = y;
                    }
                }
            };
            if (whole) args.add ? add_up(TRUE_{}, TRUE_{}) : add_up(TRUE_{}, FALSE_{});
            else args.add ? add_up(FALSE_{}, TRUE_{}) : add_up(FALSE_{}, FALSE_{});
        } else {
            const float scale = args.unscale ? *args.unscale : 1.0f;
            uint16_t* const out = upper ? args.out2 - (int64_t)args.half * args.ldo2 : args.out;
            const int64_t ld = upper ? args.ldo2 : args.ldo;
            auto round_off = [&](auto whole_c) __attribute__((always_inline)) {
#pragma unroll
                for (int fm = 0; fm < F; ++fm) {
                    const uint32_t m = row_of(fm), n = n0 + wc * WT + 8u * lg;
                    uint16_t* const at = out + (int64_t)m * ld + n;
#pragma unroll
                    for (int t = 0; t < F / 2; ++t) {
                        float v[8];
                        eight(fm, t, v);
                        if (!decltype(whole_c)::value && (m >= end || n + 32u * t >= args.N)) continue;
#pragma unroll
                        for (int e = 0; e < 8; ++e) v[e] *= scale;
                        *(u32x4*)(at + 32 * t) = pack8<DT>(v);
                    }
                }
            };
            if (whole) round_off(TRUE_{});
            else round_off(FALSE_{});
        }
    }
    }
    wait_vm<0>();  // no DMA may still target LDS when the workgroup retires
}

}  // namespace tsg
