// The weight gradient of a layer from its 8-bit activation, for gfx950 (CDNA4):
//
//   dw[o][i] = sum_r dy[r][o] * x(codes[r][i]) * s(scales[r][i / 32])
//
// dy is fp16 or bf16, x() an E4M3 element, s() an E8M0 scale (OCP Microscaling
// Formats specification v1.0).  The sum runs over the rows, across which the
// scales change, so the block-scaled matrix instruction (one scale per 32 terms
// of the sum) cannot take them: the codes are decoded on their way into LDS.
//   * bf16 dy: to bf16, which holds every element times scale exactly from scales
//     of 2^-124 (code 3; its last place is 2^-133, that of the elements 2^-9) up to
//     2^128, where fp32 ends too.
//   * fp16 dy: to fp16, times 2^kShift, which dw is divided by in the end.  That
//     is exact for scales of 2^kScaleLow ... 2^kScaleHigh: the least element
//     2^-9 becomes at least fp16's least 2^-24, the largest 448 at most 57344.
//     Blocks of activations whose largest magnitude is between 2^-13 and 2^10
//     have such scales.  A 64-row slab with a block outside (other than one of
//     zeros) is multiplied in bf16 instead, with dy split into two bf16 values
//     whose sum it is, at half the rate: no term loses a bit either way, but for
//     the ends that bf16 has above.  The factor 2^kShift stays in the accumulators,
//     so a sum of far terms overflows from 2^122 on.
//
// Both operands lie with the sum's index slowest, [row][column], and both come
// out of LDS through the transpose read ds_read_b64_tr_b16.  One workgroup of
// 4 waves (2 x 2) forms one BM x BN tile of dw over a range of 64-row slabs:
//   * dy's slabs go straight into LDS (buffer_load ... lds);
//   * codes and scales go to registers two slabs ahead, 32 codes and their scale
//     per thread and pass, are converted (v_cvt_scalef32_pk_bf16_fp8, two a time,
//     the scale's code as the exponent field) and written to LDS between MFMAs;
//   * two LDS stages; the one barrier per slab stands before the slab's second
//     k-step, when its last fragments are in registers.
// With few tiles the rows are split over workgroups, whose fp32 tiles a second
// launch adds up in order.
//
// Measured, over several boxes: 8192^3 bf16 741-795 us, 1383-1484 TFLOP/s (the
// library's bf16 product of that size 1238-1413), bound by the board's power: 1380 W
// of 1400, clocks down to 2.1 GHz; fp16 811-859 us (library 1223-1339 TFLOP/s, 821-899
// us).  32768 x 2048 x 2048 in 4 splits 212 us, of which the products' way through
// memory takes 25.  512^3 fp16 9.1 us: 16 workgroups, 8 slabs each, every one a round
// trip.  4096 x 2048 x 2048 bf16 56.5 us with its operands in HBM, 46.4 in the cache;
// there dequantizing and the library's product take 49.2.
//
// Built and not kept for the 128 x 128 tile: four stages of dy with three slabs on
// their way.  One workgroup alone went from 0.53 to 0.43 us a slab, 256 of them
// stayed at 0.62 (4096 x 2048 x 2048 44.6 -> 45.5 us), 512^3 8.5 -> 8.7: its LDS
// reads, twice those of a large tile per product, bound it, not latency.
#pragma once

#include "tile_scheduler.h"
#include "tsgemm_device.h"

namespace tsg {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

struct WgradArgs {
    const uint16_t* dy;     // [rows][out], rows lddy apart
    const uint8_t* codes;   // [rows][width]
    const uint8_t* scales;  // [rows][width / 32]
    void* dw;               // [out][width]
    float* part;            // [splits][out][width] fp32 when splits > 1
    int64_t rows, lddy;
    uint32_t out, width;
    uint32_t m_blocks, n_blocks, splits, slabs_per_split;
};

template <int BM, int BN>
struct WgradTraits {
    static constexpr int BK = 64;
    static constexpr int WM = BM / 2, WN = BN / 2, FM = WM / 16, FN = WN / 16;
    static constexpr int A_ROW = BM * 2, B_ROW = BN * 2;     // bytes of an LDS row
    static constexpr int A_STAGE = BK * A_ROW, B_STAGE = BK * B_ROW;
    static constexpr int B_OFF = 2 * A_STAGE;
    static constexpr int LDS = 2 * (A_STAGE + B_STAGE);
    static constexpr int CA = BM / 8;                        // 16-byte chunks of an A row
    static constexpr int NA = A_STAGE / 4096;                // DMAs of a wave per slab
    static constexpr int TPR = BN / 32;                      // threads of a row of codes
    static constexpr int NP = BK * TPR / 256;                // passes of 32 codes a thread
    static_assert(NP >= 1 && LDS <= 160 * 1024, "tile");
};

// How a slab is multiplied: bf16 dy; fp16 dy with codes as fp16; fp16 dy split.
enum { WG_BF16 = 0, WG_FP16 = 1, WG_SPLIT = 2 };
constexpr int kShift = 6, kScaleLow = -15 - kShift, kScaleHigh = 7 - kShift;
constexpr uint32_t kSplitSlabs = 16;  // slabs multiplied in bf16 before fp16 is tried again

// acc += a * b as mfma16x16x32, for operands that vector instructions have just
// written: the two wait states cover what the compiler would place.
__device__ __forceinline__ void mfma_bf16_settled(f32x4& acc, i16x8 a, i16x8 b) {
    asm volatile("s_nop 1\n\tv_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+a"(acc) : "v"(a), "v"(b));
}

// Race-detection build (TSG_STRESS): a pause of 0 to ~2048 cycles, as stress_pause,
// whose length comes from a linear congruential sequence that each wave starts
// elsewhere.  All of it is one asm block: branches or arithmetic that the compiler
// sees at every pause take the registers that the accumulators need, which it then
// copies right beside MFMAs that it cannot see to wait for.  The count only falls,
// so the loop ends.
__device__ __forceinline__ uint32_t pause_seed(uint32_t wave) { return (blockIdx.x * 4u + wave + 1u) * 0x9E3779B1u; }
__device__ __forceinline__ void wgrad_pause(uint32_t& state) {
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

// 8 fp16 values times 2^kShift = hi + lo in bf16, exactly (11 significant bits in 8 + 3).
__device__ __forceinline__ void split_f16(i16x8 v, i16x8& hi, i16x8& lo) {
    const f16x8 x = __builtin_bit_cast(f16x8, v);
    bf16x8 h, l;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float f = (float)x[e] * (float)(1 << kShift);
        h[e] = (__bf16)f;
        l[e] = __builtin_isinf(f) ? (__bf16)0.f : (__bf16)(f - (float)h[e]);  // inf - inf is no number
    }
    hi = __builtin_bit_cast(i16x8, h);
    lo = __builtin_bit_cast(i16x8, l);
}

template <int DT, int ODT, int BM, int BN>
__global__ __launch_bounds__(256, BM == 256 ? 1 : 2) void wgrad_kernel(WgradArgs args) {
    using T = WgradTraits<BM, BN>;
    constexpr int FM = T::FM, FN = T::FN, NA = T::NA, NP = T::NP;
    __shared__ __attribute__((aligned(1024))) uint8_t smem[T::LDS];
    __shared__ __attribute__((aligned(16))) uint32_t flags[2][4];  // fp16: a slab needs the split, by wave
    typedef __attribute__((address_space(3))) uint8_t lds_u8;
    typedef __attribute__((address_space(3))) u32x4 lds_u32x4;
    const uint32_t lds_base = (uint32_t)reinterpret_cast<uintptr_t>((lds_u8*)smem);
    const uint32_t lane = threadIdx.x & 63u;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    uint32_t pauses = pause_seed(wave);  // race-detection build only
    auto pause = [&]() __attribute__((always_inline)) { wgrad_pause(pauses); };
    const uint32_t wr = wave >> 1, wc = wave & 1u;
    const uint32_t out = args.out, width = args.width, w32 = width / 32u;

    // ---- this workgroup's tile and rows ----
    const uint32_t tiles = args.m_blocks * args.n_blocks, units = tiles * args.splits;
    const uint32_t unit = worker_of_workgroup(blockIdx.x, units, 8u, units);
    const uint32_t split = unit / tiles;
    TileScheduler sched;
    sched.setup(tiles, args.m_blocks, args.n_blocks, 8u, 1u, 0u);
    sched.init(unit - split * tiles);
    const uint32_t m0 = sched.m_idx * BM, n0 = sched.n_idx * BN;
    const uint32_t all_slabs = (uint32_t)((args.rows + T::BK - 1) / T::BK);
    const uint32_t slab0 = split * args.slabs_per_split;
    const uint32_t slabs = slab0 >= all_slabs ? 0u
                           : all_slabs - slab0 < args.slabs_per_split ? all_slabs - slab0 : args.slabs_per_split;

    // ---- sources: origin and range of the next slab to fetch ----
    // A slab's descriptor spans its rows up to the matrix's last value, so rows
    // past the end read zeros; columns past the end read the next row's values,
    // which only reach columns of dw that are not stored.
    const uint32_t a_pitch = (uint32_t)args.lddy * 2u;
    uint64_t a_ptr = 0, c_ptr = 0, s_ptr = 0;
    int32_t a_left = 0, c_left = 0;
    auto seek = [&](uint32_t slab) __attribute__((always_inline)) {  // of this workgroup's
        const int64_t r0 = (int64_t)(slab0 + slab) * T::BK;
        a_ptr = reinterpret_cast<uint64_t>(args.dy) + (uint64_t)r0 * a_pitch + (uint64_t)m0 * 2u;
        c_ptr = reinterpret_cast<uint64_t>(args.codes) + (uint64_t)r0 * width + n0;
        s_ptr = reinterpret_cast<uint64_t>(args.scales) + (uint64_t)r0 * w32 + n0 / 32u;
        const int64_t all = args.rows - r0, here = (int64_t)(slabs - slab) * T::BK;
        a_left = c_left = (int32_t)(all < here ? all : here);  // rows < 2^31
    };
    auto span = [](int32_t l, uint32_t pitch, uint32_t last) __attribute__((always_inline)) -> uint32_t {
        const uint32_t r = l <= 0 ? 0u : l < T::BK ? (uint32_t)l : (uint32_t)T::BK;
        return r == 0u ? 0u : (r - 1u) * pitch + last;
    };
    i32x4 rs_a;
    __amdgpu_buffer_rsrc_t rs_c = make_rsrc(args.codes, 0u), rs_s = make_rsrc(args.scales, 0u);
    auto next_a = [&]() __attribute__((always_inline)) {
        rs_a = rsrc_words_u64(a_ptr, span(a_left, a_pitch, (out - m0) * 2u));
        a_ptr += (uint64_t)T::BK * a_pitch;
        a_left -= T::BK;
    };
    auto next_c = [&]() __attribute__((always_inline)) {
        rs_c = make_rsrc(reinterpret_cast<const void*>(c_ptr), span(c_left, width, width - n0));
        rs_s = make_rsrc(reinterpret_cast<const void*>(s_ptr), span(c_left, w32, w32 - n0 / 32u));
        c_ptr += (uint64_t)T::BK * width;
        s_ptr += (uint64_t)T::BK * w32;
        c_left -= T::BK;
    };

    // ---- dy: DMA q of a wave fills 64 16-byte places in order, row by row; a
    // lane fetches the chunk that the row's swizzle puts at its place ----
    uint32_t a_voff[NA];
#pragma unroll
    for (int q = 0; q < NA; ++q) {
        const uint32_t p = (wave * NA + q) * 64u + lane, row = p / T::CA, slot = p % T::CA;
        a_voff[q] = row * a_pitch + (slot ^ swz_b(row)) * 16u;
    }
    auto dma = [&](auto q_c, auto s_c) __attribute__((always_inline)) {
        constexpr int q = decltype(q_c)::value, S = decltype(s_c)::value;
        pause();
        dma16_at<(uint32_t)(S * T::A_STAGE + q * 1024)>(lds_base + wave * NA * 1024u, a_voff[q], rs_a);
    };

    // ---- codes: a thread takes block nb of row kr (+ 32 per pass).  Four
    // neighbouring lanes read 128 bytes of a row, the next four of the row
    // after, whose swizzle differs in its lowest bit.  A block fills 64 bytes of
    // LDS, half of the banks, so blocks 2 and 3 of four begin with their second
    // half: then eight lanes' writes meet no common bank (without
    // it a quarter of the LDS cycles were conflicts: 8192^3 bf16 773 -> 764 us,
    // 4096 x 2048 x 2048 48.3 -> 46.4) ----
    const uint32_t tid = threadIdx.x;
    const uint32_t nb = T::TPR == 8 ? (tid & 3u) | ((tid >> 1) & 4u) : tid & 3u;
    const uint32_t kr = T::TPR == 8 ? ((tid >> 4) << 1) | ((tid >> 2) & 1u) : tid >> 2;
    const uint32_t half = (nb >> 1) & 1u;  // that comes first
    uint32_t c_voff[NP][2], s_voff[NP];
#pragma unroll
    for (int p = 0; p < NP; ++p) {
        c_voff[p][0] = (kr + 32u * p) * width + nb * 32u + half * 16u;
        c_voff[p][1] = c_voff[p][0] ^ 16u;  // the width is a multiple of 32
        s_voff[p] = (kr + 32u * p) * w32 + nb;
    }
    u32x4 raw[2][NP][2];
    uint32_t scl[2][NP];
    auto load_codes = [&](auto s_c, auto i_c) __attribute__((always_inline)) {  // op i of 3 * NP
        constexpr int S = decltype(s_c)::value, p = decltype(i_c)::value / 3, w = decltype(i_c)::value % 3;
        if constexpr (w < 2)
            raw[S][p][w] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rs_c, c_voff[p][w], 0, 0));
        else
            scl[S][p] = __builtin_amdgcn_raw_buffer_load_b8(rs_s, s_voff[p], 0, 0);
    };
    uint32_t b_wr[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) b_wr[j] = lds_base + T::B_OFF + kr * T::B_ROW + ((nb * 4u + (j ^ (2u * half))) ^ swz_b(kr)) * 16u;
    auto convert = [&](auto mode_c, auto s_c, auto i_c) __attribute__((always_inline)) {  // stage and raw set, op i of 4 * NP
        constexpr int MODE = decltype(mode_c)::value, S = decltype(s_c)::value, R = S;
        constexpr int p = decltype(i_c)::value / 4, j = decltype(i_c)::value % 4;
        uint32_t field = scl[R][p];
        if constexpr (MODE == WG_FP16) field = field + kShift < 255u ? field + kShift : 255u;  // 255, a NaN, stays one
        const float s = __builtin_bit_cast(float, field << 23);
        const uint32_t w0 = raw[R][p][j / 2][2 * (j % 2)], w1 = raw[R][p][j / 2][2 * (j % 2) + 1];
        u32x4 v;
        if constexpr (MODE == WG_FP16) {
            v.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w0, s, false));
            v.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w0, s, true));
            v.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w1, s, false));
            v.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w1, s, true));
        } else {
            v.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w0, s, false));
            v.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w0, s, true));
            v.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w1, s, false));
            v.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w1, s, true));
        }
        *(lds_u32x4*)((lds_u8*)(uintptr_t)b_wr[j] + S * T::B_STAGE + p * 32 * T::B_ROW) = v;
    };

    // fp16: does one of this thread's blocks in raw set S need the split?  A wave's
    // answer goes to its word of flag row S; the workgroup's is read after the
    // next barrier.
    auto far_block = [&](auto s_c) __attribute__((always_inline)) -> bool {
        constexpr int S = decltype(s_c)::value;
        bool far = false;
#pragma unroll
        for (int p = 0; p < NP; ++p) {
            uint32_t any = 0;
#pragma unroll
            for (int w = 0; w < 8; ++w) any |= raw[S][p][w / 4][w % 4];
            const bool zeros = (any & 0x7F7F7F7Fu) == 0u && scl[S][p] + kShift < 255u;
            far |= scl[S][p] - (uint32_t)(127 + kScaleLow) > (uint32_t)(kScaleHigh - kScaleLow) && !zeros && scl[S][p] != 255u;
        }
        return far;
    };
    auto put_flag = [&](auto s_c) __attribute__((always_inline)) {
        const bool far = __builtin_amdgcn_ballot_w64(far_block(s_c)) != 0u;
        if (lane == 0u) flags[decltype(s_c)::value][wave] = far ? 1u : 0u;
    };
    auto get_flag = [&](auto s_c) __attribute__((always_inline)) -> bool {
        const u32x4 f = *(const u32x4*)flags[decltype(s_c)::value];
        return __builtin_amdgcn_readfirstlane(f.x | f.y | f.z | f.w) != 0u;
    };

    // ---- fragments.  As in the fp16/bf16 GEMM's B operand: the columns of a
    // pair of 16-wide blocks are interleaved, block b's lane group g holding
    // columns 8g + 4 (b ^ (g & 1)) + 0..3 of the pair's 32, so that one read's
    // 16 lanes spread over the banks and a lane of the result holds 8
    // consecutive columns of dw ----
    const uint32_t l16 = lane & 15u, lg = lane >> 4;
    uint32_t a_off[FM], b_off[FN];
    {
        const uint32_t k0 = 8u * lg + (l16 >> 2), sw = swz_b(k0);
#pragma unroll
        for (int f = 0; f < FM; ++f) {
            const uint32_t chunk = (wr * T::WM + 32u * (f / 2)) / 8u + (l16 & 3u);
            a_off[f] = lds_base + k0 * T::A_ROW + (chunk ^ sw) * 16u + 8u * ((f & 1u) ^ (l16 & 1u));
        }
#pragma unroll
        for (int f = 0; f < FN; ++f) {
            const uint32_t chunk = (wc * T::WN + 32u * (f / 2)) / 8u + (l16 & 3u);
            b_off[f] = lds_base + T::B_OFF + k0 * T::B_ROW + (chunk ^ sw) * 16u + 8u * ((f & 1u) ^ (l16 & 1u));
        }
    }
    i16x4 fa[2][FM][2], fb[2][FN][2];
    // read op r of a k-step (stage S, k-step K, into set K), in the order of use
    constexpr int R = 2 * FM + 2 * FN;
    auto read = [&](auto r_c, auto s_c, auto k_c) __attribute__((always_inline)) {
        constexpr int r = decltype(r_c)::value, S = decltype(s_c)::value, K = decltype(k_c)::value, h = r % 2;
        constexpr bool is_a = r < 2 || r >= 2 + 2 * FN;
        if constexpr (is_a) {
            constexpr int f = r < 2 ? 0 : (r - 2 * FN) / 2;
            fa[K][f][h] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                (lds_i16x4*)((lds_u8*)(uintptr_t)a_off[f] + S * T::A_STAGE + (K * 32 + h * 4) * T::A_ROW));
        } else {
            constexpr int f = (r - 2) / 2;
            fb[K][f][h] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                (lds_i16x4*)((lds_u8*)(uintptr_t)b_off[f] + S * T::B_STAGE + (K * 32 + h * 4) * T::B_ROW));
        }
    };

    f32x4 acc[FM][FN];
#pragma unroll
    for (int fm = 0; fm < FM; ++fm)
#pragma unroll
        for (int fn = 0; fn < FN; ++fn) {
            acc[fm][fn] = f32x4{0.f, 0.f, 0.f, 0.f};
            asm volatile("" : "+a"(acc[fm][fn]));  // cleared here, in registers of its own
        }
    // A vector write of a register -> an MFMA that reads it: two wait states.  The
    // MFMAs are asm, before which the compiler places none; left to itself it
    // cleared each accumulator right in front of its first MFMA.
    asm volatile("s_nop 1" ::: "memory");

    // One 32-row k-step on set K: FM * FN MFMAs, rows of blocks in order, the
    // columns there and back.  `between(s)` issues what goes after MFMA s.
    i16x8 hi, lo;
    auto kstep = [&](auto mode_c, auto k_c, auto&& between) __attribute__((always_inline)) {
        constexpr int MODE = decltype(mode_c)::value, K = decltype(k_c)::value;
        static_for<0, FM * FN>([&](auto s_c) __attribute__((always_inline)) {
            constexpr int s = decltype(s_c)::value, fm = s / FN, fn = (fm & 1) ? FN - 1 - s % FN : s % FN;
            const i16x8 bv = __builtin_shufflevector(fb[K][fn][0], fb[K][fn][1], 0, 1, 2, 3, 4, 5, 6, 7);
            const i16x8 av = __builtin_shufflevector(fa[K][fm][0], fa[K][fm][1], 0, 1, 2, 3, 4, 5, 6, 7);
            if constexpr (MODE == WG_SPLIT) {
                if constexpr (s % FN == 0) split_f16(av, hi, lo);
                mfma_bf16_settled(acc[fm][fn], bv, hi);
                mfma_bf16_settled(acc[fm][fn], bv, lo);
            } else {
                mfma16x16x32<MODE == WG_FP16 ? DT_FP16 : DT_BF16>(acc[fm][fn], bv, av);
            }
            between(s_c);
            __builtin_amdgcn_sched_barrier(0);
        });
    };
    using I0 = std::integral_constant<int, 0>;
    using I1 = std::integral_constant<int, 1>;

    // ops [n * s / slots, n * (s + 1) / slots) of n spread over `slots` gaps
    auto spread = [](auto n_c, auto slots_c, auto s_c, auto&& op) __attribute__((always_inline)) {
        constexpr int n = decltype(n_c)::value, slots = decltype(slots_c)::value, s = decltype(s_c)::value;
        if constexpr (s >= 0 && s < slots)
            static_for<n * s / slots, n*(s + 1) / slots>([&](auto i_c) __attribute__((always_inline)) { op(i_c); });
    };
    constexpr int STEPS = FM * FN;
    // the first gaps hold no LDS read: a fragment's registers are not refilled
    // while the last MFMA that read them may still fetch its operands
    constexpr int START = 4;
    constexpr int GAPS = 2 * STEPS - START;            // of a period
    // From a slab's second k-step to the end of the next slab's first: stage S
    // (the slab's) is refilled with the slab after next while the fragments come
    // from stage 1 - S.
    constexpr int LOADS = NA + 3 * NP;                 // DMAs, then loads of codes and scales
    auto fill = [&](auto mode_c, auto s_c, auto gap_c) __attribute__((always_inline)) {
        constexpr int S = decltype(s_c)::value;
        spread(std::integral_constant<int, LOADS>{}, std::integral_constant<int, GAPS / 2>{}, gap_c, [&](auto i_c) __attribute__((always_inline)) {
            constexpr int i = decltype(i_c)::value;
            if constexpr (i < NA) dma(i_c, s_c);
            else load_codes(std::integral_constant<int, 1 - S>{}, std::integral_constant<int, i - NA>{});
        });
        spread(std::integral_constant<int, 4 * NP>{}, std::integral_constant<int, GAPS - STEPS / 4>{}, gap_c,
               [&](auto i_c) __attribute__((always_inline)) { convert(mode_c, s_c, i_c); });
    };
    // `end`: the slab that this pipeline stops before; brought forward when the
    // codes of slab `next` (those that this period converts) need the split.
    auto period = [&](auto mode_c, auto s_c, uint32_t next, uint32_t& end) __attribute__((always_inline)) {
        constexpr int MODE = decltype(mode_c)::value, S = decltype(s_c)::value;
        using OTHER = std::integral_constant<int, 1 - S>;
        pause();
        wait_vm<0>();    // the next slab's dy and the codes after it have landed
        if constexpr (MODE == WG_FP16) {
            put_flag(s_c);
            pause();
        }
        lds_barrier();   // ... for every wave; stage S is read out, its successor written
        pause();
        next_a();
        next_c();
        kstep(mode_c, I1{}, [&](auto g_c) __attribute__((always_inline)) {
            constexpr int g = decltype(g_c)::value;
            if constexpr (g >= START) {
                spread(std::integral_constant<int, R>{}, std::integral_constant<int, STEPS - START>{},
                       std::integral_constant<int, g - START>{}, [&](auto r_c) __attribute__((always_inline)) { read(r_c, OTHER{}, I0{}); });
                fill(mode_c, s_c, std::integral_constant<int, g - START>{});
            }
        });
        bool far = false;
        if constexpr (MODE == WG_FP16) {
            pause();
            far = get_flag(s_c);
        }
        kstep(mode_c, I0{}, [&](auto g_c) __attribute__((always_inline)) {
            constexpr int g = decltype(g_c)::value;
            if constexpr (g >= START)
                spread(std::integral_constant<int, R>{}, std::integral_constant<int, STEPS - START>{},
                       std::integral_constant<int, g - START>{}, [&](auto r_c) __attribute__((always_inline)) { read(r_c, OTHER{}, I1{}); });
            fill(mode_c, s_c, std::integral_constant<int, STEPS + g - START>{});
        });
        if (MODE == WG_FP16 && far && next < end) end = next;
    };

    // Slabs [from, to) of this workgroup's; returns where it stopped (before
    // `to` only in WG_FP16, at a slab that needs the split).
    auto pipeline = [&](auto mode_c, uint32_t from, uint32_t to) __attribute__((always_inline)) -> uint32_t {
        constexpr int MODE = decltype(mode_c)::value;
        // slabs 0 and 1 into the stages, the codes of slab 2 on their way
        seek(from);
        next_a();
        static_for<0, NA>([&](auto q_c) __attribute__((always_inline)) { dma(q_c, I0{}); });
        next_a();
        static_for<0, NA>([&](auto q_c) __attribute__((always_inline)) { dma(q_c, I1{}); });
        next_c();
        static_for<0, 3 * NP>([&](auto i_c) __attribute__((always_inline)) { load_codes(I0{}, i_c); });
        next_c();
        static_for<0, 3 * NP>([&](auto i_c) __attribute__((always_inline)) { load_codes(I1{}, i_c); });
        if constexpr (MODE == WG_FP16) {
            put_flag(I0{});
            put_flag(I1{});
        }
        static_for<0, 4 * NP>([&](auto i_c) __attribute__((always_inline)) { convert(mode_c, I0{}, i_c); });
        static_for<0, 4 * NP>([&](auto i_c) __attribute__((always_inline)) { convert(mode_c, I1{}, i_c); });
        next_c();
        static_for<0, 3 * NP>([&](auto i_c) __attribute__((always_inline)) { load_codes(I0{}, i_c); });
        pause();
        wait_vm<0>();
        lds_barrier();
        pause();
        uint32_t end = to;
        if constexpr (MODE == WG_FP16) {
            const bool far0 = get_flag(I0{}), far1 = get_flag(I1{});
            pause();
            lds_barrier();  // the flags are read before the first period's
            pause();
            if (far0) return from;
            if (far1 && from + 1u < end) end = from + 1u;
        }
        static_for<0, R>([&](auto r_c) __attribute__((always_inline)) { read(r_c, I0{}, I0{}); });
        kstep(mode_c, I0{}, [&](auto g_c) __attribute__((always_inline)) {
            constexpr int g = decltype(g_c)::value;
            if constexpr (g >= START)
                spread(std::integral_constant<int, R>{}, std::integral_constant<int, STEPS - START>{},
                       std::integral_constant<int, g - START>{}, [&](auto r_c) __attribute__((always_inline)) { read(r_c, I0{}, I1{}); });
        });
        uint32_t k = from;
        while (k + 1u < end) {
            period(mode_c, I0{}, k + 2u, end);
            if (++k + 1u >= end) break;
            period(mode_c, I1{}, k + 2u, end);
            ++k;
        }
        kstep(mode_c, I1{}, [](auto) __attribute__((always_inline)) {});
        gap_nops();      // the last MFMAs have written their accumulators
        pause();
        wait_vm<0>();    // no DMA may still target LDS when the next pipeline starts or the workgroup retires
        lds_barrier();
        pause();
        return end;
    };

    if constexpr (DT == DT_BF16) {
        if (slabs != 0u) pipeline(std::integral_constant<int, WG_BF16>{}, 0u, slabs);
    } else {
        for (uint32_t at = 0; at < slabs;) {
            at = pipeline(std::integral_constant<int, WG_FP16>{}, at, slabs);
            if (at < slabs) {
                const uint32_t to = slabs - at < kSplitSlabs ? slabs : at + kSplitSlabs;
                pipeline(std::integral_constant<int, WG_SPLIT>{}, at, to);
                at = to;
            }
        }
    }
#pragma unroll
    for (int fm = 0; fm < FM; ++fm)
#pragma unroll
        for (int fn = 0; fn < FN; ++fn) asm volatile("" : "+a"(acc[fm][fn]));  // not read before the gap above

    // ---- store: lane (lg, l16) of block pair t holds columns 32t + 8 lg + 0..7
    // of one row of dw; in odd lane groups the pair's halves change places ----
    const bool swap = (lg & 1u) != 0u;
    const bool whole = args.splits == 1u;
    float* part = args.part + (whole ? 0u : (size_t)split * out * width);
#pragma unroll
    for (int fm = 0; fm < FM; ++fm) {
        const uint32_t p = l16 >> 2;
        const uint32_t m = m0 + wr * T::WM + 32u * (fm / 2) + 8u * p + 4u * ((fm & 1u) ^ (p & 1u)) + (l16 & 3u);
#pragma unroll
        for (int t = 0; t < FN / 2; ++t) {
            const uint32_t n = n0 + wc * T::WN + 32u * t + 8u * lg;
            if (m >= out || n >= width) continue;
            const f32x4 x = acc[fm][2 * t], y = acc[fm][2 * t + 1];
            f32x4 a = swap ? y : x, b = swap ? x : y;
            if constexpr (DT == DT_FP16) {
                a *= 1.0f / (1 << kShift);
                b *= 1.0f / (1 << kShift);
            }
            const size_t at = (size_t)m * width + n;
            if (!whole || ODT == 4) {
                float* p32 = (whole ? (float*)args.dw : part) + at;
                *(f32x4*)p32 = a;
                *(f32x4*)(p32 + 4) = b;
            } else if constexpr (ODT == DT_BF16) {
                const bf16x8 v = {(__bf16)a[0], (__bf16)a[1], (__bf16)a[2], (__bf16)a[3], (__bf16)b[0], (__bf16)b[1], (__bf16)b[2], (__bf16)b[3]};
                *(bf16x8*)((__bf16*)args.dw + at) = v;
            } else if constexpr (ODT == DT_FP16) {
                const f16x8 v = {(_Float16)a[0], (_Float16)a[1], (_Float16)a[2], (_Float16)a[3], (_Float16)b[0], (_Float16)b[1], (_Float16)b[2], (_Float16)b[3]};
                *(f16x8*)((_Float16*)args.dw + at) = v;
            }
        }
    }
}

// dw from the splits' fp32 products, 8 values per thread.  G threads share the
// splits of the same values, every G-th one in order; their sums meet in order.
// (65536 x 64 x 64 bf16 in 64 splits 20.8 -> 16.3 us, 65536 x 256 x 256 25.7 -> 22.4.)
template <int ODT, int G>
__global__ __launch_bounds__(256) void wgrad_sum_kernel(const float* part, uint32_t splits, uint64_t count, void* dw) {
    constexpr uint32_t V = 256u / G;  // threads of different values
    __shared__ f32x4 sums[G > 1 ? 2 : 1][G][V];
    const uint32_t v = threadIdx.x % V, g = threadIdx.x / V;
    const uint64_t i = ((uint64_t)blockIdx.x * V + v) * 8u;
    if (G == 1 && i >= count) return;  // count is a multiple of 8
    f32x4 a = {0.f, 0.f, 0.f, 0.f}, b = a;
    if (i < count) {
#pragma unroll 4
        for (uint32_t s = g; s < splits; s += G) {
            a += *(const f32x4*)(part + s * count + i);
            b += *(const f32x4*)(part + s * count + i + 4);
        }
    }
    if constexpr (G > 1) {
        sums[0][g][v] = a;
        sums[1][g][v] = b;
        lds_barrier();
        if (g != 0u || i >= count) return;
#pragma unroll
        for (int k = 1; k < G; ++k) {
            a += sums[0][k][v];
            b += sums[1][k][v];
        }
    }
    if constexpr (ODT == 4) {
        *(f32x4*)((float*)dw + i) = a;
        *(f32x4*)((float*)dw + i + 4) = b;
    } else if constexpr (ODT == DT_BF16) {
        const bf16x8 v = {(__bf16)a[0], (__bf16)a[1], (__bf16)a[2], (__bf16)a[3], (__bf16)b[0], (__bf16)b[1], (__bf16)b[2], (__bf16)b[3]};
        *(bf16x8*)((__bf16*)dw + i) = v;
    } else {
        const f16x8 v = {(_Float16)a[0], (_Float16)a[1], (_Float16)a[2], (_Float16)a[3], (_Float16)b[0], (_Float16)b[1], (_Float16)b[2], (_Float16)b[3]};
        *(f16x8*)((_Float16*)dw + i) = v;
    }
}

}  // namespace tsg
