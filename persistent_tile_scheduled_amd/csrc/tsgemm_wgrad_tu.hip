// The weight gradient's kernels and the rule that chooses tile and split.
#include "tsgemm_wgrad_kernel.h"
#include "tsgemm_ops_launch.h"

namespace tsg {

namespace {

constexpr int64_t kCus = 256;  // MI355X

struct WgradShape {
    int tile;
    int64_t m_blocks, n_blocks, slabs, splits, per_split;
};

// Tile edge and row split by the time they should take, in us: rounds of
// workgroups (one 256 x 256 tile or two 128 x 128 tiles per compute unit) times
// the slabs of one (1.4 of a large tile; of a small one 0.56 alone and 0.95 beside
// another) and a start of 3, plus a second launch of 3, the splits' fp32 products
// written and read at 4 TB/s and 0.03 a split for adding them up.  Measured with
// both sides of each choice: 4096 x 2048 x 2048 bf16 small tiles unsplit 45,
// large ones in 4 splits 51; 32768 x 2048 x 2048 large in 4 splits 212, small in 2
// 273; 65536 x 64 x 64 small in 64, 128 and 256 splits 16.3, 13.3 and 13.9;
// 512^3 small unsplit 8.5, in 2 splits 9.9.
WgradShape wgrad_shape(int64_t rows, int64_t out, int64_t width) {
    WgradShape best = {};
    double best_us = 0;
    for (int tile : {256, 128}) {
        const int64_t mb = (out + tile - 1) / tile, nb = (width + tile - 1) / tile, tiles = mb * nb;
        const int64_t slabs = (rows + 63) / 64, room = tile == 256 ? kCus : 2 * kCus;
        // every count of slabs that a split can have, with the fewest splits that give it
        for (int64_t splits = 1, per = slabs; splits <= 256; splits = (slabs + per - 2) / (per - 1)) {
            per = (slabs + splits - 1) / splits;
            if (splits > 1 && tiles * splits > 4 * room) break;
            const double slab_us = tile == 256 ? 1.4 : tiles * splits <= kCus ? 0.56 : 0.95;
            const double rounds = (double)((tiles * splits + room - 1) / room);
            const double product = 8e-6 * (double)(out * width) / 4.0 + 0.03;
            const double us = rounds * ((double)per * slab_us + 3.0) + (splits > 1 ? 3.0 + (double)splits * product : 0.0);
            if (best.tile == 0 || us < best_us) {
                best = {tile, mb, nb, slabs, splits, per};
                best_us = us;
            }
            if (per <= 1) break;
        }
    }
    return best;
}

template <int DT, int ODT>
void wgrad_of(const WgradArgs& a, int tile, hipStream_t s) {
    const dim3 grid(a.m_blocks * a.n_blocks * a.splits), block(256);
    if (tile == 256) hipLaunchKernelGGL((wgrad_kernel<DT, ODT, 256, 256>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((wgrad_kernel<DT, ODT, 128, 128>), grid, block, 0, s, a);
}

template <int ODT>
void wgrad_sum(const WgradArgs& a, hipStream_t s) {
    const uint64_t count = (uint64_t)a.out * a.width;
    const dim3 block(256);
    if (a.splits < 8u || count > 1u << 18)  // threads enough without sharing
        hipLaunchKernelGGL((wgrad_sum_kernel<ODT, 1>), dim3((unsigned)((count / 8u + 255u) / 256u)), block, 0, s, a.part, a.splits, count, a.dw);
    else
        hipLaunchKernelGGL((wgrad_sum_kernel<ODT, 8>), dim3((unsigned)((count / 8u + 31u) / 32u)), block, 0, s, a.part, a.splits, count, a.dw);
}

}  // namespace

int64_t wgrad_workspace(int64_t rows, int64_t out, int64_t width) {
    const WgradShape w = wgrad_shape(rows, out, width);
    return w.splits > 1 ? w.splits * out * width * (int64_t)sizeof(float) : 0;
}

void launch_wgrad(int dt, int odt, const WgradArgs& args, hipStream_t s) {
    WgradArgs a = args;
    const WgradShape w = wgrad_shape(a.rows, a.out, a.width);
    a.m_blocks = (uint32_t)w.m_blocks;
    a.n_blocks = (uint32_t)w.n_blocks;
    a.splits = (uint32_t)w.splits;
    a.slabs_per_split = (uint32_t)w.per_split;
    if (dt == DT_FP16) odt == DT_FP16 ? wgrad_of<DT_FP16, DT_FP16>(a, w.tile, s) : wgrad_of<DT_FP16, 4>(a, w.tile, s);
    else odt == DT_BF16 ? wgrad_of<DT_BF16, DT_BF16>(a, w.tile, s) : wgrad_of<DT_BF16, 4>(a, w.tile, s);
    if (w.splits > 1) {
        if (odt == DT_FP16) wgrad_sum<DT_FP16>(a, s);
        else if (odt == DT_BF16) wgrad_sum<DT_BF16>(a, s);
        else wgrad_sum<4>(a, s);
    }
}

}  // namespace tsg
