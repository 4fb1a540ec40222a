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

// Tile edge and row split by the time they should take: rounds of workgroups
// (one 256 x 256 tile or two 128 x 128 tiles per compute unit) times the slabs of
// one, plus the traffic of the splits' fp32 products.
WgradShape wgrad_shape(int64_t rows, int64_t out, int64_t width) {
    WgradShape best = {};
    double best_us = 0;
    for (int tile : {256, 128}) {
        const int64_t mb = (out + tile - 1) / tile, nb = (width + tile - 1) / tile, tiles = mb * nb;
        const int64_t slabs = (rows + 63) / 64, room = tile == 256 ? kCus : 2 * kCus;
        const double slab_us = tile == 256 ? 1.1 : 0.7;
        for (int64_t splits = 1; splits <= 64 && (splits == 1 || splits <= slabs); ++splits) {
            const int64_t per = slabs ? (slabs + splits - 1) / splits : 0;
            if (splits > 1 && (per * (splits - 1) >= slabs || tiles * splits > 4 * room)) continue;
            const double rounds = (double)((tiles * splits + room - 1) / room);
            const double product = 8e-6 * (double)(out * width) / 4.0;  // write and read of one fp32 product, us at 4 TB/s
            const double us = rounds * ((double)per * slab_us + 3.0) + (splits > 1 ? 3.0 + (double)splits * product : 0.0);
            if (best.tile == 0 || us < best_us) {
                best = {tile, mb, nb, slabs, splits, per};
                best_us = us;
            }
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
        const uint64_t count = (uint64_t)a.out * a.width;
        const dim3 grid((unsigned)((count / 8u + 255u) / 256u)), block(256);
        if (odt == DT_FP16) hipLaunchKernelGGL((wgrad_sum_kernel<DT_FP16>), grid, block, 0, s, a.part, a.splits, count, a.dw);
        else if (odt == DT_BF16) hipLaunchKernelGGL((wgrad_sum_kernel<DT_BF16>), grid, block, 0, s, a.part, a.splits, count, a.dw);
        else hipLaunchKernelGGL((wgrad_sum_kernel<4>), grid, block, 0, s, a.part, a.splits, count, a.dw);
    }
}

}  // namespace tsg
