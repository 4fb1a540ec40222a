// The weight gradient's launches.
#include "tsgemm_wgrad_kernel.h"
#include "tsgemm_wgrad_shape.h"
#include "tsgemm_ops_launch.h"

namespace tsg {

namespace {

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
