// The rule that chooses the weight gradient's tile and row split: plain C++, for
// the launches (tsgemm_wgrad_tu.hip) and for tests that ask which kernel a shape
// takes.
#pragma once

#include <stdint.h>

#include <initializer_list>

namespace tsg {

struct WgradShape {
    int tile;
    int64_t m_blocks, n_blocks, slabs, splits, per_split;
};

// Tile edge and row split by the time they should take, in us: rounds of
// workgroups (one 256 x 256 tile or two 128 x 128 tiles per compute unit) times
// the slabs of one (1.4 of a large tile; of a small one 0.56 alone and 0.95 beside
// another) and a start of 3, plus a second launch of 3, the splits' fp32 products
// written and read at 4 TB/s and 0.03 a split for adding them up.  Measured with
// both sides of each choice, operands in the cache: 4096 x 2048 x 2048 bf16 small
// tiles unsplit 45, large ones in 4 splits 51; 32768 x 2048 x 2048 large in 4 splits
// 212, small in 2 273; 65536 x 64 x 64 small in 64, 128 and 256 splits 16.3, 13.3 and
// 13.9; 512^3 small unsplit 8.5, in 2 splits 9.9.
inline WgradShape wgrad_shape(int64_t rows, int64_t out, int64_t width) {
    constexpr int64_t kCus = 256;  // MI355X
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

}  // namespace tsg
