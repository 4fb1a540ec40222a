// The rules that choose tiles, splits of the sum and pieces of the vocabulary for
// the products of tsgemm_linear_kernel.h: plain C++, for the launches and for
// tests that ask which kernel a shape takes.
#pragma once

#include <stdint.h>

#include <initializer_list>

namespace tsg {

struct LinShape {
    int tile;
    int64_t m_blocks, n_blocks, slabs, splits, per_split;
    double us;  // by the rule below
};

// Tile edge (and, where the product may be split along its sum, the splits) by the
// time they should take, in us: rounds of workgroups (one 256 x 256 tile or two 128
// x 128 tiles per compute unit) times the slabs of one (1.1 of a large tile, 1.3 where
// few share what they read; of a small one 0.7 alone and 1.0 beside another) and a start
// of 4, plus the splits' fp32 products written and read at 6 TB/s and a second launch.
// Measured with both sides of each choice, bf16, the activation's gradient (about 10)
// included: dx 2000 x 2048, hidden 2048: large tiles in 1, 2 and 4 splits 94, 67 and 57,
// small ones in 1 and 2 63 and 55; dx 1000 x 2504, hidden 6001: large in 4, 6 and 8 splits
// 98, 85 and 118, small in 3 90; 512 x 512, hidden 1024: small in 1, 4 and 8 33, 19.2 and
// 19.2; the projection 2000 x 2048 x 2048 large 40.6, small 32.0.
// `columns`: of the product per tile edge T, T or (two projections) T / 2.
inline LinShape linear_shape(int64_t M, int64_t N, int64_t slabs, bool halves, bool may_split) {
    constexpr int64_t kCus = 256;  // MI355X
    LinShape best = {};
    for (int tile : {256, 128}) {
        const int64_t cols = halves ? tile / 2 : tile;
        const int64_t mb = (M + tile - 1) / tile, nb = (N + cols - 1) / cols, tiles = mb * nb, room = tile == 256 ? kCus : 2 * kCus;
        for (int64_t splits = 1, per = slabs; splits <= 64; splits = (slabs + per - 2) / (per - 1)) {
            per = (slabs + splits - 1) / splits;
            if (splits > 1 && tiles * splits > 2 * room) break;
            const double slab_us = tile == 256 ? (tiles * splits <= kCus / 2 ? 1.3 : 1.1) : tiles * splits <= kCus ? 0.7 : 1.0;
            const double rounds = (double)((tiles * splits + room - 1) / room);
            const double product = 8e-6 * (double)(M * N) / 6.0 + 0.03;
            const double us = rounds * ((double)per * slab_us + 4.0) + (splits > 1 ? 3.0 + (double)splits * product : 0.0);
            if (best.tile == 0 || us < best.us) best = {tile, mb, nb, slabs, splits, per, us};
            if (!may_split || per <= 1) break;
        }
    }
    return best;
}

// Up to this many rows there is a kernel (tsgemm_linear_few.h) for the products that read
// x and the weights alone, in `few_groups` workgroups.
constexpr int64_t kFewRows = 32;

// Whether it takes a product: by the time that either kernel should take, in us.  A million
// values of the weights are 0.30 there and every row 0.008 on top (0.0042 where two weights
// share it), as each group of 16 weight rows fetches x for itself; the tile kernel pays
// none for rows up to 128, but 0.38 a million (the weights' way through the chip), and at
// least 1.2 of the rule above.  Measured bf16, weights from HBM, few and tile: cross
// entropy 4096 x 8192 of 1 and 32 rows 20.7 and 62, 32 and 63; 4096 x 131072 of 1, 16, 17
// and 32 rows 174 and 240, 239 and 241, 267 and 241, 352 and 242; 1000 x 50001 of 8 and 24
// rows 28 and 35, 38 and 36; gated 4096 x 14336 of 1 and 32 rows 45 and 67, 65 and 67; 1024
// x 65536 of 1 and 32 rows 44 and 49, 67 and 50.  Of 189 such shapes the rule's choice is
// on average 0.5% slower than the better one, at worst 17%; always this kernel 6% and 79%.
inline bool takes_few(const LinShape& s, int64_t rows, int64_t columns, int64_t width, int weights) {
    const double values = 1e-6 * (double)weights * (double)columns * (double)width;
    const double few = values * (0.30 + (weights == 2 ? 0.0042 : 0.008) * (double)rows);
    const double tile = 1.2 * s.us > 0.38 * values ? 1.2 * s.us : 0.38 * values;
    return rows <= kFewRows && few < tile;
}
inline int64_t few_groups(int64_t columns) {
    const int64_t tiles = (columns + 15) / 16;
    return tiles < 512 ? tiles : 512;
}

inline int64_t round_up(int64_t v, int64_t to) { return (v + to - 1) / to * to; }

// Columns of a gradient's halves dg and du: whole tiles.
inline int64_t gated_pitch(int64_t hidden) { return round_up(hidden, 256); }

// Columns of the vocabulary that the gradient of the logits is held for at a time:
// whole tiles, all of them if their 16-bit values take at most 128 MiB or if they are
// 2048 or fewer; else as many pieces as there are of that size, made alike (40000 rows of
// 2100 words: two of 1280).  At most 2^22 (32-bit offsets in a quarter of a slab).  A
// piece that the Infinity Cache (256 MiB) holds is read by both products without going
// to HBM again: 8192 x 4096 x 131072 bf16 17.9 ms; with 64, 256 and 512 MiB 19.2, 18.5 and 18.2.
inline int64_t vocab_piece(int64_t rows, int64_t vocab) {
    const int64_t most = (int64_t(1) << 26) / (rows > 0 ? rows : 1) / 256 * 256;
    const int64_t all = round_up(vocab, 256), piece = most < 2048 ? 2048 : most < (1 << 22) ? most : 1 << 22;
    if (all <= piece) return all;
    const int64_t pieces = (all + piece - 1) / piece;
    return round_up((vocab + pieces - 1) / pieces, 256);
}

}  // namespace tsg
