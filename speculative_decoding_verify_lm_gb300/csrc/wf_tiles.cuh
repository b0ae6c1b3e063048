// How a sweep cuts a head's weights into tiles.  Host arithmetic only.
#pragma once

namespace wf {

// Weight rows per tile: as many tiles as the CTAs (or pairs) take in the fewest
// rounds, so that every CTA gets about the same rows in each.  Tiles have one of
// two heights, `step` apart.  (2,048 rows over 32,000 ids: 125 tiles of 256 are
// 13.2 rounds for 76 pairs; 133 of two heights are 14 full ones.  Tiles of one
// smaller height that fill the rounds, 192 of them, took 236 us a call, since both
// operands cross to the SMs once for each tile.)
struct Tiles {
    int num_n, bn, nbig, step;   // nbig tiles of bn rows, then num_n - nbig of bn - step
};
constexpr int MAX_TILE = 256, MIN_TILE = 64;

// A CTA's own products have 128 rows and take N in steps of 16.  A pair's have 256
// rows and are given N in steps of 32, the half of each CTA a multiple of 16; kept
// logits leave in boxes of 32 columns.  (Steps of 16 for pairs: 300 rows of 256 over
// 20,000 ids with 10 best 34.7 us in place of 31.0, 1,248 of 2,560 over 151,936 515 either way.)
constexpr int tile_step(bool pair, bool kept) { return pair || kept ? 32 : 16; }

inline Tiles tiles_of(int V, int slots, int num_mt, int step) {
    Tiles t{};
    t.step = step;
    const int least = (int)(((long)V + MAX_TILE - 1) / MAX_TILE);
    const long rounds = ((long)num_mt * least + slots - 1) / slots;
    long n = rounds * slots / num_mt;
    if (n > V / MIN_TILE) n = V / MIN_TILE;
    if (n < least) n = least;
    t.num_n = (int)n;
    if (V < MIN_TILE) {
        t.bn = MIN_TILE;
        t.nbig = t.num_n;
        return t;
    }
    const int h = (int)(V / n) / step * step;   // at least MIN_TILE
    t.bn = h + step;
    t.nbig = (int)((V - n * h + step - 1) / step);
    if (t.nbig == 0) {
        t.bn = h;
        t.nbig = t.num_n;
    }
    return t;
}

}  // namespace wf
