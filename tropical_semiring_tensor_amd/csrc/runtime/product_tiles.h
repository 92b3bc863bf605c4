// Tiles of the matrix cores' products (mfma_gemm.h): their sizes and what they
// cost, by which a call chooses among them.
#pragma once
#include <cstdint>

namespace trop {

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline int64_t round_up(int64_t a, int64_t b) { return ceil_div(a, b) * b; }

// A tile's time (us) over `k` tiles of 64 along k, and how many run at once,
// in a launch of `tiles` (kind 0: 256 x 256, 1: 128 x 128, 2: 64 x 64).
// Measured on one MI355X (256 CUs): a 256 x 256 workgroup has a CU to itself
// and takes 1.75 us a k tile; a 128 x 128 one 0.7 us alone on a CU, 1.15
// beside another; a 64 x 64 one 0.3 us alone, 0.5 with two and 0.85 with
// four on a CU; a tile costs 6, 5 or 4 us besides (first loads, epilogue).
// A k tile of 32 of float32's two planes takes 1.25 of these (in the
// gradients, which also split G, 1.35: alike for every tile, and left out).
struct TileRate {
    double us;
    int64_t slots;
};
inline TileRate tile_rate(int kind, int64_t tiles, double k) {
    if (kind == 0) return {k * 1.75 + 6.0, 256};
    if (kind == 1) return tiles <= 256 ? TileRate{k * 0.7 + 5.0, 256} : TileRate{k * 1.15 + 5.0, 512};
    return tiles <= 256   ? TileRate{k * 0.3 + 4.0, 256}
           : tiles <= 512 ? TileRate{k * 0.5 + 4.0, 512}
                          : TileRate{k * 0.85 + 4.0, 1024};
}
inline double tile_time(int kind, int64_t tiles, double k) {
    const TileRate r = tile_rate(kind, tiles, k);
    return (double)ceil_div(tiles, r.slots) * r.us;
}

inline int64_t tile_edge(int tile) { return tile == 3 ? 128 : 256 >> tile; }
inline uint32_t tile_threads(int tile) { return tile == 0 ? 512 : 256; }

}  // namespace trop
