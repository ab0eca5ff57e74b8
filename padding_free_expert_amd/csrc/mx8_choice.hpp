// Which kernel a product on 8-bit rows runs: rules on the sizes of a call alone.
// Host code without HIP, so that it can be checked on its own.
#pragma once

#include <algorithm>
#include <cstdint>

namespace xmoe {

constexpr int kMxComputeUnits = 256;

struct Mx8Choice {
    int stream;  // 16-row blocks of the stream kernel (1, 2); 0: the tile kernel
    bool once;   // tile kernel: weights loaded past the caches
};

// Rows of at most E experts; N results a row; NB matrices side by side (2: the
// up-projection).
inline Mx8Choice mx8_choose(int64_t rows, int E, int N, int NB) {
    // Up + down, 64 experts of d = 2048, h = 1408: the stream kernel with 16 rows a
    // block, with 32, and the tile kernel take at 9 rows an expert 60 + 33, 63 + 33
    // and 73 + 41 us; at 12 63 + 35, 63 + 33 and 74 + 41; at 16 75 + 41, 64 + 34 and
    // 74 + 41; at 26 the last two 73 + 40 and 76 + 42; at 28 79 + 43 and 76 + 41; at 40
    // 116 + 63 and 77 + 43.  With more rows each 32 of them read the weights again,
    // which pays only where the launch is so small that the tile kernel leaves
    // compute units idle: three stream blocks for each unit at most (4 such experts of
    // 64, 96 and 128 rows 13 + 10, 17 + 10 and 23 + 14 us, tiles 21 + 16; 16 experts of
    // d = 512, h = 256 with 128 and 500 rows 8 + 6 and 21 + 15, tiles 12 + 9 and 13 + 10).
    const int64_t active = std::min<int64_t>(E, rows), width = 64 / NB;
    const int64_t blocks = (rows / 32 + active) * ((N + width - 1) / width);
    if (rows <= 12 * active) return {1, false};
    if (rows <= 26 * active || blocks <= 3 * kMxComputeUnits) return {2, false};
    // Weights that one row tile reads go past the caches: 64 experts of d = 2048, h =
    // 1408 with 40 rows 82 + 47 -> 78 + 43 us, of d = 4096, h = 1024 with 62 rows 123 +
    // 72 -> 117 + 71; with two row tiles they meet again (384 rows 162 + 88 -> 173 + 98).
    // A launch without a tile for each compute unit keeps to the caches (4 experts
    // with 64 rows 21 + 16 against 25 + 19, their weights in the last-level cache).
    const int64_t cols = (N + 256 / NB - 1) / (256 / NB);
    return {0, rows <= 128 * active && active * cols >= kMxComputeUnits};
}

}  // namespace xmoe
