// Which of the product kernels serves a call (host side, no HIP): the choice
// that product.hpp launches by and that ep_probe_product_path tells.
#pragma once

#include <stdint.h>

namespace epk {

// Storage formats as the kernels are instantiated for them.
enum WeightKind { kBf16 = 0, kMxfp4 = 1, kInt4G32 = 2, kInt4G64 = 3, kInt4G128 = 4 };

namespace prod {

// Columns of a line (128 bytes of a weight row).
constexpr int line_columns(int kind) { return kind == kBf16 ? 64 : 256; }

// Bytes of a row of x in LDS: whole lines, and 16 so that rows start in
// different banks.
constexpr int64_t x_stride(int kind, int64_t cols)
{
    const int64_t line = line_columns(kind);
    return (cols + line - 1) / line * line * 2 + 16;
}

// Dynamic LDS of a block, at most (its static arrays take 13 KB of the CU's
// 160 KB), and of a small block.
constexpr int64_t kLdsRoom = 131072, kLdsSmall = 65536;

// LDS in which the waves of a team add their sums: two buffers.
constexpr int64_t sums_bytes(int waves, int kw, int tt)
{
    return kw > 1 ? 2 * (int64_t)waves * 2 * tt * 64 * 16 : 0;
}

// Spans of weights that a wave of the eight-wave kernels loads ahead: fewer
// where x (from memory) or the scales take more registers.
constexpr int spans_ahead(int kind, bool direct)
{
    return direct ? (kind == kBf16 ? 4 : 2) : (kind == kInt4G32 ? 2 : 4);
}
constexpr int kSpansSmall = 2;

// INT4 with two row tiles needs more than the 256 registers of eight waves.
constexpr int two_tile_waves(int kind) { return kind >= kInt4G32 ? 4 : 8; }

// Waves of the big blocks (one of eight waves a CU) that run at a time.
constexpr int64_t kAtOnce = 2048;

// Few tiles: blocks of four waves and short rings, two or three to a CU.
// Small blocks' time over big ones', 2048 columns (MXFP4, bf16, INT4):
//   128 tiles  0.78 1.06 0.93   8 us
//   256        0.84 1.03 0.96
//   384        0.97 0.97 1.00
//   512        1.03 1.03 1.07   11, 18, 14 us with big blocks
//   640        1.25 1.19 1.15
//   768        1.31 1.19 1.19
//   1984       1.68 1.13 1.45   17, 41, 23 us
//   8192       1.62 1.41 1.67
constexpr int64_t kSmallTiles = 512;

enum Path {
    kPathNone = 0,      // no rows
    kPathSmall = 1,     // blocks of four waves
    kPathOneTile = 2,   // of eight, 16 rows of x at a time
    kPathMemory = 3,    // the same, x from memory
    kPathTwoTiles = 4   // 32 rows at a time
};

struct Shape {
    Path path;
    int kw;             // waves that share a tile's columns
    int64_t rows;       // rows of an expert that are multiplied at once
    int64_t room;       // LDS for x and the sums
    int64_t tiles;      // of all experts' passes, if their rows are spread evenly
};

// experts: 1 for a dense product; rows: of all experts (pairs, for a layer);
// units: outputs, of which a tile holds 16 with a gate and else 32; planes: 2
// where x comes in two terms.
inline Shape choose_shape(int kind, bool gate, int planes, int64_t cols, int64_t units, int64_t experts,
                          int64_t rows)
{
    Shape s = {kPathNone, 1, 0, 0, 0};
    if (rows <= 0) return s;
    if (experts > rows) experts = rows;
    const int64_t likely = (rows + experts - 1) / experts;     // rows of an expert
    const int tt = likely > 16 ? 2 : 1;
    const int64_t passes = experts * ((likely + 16 * tt - 1) / (16 * tt));
    s.tiles = passes * ((units + (gate ? 15 : 31)) / (gate ? 16 : 32));
    const int64_t stride = planes * x_stride(kind, cols);
    const int64_t row_bytes = kind == kBf16 ? 2 * cols : cols / 2;
    // waves of a team: as long as all waves' work fits the GPU at once
    auto waves_per_tile = [&](int most, int spans, int64_t at_once) {
        const int64_t blocks = (row_bytes / 64 + spans - 1) / spans;
        int kw = 1;
        while (kw < most && kw * 2 <= blocks && s.tiles * kw * 2 <= at_once) kw *= 2;
        return kw;
    };
    if (tt == 1 && s.tiles < kSmallTiles) {
        s.kw = waves_per_tile(4, kSpansSmall, 4 * kAtOnce);
        const int64_t fit = (kLdsSmall - sums_bytes(4, s.kw, 1)) / stride;
        if (fit >= likely) {
            s.path = kPathSmall;
            s.rows = fit < 16 ? fit : 16;
            s.room = kLdsSmall;
            return s;
        }
    }
    s.kw = waves_per_tile(8, spans_ahead(kind, false), kAtOnce);
    s.room = kLdsRoom;
    const int64_t fit = (kLdsRoom - sums_bytes(8, s.kw, tt)) / stride;     // rows of x in LDS
    if (fit < (likely < 16 ? likely : 16)) {
        s.path = kPathMemory;
        s.rows = 16;
    } else if (tt == 1) {
        s.path = kPathOneTile;
        s.rows = fit < 16 ? fit : 16;
    } else {
        s.path = kPathTwoTiles;
        s.rows = fit < 32 ? fit : 32;
        if (s.kw > two_tile_waves(kind)) s.kw = two_tile_waves(kind);
    }
    return s;
}

// ---- a layer's down projection of a handful of tokens ------------------------

constexpr int kFewWaves = 16;
constexpr int kFewTokens = 16;      // rows of the operand

// Pairs up to which it is no slower than the general kernel and the sum behind
// it.  Its time of a layer over theirs (2048 x 768, 512 or 256):
//   pairs            4     8        16 and 20   32          48
//   MXFP4            0.77  0.83     0.85-0.97   0.91-0.98   1.01
//   bf16             0.89  0.91     0.81-0.91   0.99-1.05   1.04-1.07
//   INT4, 128        0.74  0.86     0.88-1.03   0.97-1.03   1.02-1.04
//   INT4, 64         0.83  1.02     1.03-1.24   1.03-1.10   1.09
//   INT4, 32         0.84  0.98     1.00-1.17   1.07-1.12   1.13-1.15
// (the scales of small groups are loaded one by one here).
constexpr int few_pairs(int kind) { return kind == kInt4G32 || kind == kInt4G64 ? 8 : 32; }

// Its LDS: the pairs' activations in two terms, or the waves' sums.
constexpr int64_t few_bytes(int kind, int64_t pairs, int64_t cols)
{
    const int64_t x = 2 * pairs * x_stride(kind, cols), red = (int64_t)kFewWaves * 64 * 16;
    return x > red ? x : red;
}

constexpr bool few_fits(int kind, int64_t tokens, int64_t pairs, int64_t cols)
{
    return pairs <= few_pairs(kind) && tokens <= kFewTokens && few_bytes(kind, pairs, cols) <= kLdsSmall;
}

}  // namespace prod
}  // namespace epk
