// Which kernel serves a product in 8-bit integers (host side, no HIP): the
// choice that matmul.hip launches by and that ep_probe_matmul_path tells.
#pragma once

#include <stdint.h>

namespace epk {
namespace mm {

constexpr int kStep = 128;          // columns of a step of the tiled kernels
constexpr int kThinWaves = 8;       // waves of a block of the thin kernel

enum Path {
    kPathNone = 0,          // no rows
    kPathFew = 1,           // the few-row kernels of product.hpp
    kPathThin = 2,          // one matrix, few rows and outputs
    kPathTile64x64 = 3,     // tiles of 64 rows of x and 64 weight rows
    kPathTile64x128 = 4,
    kPathTile128 = 5,       // 128 x 128
    kPathTile256 = 6        // 256 x 256
};

// Buffers of columns on their way (stages) of the tiled kernels, and of tiles'
// scales.  Loads run S - 1 steps ahead of the arithmetic, a tile's scales are loaded
// behind the last columns of the tile before; with B buffers they overwrite those
// of B tiles before, whose arithmetic is then over if (B - 1) * steps > S - 1.
constexpr int stages(Path p) { return p == kPathTile64x64 ? 4 : p == kPathTile64x128 ? 3 : 2; }
constexpr int scale_buffers(int S) { return S == 2 ? 3 : 2; }
constexpr bool enough_steps(Path p, int64_t steps) { return (scale_buffers(stages(p)) - 1) * steps > stages(p) - 1; }

// All figures of this choice, the number of blocks at once and the band of the thin
// kernel's pairs among them, are for 256 CUs.  On another number every call is right
// all the same: only the launches, which take the CUs that there are, differ.
//
// The tiled kernels' time, in steps of a 256 x 256 tile (1.8 us): a step of a
// round of tiles (one or two blocks to each CU) and what a round costs beside its
// steps.  Measured, in us, with 7168 columns and no gate where one expert:
//   rows x outputs          64x64  64x128  128x128  256x256
//   64 x 4096                  21      30       37       64
//   256 x 4096                 22      30       41       89
//   512 x 4096                 26      31       41       89
//   1024 x 4096                49      40       42       89
//   2048 x 4096               101      83       60       91
//   4096 x 4096                        155      113      100
//   64 experts, 2048 columns, 2 x 768 outputs with the gate, rows an expert:
//   16                         42      39       44       54
//   64                         57      50       46       58
//   128                        83      69       64       65
//   256                       144     110       88       97
//   512                       255     190      149      137
struct TileCost {
    Path path;
    int bm, bn, at_once;    // blocks that 256 CUs hold
    float alone, step;      // a step, with one block a CU and with all
    float round;
};
constexpr TileCost kTileCosts[] = {
    {kPathTile64x64, 64, 64, 512, 0.21f, 0.27f, 0.4f},
    {kPathTile64x128, 64, 128, 512, 0.295f, 0.40f, 0.5f},
    {kPathTile128, 128, 128, 512, 0.41f, 0.59f, 0.8f},
    {kPathTile256, 256, 256, 256, 1.0f, 1.0f, 2.0f},
};

// Weight tiles of 16 rows for each 16 rows of x.
inline int64_t thin_tiles(bool gate, int64_t units, int64_t rows)
{
    return (rows + 15) / 16 * ((units + 15) / 16) * (gate ? 2 : 1);
}

// A lane offset past every buffer: reads 0.
constexpr uint32_t kNowhere = 0x80000000u;

// Group g of the thin kernel's block whose outputs begin at unit0: its first weight
// row and how many it has.  A group behind the last output takes the block's first
// (which is not stored twice): a buffer of no rows there is no bound, since the
// hardware compares lane offsets with its size less the scalar offset, which wraps.
struct ThinGroup {
    int first, have;
};
constexpr ThinGroup thin_group(int unit0, int g, int units)
{
    const int u = unit0 + 16 * g < units ? unit0 + 16 * g : unit0;
    return {u, units - u < 16 ? units - u : 16};
}

// Lane offset of weight load v (rows 8 v to 8 v + 7) of a line, of which `left`
// columns are in the row.
constexpr uint32_t thin_offset(int lane, int v, int cols, int left)
{
    return 16 * (lane >> 3) < left ? (uint32_t)(8 * v + (lane & 7)) * (uint32_t)cols + 16u * (lane >> 3) : kNowhere;
}

// One behind the last byte of a gateless matrix that the thin kernel's weight loads
// can read with `groups` groups a block, taking the bound as it wraps.
inline int64_t thin_reach(int groups, int cols, int units)
{
    int64_t most = 0;
    const int lines = (cols + 127) / 128, outputs = 16 * groups, last = (units - 1) / outputs * outputs;
    for (int unit0 = last >= outputs ? last - outputs : last; unit0 <= last; unit0 += outputs)
        for (int g = 0; g < groups; ++g) {
            const ThinGroup at = thin_group(unit0, g, units);
            for (int line = 0; line < lines; ++line)
                for (int i = 0; i < 128; ++i) {
                    const uint32_t off = thin_offset(i / 2, i % 2, cols, cols - 128 * line), scalar = 128u * line;
                    if (off >= (uint32_t)at.have * (uint32_t)cols - scalar) continue;
                    const int64_t to = (int64_t)at.first * cols + off + scalar + 16;
                    most = to > most ? to : most;
                }
        }
    return most;
}

// cols, units of the weight matrix; experts: 0 for one matrix; rows: of all
// experts.
inline Path choose_path(bool gate, int64_t cols, int64_t units, int64_t experts, int64_t rows)
{
    if (rows <= 0) return kPathNone;
    const bool grouped = experts > 0;
    if (!grouped) experts = 1;
    if (experts > rows) experts = rows;
    const int64_t likely = (rows + experts - 1) / experts;      // rows of an expert
    const int64_t outputs = gate ? 2 * units : units;
    const int64_t steps = (cols + kStep - 1) / kStep;
    // the thin kernel's time follows its weight tiles of 16, 64 x 64 tiles' hardly
    // does below 256: us with 7168 columns (and 2048), 1 to 16 rows:
    //   tiles    256             512             640             896
    //   thin     8.3-10 (4.5-5)  13-14 (6-7)     18-23 (7-9)     21-26 (9-10)
    //   64 x 64  21     (7.8)    21    (7.8)     22    (8.6)     22    (9.0)
    if (!grouped && rows <= 32 && thin_tiles(gate, units, rows) <= 640) return kPathThin;
    // decode batches of many experts: 256 experts, 7168 -> 2048, 4, 8, 12 rows an
    // expert 554, 572, 668 us, with 64 x 128 tiles 610, 618, 626; 64 experts, 2048
    // -> 2 x 768, 8 and 12 rows 37, 42, with tiles 38, 39.  Of few experts that have
    // rows the tiles are faster: one row each of 48, 2048 -> 2 x 768 32 us and 36, of
    // 32, 4096 -> 2 x 1408 68 and 82, of 128, 2048 -> 2 x 768 73 and 67
    if (grouped && likely <= 8 && experts * ((outputs + 127) / 128) >= 1024) return kPathFew;
    // and of few tiles and many columns those kernels are faster, whose waves share
    // the columns: 8 experts of 1 to 8 rows, 4096 -> 67 10 us, with 64 x 64 tiles 15;
    // 7168 -> 2 x 512 18 and 23; 16 rows 27 and 24; 2560 -> 1024 11.1 and 10.8
    if (grouped && likely <= 8 && experts * ((outputs + 31) / 32) <= 256 && steps >= 24) return kPathFew;
    // (two-stage tiles take any number of columns: 4096 rows, 256 -> 4096 13 us, the
    // few-row kernels 37; 128 experts of 64 rows, 256 -> 2048 31 and 55)
    Path best = kPathNone;
    float least = 0.f;
    for (const TileCost& t : kTileCosts) {
        if (!enough_steps(t.path, steps)) continue;
        // an expert's tiles of rows: experts differ, so half a tile more where the
        // mean is near a whole number of them
        const float tiles_m = !grouped ? (float)((likely + t.bm - 1) / t.bm)
                              : 10 * likely <= 8 * t.bm ? 1.f : (float)likely / t.bm + 0.5f;
        const float fill = (float)likely / (tiles_m * t.bm);
        const int64_t tiles = (int64_t)(tiles_m * experts + 0.5f) * ((outputs + t.bn - 1) / t.bn);
        const int64_t whole = tiles / t.at_once, rest = tiles % t.at_once;
        // half of a step's cost goes with the weights, half with the rows there are
        const float step = whole * t.step + (rest == 0 ? 0.f : rest <= 256 ? t.alone : t.step);
        const float cost = step * (0.5f + 0.5f * fill) * steps + (whole + (rest > 0 ? 1 : 0)) * t.round;
        if (best == kPathNone || cost < least) {
            best = t.path;
            least = cost;
        }
    }
    return best;
}

// Tiles of 64 x 64 of one matrix are often fewer than CUs, and what bounds a block
// alone is the way of its columns into LDS (a step 0.36 us, with any number of
// stages); the thin kernel's blocks wait 2 us for each 4096 columns.  With a
// workspace for the sums the columns are split over blocks, at most 256 in all
// (4 MB of sums) and 32 for a tile, eight steps each at least, and a second kernel
// joins them, which costs 6.5 us in all.  In us, alone and split in (n):
//   64 rows   2048 -> 2048  8.6, 9.2 (4)     7168 -> 4096  22, 14 (4)
//             16384 -> 4096  47, 21 (4)      18432 -> 7168  53, 35 (2)
//   16 rows   32768 -> 1024  30, 17 (16)
//   256 rows  4096 -> 4096 (256 tiles)  14.6, 17.5 (2)
//   33 rows   131056 -> 64  345, split in 32, 64, 128: 28, 30, 41
// The second launch also costs its caller some 4 us.
inline int choose_splits(bool gate, int64_t cols, int64_t units, int64_t rows)
{
    const int64_t steps = (cols + kStep - 1) / kStep;
    const int64_t tiles = (rows + 63) / 64 * (((gate ? 2 : 1) * units + 63) / 64);
    if (tiles < 1 || tiles > 128) return 1;
    int64_t n = 256 / tiles < steps / 8 ? 256 / tiles : steps / 8;
    if (n > 32) n = 32;
    if (n < 2) return 1;
    float alone = 1.f + 0.36f * steps;
    if (choose_path(gate, cols, units, 0, rows) == kPathThin) {
        const float all = 3.f + (float)(thin_tiles(gate, units, rows) * 16 * cols) / 4.2e6f, wait = 4.f + cols / 2048.f;
        alone = all > wait ? all : wait;
    }
    return alone > 11.f + 0.36f * ((steps + n - 1) / n) ? (int)n : 1;
}

}  // namespace mm
}  // namespace epk
