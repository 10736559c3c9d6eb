// Which kernel serves a product in 8-bit integers (host side, no HIP): the
// choice that matmul.hip launches by and that ep_probe_matmul_path tells.
#pragma once

#include <stdint.h>

namespace epk {
namespace mm {

constexpr int kStep = 128;          // columns of a step of the tiled kernels

enum Path {
    kPathNone = 0,      // no rows
    kPathFew = 1,       // the few-row kernels of product.hpp
    kPathTile64 = 2,    // tiles of 64 rows x 128 outputs (64 with a gate)
    kPathTile128 = 3,   // 128 x 128
    kPathTile256 = 4    // 256 x 256
};

// Buffers of columns on their way (stages) of the tiled kernels.
constexpr int stages(Path p) { return p == kPathTile64 ? 3 : 2; }

// cols, rows of the weight matrix; experts: 1 for a dense product; rows: of all
// experts.
inline Path choose_path(bool gate, int64_t cols, int64_t units, int64_t experts, int64_t rows)
{
    if (rows <= 0) return kPathNone;
    if (experts > rows) experts = rows;
    const int64_t likely = (rows + experts - 1) / experts;      // rows of an expert
    // the tiled kernels keep the scales of two tiles, and a tile of fewer steps
    // than that would have those of a third on their way
    const int64_t steps = (cols + kStep - 1) / kStep;
    if (likely <= 32 || steps <= stages(kPathTile64)) return kPathFew;
    if (likely <= 64) return kPathTile64;
    const int64_t outputs = gate ? 2 * units : units;
    const int64_t tiles256 = experts * ((likely + 255) / 256) * ((outputs + 255) / 256);
    const int64_t tiles128 = experts * ((likely + 127) / 128) * ((outputs + 127) / 128);
    if (likely >= 512 && tiles256 >= 256) return kPathTile256;
    return tiles128 >= 512 ? kPathTile128 : kPathTile64;
}

}  // namespace mm
}  // namespace epk
