// lm_launch.hpp -- grid of a tiled product's launch, shared by the three operand layouts.
#pragma once

#include "ag_internal.hpp"
#include "lm_tile.hpp"

#include <algorithm>

namespace ag {
namespace lm {

constexpr int kEachTile = 1 << 20;             // per_cu: a workgroup for each tile, as far as a launch can have them

// Workgroups of a launch: no more than stay resident, each walks the tiles in steps of the grid.  How many
// tiles groups of rows make only the device knows.
template <typename Kernel>
hipError_t launch_tiles(Kernel kernel, int bm, int bn, int per_cu, TileArgs& a, hipStream_t stream)
{
    a.tiles_n = (a.N + bn - 1) / bn;
    a.plain = !(a.part || a.out.bias || a.out.pre || a.out.residual || a.out.act != kActNone);
    int cus = 0;
    hipError_t e = device_cus(&cus);
    if (e != hipSuccess)
        return e;
    int64_t rows = (a.M + bm - 1) / bm;        // bm: of the lowest tile
    if (a.group == kGroupRows)
        rows += a.E + 1;
    const int64_t tiles = rows * a.tiles_n * (a.group == kGroupK ? a.E : a.splits);
    if (tiles <= 0)
        return hipSuccess;
    // the smallest tiles are 128 wide
    const int64_t grid = std::min({tiles * (bn / 128), (int64_t)cus * per_cu, kMostWorkgroups});
    kernel<<<dim3((unsigned)grid), dim3(NT), 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace lm
}  // namespace ag
