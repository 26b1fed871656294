// lm_launch.hpp -- grid of a tiled product's launch, shared by the three operand layouts.
#pragma once

#include "ag_internal.hpp"
#include "lm_tile.hpp"

#include <algorithm>

namespace ag {
namespace lm {

// Workgroups of a launch: one per tile, but with groups of rows, whose tile count only the device
// knows, no more than stay resident (each walks the tiles in steps of the grid).
template <typename Kernel>
hipError_t launch_tiles(Kernel kernel, int bm, int bn, int per_cu, TileArgs& a, hipStream_t stream)
{
    a.tiles_m = (a.M + bm - 1) / bm;
    a.tiles_n = (a.N + bn - 1) / bn;
    int cus = 0;
    hipError_t e = device_cus(&cus);
    if (e != hipSuccess)
        return e;
    int64_t tiles = a.tiles_m * a.tiles_n * a.splits;
    if (a.group == kGroupRows)
        tiles = (a.tiles_m + a.E + 1) * a.tiles_n;
    else if (a.group == kGroupK)
        tiles *= a.E;
    if (tiles <= 0)
        return hipSuccess;
    const int64_t grid = std::min<int64_t>(tiles, (int64_t)cus * per_cu);
    kernel<<<dim3((unsigned)grid), dim3(NT), 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace lm
}  // namespace ag
