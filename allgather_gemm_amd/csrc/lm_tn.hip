// lm_tn.hip -- X (K, M) times Y (K, N): the gradient of the weight, dB = D^T A.
#include "lm_launch.hpp"

namespace ag {
namespace lm {
namespace {

template <int EPI>
__global__ __launch_bounds__(NT, 1) void tn256_kernel(TileArgs a)
{
    tile_body<256, 256, 2, 2, 2, true, true, EPI, true>(a);
}

template <int EPI>
__global__ __launch_bounds__(NT, 1) void tn128_kernel(TileArgs a)
{
    tile_body<128, 128, 2, 2, 4, true, true, EPI, false>(a);
}

template <int EPI>
__global__ __launch_bounds__(NT, 4) void tnshort_kernel(TileArgs a)
{
    tile_body<128, 128, 2, 2, 1, true, true, EPI, false>(a);
}

template <int EPI>
hipError_t launch(Tile t, TileArgs& a, hipStream_t stream)
{
    switch (t) {
    case kTile256: return launch_tiles(tn256_kernel<EPI>, 128, 256, 1, a, stream);
    case kTileShort: return launch_tiles(tnshort_kernel<EPI>, 128, 128, kEachTile, a, stream);
    default: return launch_tiles(tn128_kernel<EPI>, 128, 128, 1, a, stream);
    }
}

}  // namespace

hipError_t launch_tn(Tile t, TileArgs a, hipStream_t stream)
{
    return a.dloss_rows > 0 && !a.part ? launch<kEpiScaled>(t, a, stream) : launch<kEpiSum>(t, a, stream);
}

}  // namespace lm
}  // namespace ag
