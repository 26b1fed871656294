// lm_nn.hip -- X (M, K) times Y (K, N): the gradient of the activations, dA = D B.
#include "lm_launch.hpp"

namespace ag {
namespace lm {
namespace {

template <int EPI>
__global__ __launch_bounds__(NT, 1) void nn256_kernel(TileArgs a)
{
    tile_body<256, 256, 2, 2, 2, false, true, EPI, true>(a);
}

template <int EPI>
__global__ __launch_bounds__(NT, 1) void nn128_kernel(TileArgs a)
{
    tile_body<128, 128, 2, 2, 4, false, true, EPI, false>(a);
}

template <int EPI>
__global__ __launch_bounds__(NT, 4) void nnshort_kernel(TileArgs a)
{
    tile_body<128, 128, 2, 2, 1, false, true, EPI, false>(a);
}

template <int EPI>
__global__ __launch_bounds__(NT, 1) void nn32_kernel(TileArgs a)
{
    tile_body<32, 128, 1, 4, 4, false, true, EPI, false>(a);
}

template <int EPI>
hipError_t launch(Tile t, TileArgs& a, hipStream_t stream)
{
    switch (t) {
    case kTile256: return launch_tiles(nn256_kernel<EPI>, 128, 256, 1, a, stream);
    case kTile32: return launch_tiles(nn32_kernel<EPI>, 32, 128, 1, a, stream);
    case kTileShort: return launch_tiles(nnshort_kernel<EPI>, 128, 128, kEachTile, a, stream);
    default: return launch_tiles(nn128_kernel<EPI>, 128, 128, 1, a, stream);
    }
}

}  // namespace

hipError_t launch_nn(Tile t, TileArgs a, hipStream_t stream)
{
    return a.dloss_rows > 0 && !a.part ? launch<kEpiScaled>(t, a, stream) : launch<kEpiSum>(t, a, stream);
}

}  // namespace lm
}  // namespace ag
