// lm_nt.hip -- X (M, K) times Y (N, K): the forward products (linear, grouped by expert) and the logits.
#include "lm_launch.hpp"

namespace ag {
namespace lm {
namespace {

template <int EPI>
__global__ __launch_bounds__(NT, 1) void nt256_kernel(TileArgs a)
{
    tile_body<256, 256, 2, 2, 2, false, false, EPI, true>(a);
}

template <int EPI>
__global__ __launch_bounds__(NT, 1) void nt128_kernel(TileArgs a)
{
    tile_body<128, 128, 2, 2, 4, false, false, EPI, false>(a);
}

template <int EPI>
__global__ __launch_bounds__(NT, EPI == kEpiLinear ? 3 : 4) void ntshort_kernel(TileArgs a)
{
    tile_body<128, 128, 2, 2, 1, false, false, EPI, false>(a);
}

template <int EPI>
hipError_t launch(Tile t, TileArgs& a, hipStream_t stream)
{
    if (t == kTile256)
        return launch_tiles(nt256_kernel<EPI>, 128, 256, 1, a, stream);
    if (t == kTileShort)
        return launch_tiles(ntshort_kernel<EPI>, 128, 128, kEachTile, a, stream);
    return launch_tiles(nt128_kernel<EPI>, 128, 128, 1, a, stream);
}

}  // namespace

hipError_t launch_nt(Tile t, Epi epi, TileArgs a, hipStream_t stream)
{
    switch (epi) {
    case kEpiStat:
        a.stat_n = (a.N + kStatCols - 1) / kStatCols;
        return launch<kEpiStat>(t, a, stream);
    case kEpiGrad: return launch<kEpiGrad>(t, a, stream);
    default: break;
    }
    // a kernel of its own without what may follow the sums
    const LinearOut& o = a.out;
    const bool sum = a.splits > 1 || !(o.bias || o.pre || o.residual || o.act != kActNone);
    return sum ? launch<kEpiSum>(t, a, stream) : launch<kEpiLinear>(t, a, stream);
}

}  // namespace lm
}  // namespace ag
