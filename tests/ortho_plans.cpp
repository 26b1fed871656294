// lm_ortho.hip's host code with what its plans choose laid open, in place of lm_ortho.hip beside lm_launches.cpp.  Compiled
// and driven by ortho_plans.py.
#include "../allgather_gemm_amd/csrc/lm_ortho.hip"

// epi: 0 X X^T, 1 A A, 2 B X, for E matrices of padded extents; out: width of the tiles, tiles in quarters, parts of a reduction, and
// how many tiles there are
extern "C" void plan_of(int epi, int64_t E, int64_t M, int64_t N, int64_t K, int64_t* out)
{
    const OrthoTiles t = plan_tiles(epi == 0 ? kEpiGram : epi == 1 ? kEpiSquare : kEpiUpdate, E, M, N, K);
    out[0] = t.size;
    out[1] = t.cut;
    out[2] = t.splits;
    out[3] = t.all;
}
