// lm_internal.hpp -- host-side interface between the entry points of the language-model operators
// (lm_api.hip) and their kernels (lm_nt.hip, lm_nn.hip, lm_tn.hip, lm_small.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace ag {

namespace lm {

constexpr int kMaxGroups = 1024;
constexpr int kRowsMost = 64;        // rows of X that the few-rows kernel takes at a time
// Workgroups of 256 threads in a launch: HIP counts its threads along x in 32 bits.  (A multiple of the 8 XCDs.)
constexpr int64_t kMostWorkgroups = (1 << 24) - 8;

enum Act { kActNone = 0, kActRelu = 1, kActSilu = 2, kActGelu = 3, kActGeluTanh = 4 };
enum Group { kGroupRows = 1, kGroupK = 2 };     // 0: no groups
enum Epi { kEpiLinear = 0, kEpiStat = 1, kEpiGrad = 2, kEpiSum = 3, kEpiScaled = 4 };
// kTile128: four stages, one workgroup a CU; kTileShort: 128 x 128 with one stage, a workgroup for each tile and
// four of them on a CU, no groups
enum Tile { kTile256 = 0, kTile128 = 1, kTile32 = 2, kTileShort = 3 };

// C = act(sum + bias) + residual, pre = sum + bias (pre, bias, residual may be null)
struct LinearOut {
    __bf16* C;
    const __bf16* bias;
    const __bf16* residual;
    __bf16* pre;
    int64_t ldc;
    int act;
};

struct TileArgs {
    const __bf16 *A, *B;
    int64_t lda, ldb;        // row strides in elements, multiples of 8
    int64_t M, N, K;
    int64_t k_valid;         // rows that a (K, N) B has where X's rows are zero-padded to K (launch_nn)
    int64_t tiles_n;
    // groups: rows [ends[e-1], ends[e]) of A (kGroupRows), or of the reduction (kGroupK; out.C of
    // group e starts at e * M * ldc)
    const int32_t* ends;
    int E, group;
    int64_t strideB;         // elements from one group's B to the next
    // split reduction: split s takes K steps [s * split_steps, ...) and writes its fp32 sums to
    // part + s * M * ldp
    int splits;
    int64_t split_steps;
    float* part;
    int64_t ldp;             // multiple of 8
    int accumulate;          // add to part instead of writing it
    LinearOut out;
    int plain;               // nothing follows the sums but their rounding into out.C (filled in at the launch)
    // softmax statistics of each row's columns: stat[row][stat_n][2] = (maximum, sum of exponentials)
    float* stat;
    int64_t stat_n;
    float* hit;              // the target's logit
    const int64_t* targets;
    // d logits into out.C, in units of a value of dloss (loss_unit); launch_nn, launch_tn: the sums are in units of it
    // where dloss_rows > 0, and so is what goes to `part`
    const float* lse;
    const float* dloss;
    int64_t dloss_rows;
    int64_t vocab, col0;     // size of the vocabulary; its first column in this piece
};

constexpr int kStatCols = 64;      // columns that one statistics pair of a tiled product covers

// X (M, K) Y (N, K); X (M, K) Y (K, N); X (K, M) Y (K, N).  tiles_n is filled in here.
hipError_t launch_nt(Tile t, Epi epi, TileArgs a, hipStream_t stream);
// X (M, K) Y (N, K) for few rows (a.M, or a group's, about `rows`); out.part is not used.
int rows_cols(int64_t N, int64_t rows);     // columns that one of its statistics pairs covers
hipError_t launch_rows(Epi epi, int64_t rows, TileArgs a, hipStream_t stream);
hipError_t launch_nn(Tile t, TileArgs a, hipStream_t stream);
hipError_t launch_tn(Tile t, TileArgs a, hipStream_t stream);

// out = epilogue of the sum over splits of part[s][row][col], in units of a value of dloss where dloss_rows > 0
hipError_t launch_join(const float* part, int splits, int64_t M, int64_t N, int64_t ldp, const LinearOut& out,
                       hipStream_t stream, const float* dloss = nullptr, int64_t dloss_rows = 0);

// d (M, ldd) = dC act'(pre), columns [N, ldd) zero (d may be null); dbias: null, or with colsum_rows(M) == 1 the
// column sums of the unrounded products, with more colsum gets [colsum_rows(M)][N] partial ones in fp32
int64_t colsum_rows(int64_t M);
hipError_t launch_act_bwd(const __bf16* dC, const __bf16* pre, int act, int64_t M, int64_t N, __bf16* d, int64_t ldd,
                          float* colsum, __bf16* dbias, hipStream_t stream);
hipError_t launch_colsum_join(const float* colsum, int64_t rows, int64_t N, __bf16* out, hipStream_t stream);

// lse and loss of each row from its statistics
hipError_t launch_xent_join(const float* stat, int64_t stat_n, const float* hit, const int64_t* targets, int64_t T,
                            int64_t vocab, float* loss, float* lse, hipStream_t stream);

}  // namespace lm
}  // namespace ag
