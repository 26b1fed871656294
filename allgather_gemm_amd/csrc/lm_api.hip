// lm_api.hip -- entry points of the language-model operators declared in include/aggemm.h: argument
// checks, the plan of each product (tile, splits, workspace layout) and the launches.  They keep no
// state: the workspace is the caller's, so calls on different streams are independent and a call can
// be captured into a graph.
#include "../../include/aggemm.h"
#include "ag_internal.hpp"
#include "lm_internal.hpp"

#include <algorithm>

namespace ag {
namespace lm {
namespace {

constexpr int64_t kMaxDim = 1 << 21;              // columns of any operand: 32-bit tile offsets
constexpr int64_t kMaxRows = (int64_t)1 << 30;
constexpr int64_t kPieceBytes = 512 << 20;        // d logits held at a time

#define LM_HIP(call, what)               \
    do {                                 \
        hipError_t e_ = (call);          \
        if (e_ != hipSuccess)            \
            return hip_error(e_, what);  \
    } while (0)

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
// a tensor that must be there when it has elements
bool bad(const void* p, int64_t elements, uintptr_t n = 16) { return (elements > 0 && !p) || !aligned(p, n); }
int64_t up(int64_t x, int64_t n) { return (x + n - 1) / n * n; }
int64_t region(int64_t bytes) { return up(bytes, 256); }

int64_t cus()
{
    int n = 0;
    if (device_cus(&n) != hipSuccess || n <= 0)
        n = 256;
    return n;
}

// One product (M, N, K): its tile and how many parts the reduction is split into.
struct Plan {
    Tile tile;
    int splits;
    int64_t split_steps;
    int64_t part_bytes(int64_t M, int64_t N) const { return splits > 1 ? region(splits * M * up(N, 8) * 4) : 0; }
};

// What follows a product's sums, for the time that it adds to a tile.
enum After { kSum = 0, kStatistics = 1, kActivation = 2 };

// Time of one product's tiles, us, by rates measured on this card.  A 256 x 256 tile takes 1.6 us for a step of 64
// and 7 us besides, its half 0.9 and 4, its quarter and a 128 x 128 tile 0.44 and 3 (a fifth more once there is more
// than a round of them, for they read twice as much per product out of the caches).  Short tiles, four a CU at a time,
// take 0.49 and 1 each (0.6 where there are fewer), but 0.94 a step for one that is alone.  What follows the sums is
// the more expensive the fewer workgroups a CU has to cover it.  (us, large | short tiles: 16384 x 4096 x 512 81 | 75,
// with gelu 144 | 120; 16384 x 4096 x 128 46 | 36, 104 | 76; 8192 x 8192 x 1024 129 | 140, 191 | 174; 128 x 128 |
// short: 2048 x 2048 x 2048 22 | 36.)
double tile_time(Tile t, int64_t M, int64_t N, int64_t steps, int64_t parts, int64_t n, After after)
{
    static const double kAfter[3][4] = {{0, 0, 0, 0}, {3, 1.6, 1.5, 0.3}, {12, 6.5, 3.5, 2.4}};
    const double* const more = kAfter[after];
    if (t == kTile128 || t == kTileShort) {
        const int64_t tiles = ((M + 127) / 128) * ((N + 127) / 128) * parts;
        if (t == kTile128)
            return (double)((tiles + n - 1) / n) * (0.44 * steps + 3 + more[2]) * (tiles > n ? 1.2 : 1.0);
        const double each = 0.49 * steps + 1 + more[3], fours = (double)(tiles / (4 * n) * 4);
        const double rest = (double)tiles / n - fours;
        return fours * each + (rest > 0 ? std::max(0.94 * steps + 3, rest * (each + 0.11 * steps)) : 0);
    }
    const int64_t c = (N + 255) / 256 * parts, units = M / 256 + (M % 256 > 128), lone = M % 256 > 0 && M % 256 <= 128;
    const double full = 1.6 * steps + 7 + more[0], half = 0.9 * steps + 4 + more[1];
    const int64_t rounds = units * c / n, last = units * c % n;
    // the tail as the kernel chooses it: whole, in halves or in quarters
    const double quarter = 0.44 * steps + 3 + more[2];
    const int64_t cq = (N + 127) / 128 * parts;
    const auto halves = [&](int64_t tiles) { return (double)((std::max<int64_t>(0, tiles) + n - 1) / n) * half; };
    const auto quarters = [&](int64_t tiles) {
        return (double)((std::max<int64_t>(0, tiles) + n - 1) / n) * quarter * (tiles > n ? 1.2 : 1.0);
    };
    double tail = std::min(halves(lone * c), quarters(lone * cq));
    if (last > 0) {
        const int64_t d = (last + c - 1) / c, idle = d * c - last;
        tail = full + std::min(halves(lone * c - 2 * (n - last)), quarters(lone * cq - 3 * (n - last)));
        tail = std::min(tail, halves((lone + 2 * d) * c - 2 * idle));
        tail = std::min(tail, quarters((lone + 2 * d) * cq - 3 * idle));
    }
    return rounds * full + tail;
}

// The tile and the split that take the least time.  A split product writes and reads its fp32 sums, at 2.7 TB/s, and
// joining them is a launch.  (us, 128 x 128 against 256 x 256: 2048 x 2048 x 2048 23 | 31, 1024 x 4096 x 4096 37 | 52,
// 3000 x 3000 x 3000 100 | 90; 128 x 4096 x 4096 33 in one part, 18.5 in four.)
Plan plan_product(int64_t M, int64_t N, int64_t K, After after, bool split = true, bool grouped = false)
{
    Plan p;
    const int64_t steps = std::max<int64_t>(1, (K + 63) / 64), n = cus();
    int64_t parts = 1;
    p.tile = kTile128;
    double best = 1e30;
    for (const Tile t : {kTile128, kTile256, kTileShort}) {
        if (t == kTileShort && grouped)
            break;
        for (const int64_t s : {1, 2, 3, 4, 6, 8, 12, 16, 24, 32}) {
            if (s > 1 && (!split || t == kTileShort || s * 2 > steps))
                break;
            const double us =
                tile_time(t, M, N, (steps + s - 1) / s, s, n, s > 1 ? kSum : after) + (s > 1 ? 4 + 3e-6 * s * M * N : 0);
            if (us < best) {
                best = us;
                p.tile = t;
                parts = s;
            }
        }
    }
    p.split_steps = (steps + parts - 1) / parts;
    p.splits = (int)((steps + p.split_steps - 1) / p.split_steps);
    return p;
}

// A linear layer's: split by its extents alone, which are what its workspace is asked for with.
Plan plan_linear(int64_t M, int64_t N, int64_t K, After after)
{
    const Plan p = plan_product(M, N, K, kSum);
    return p.splits > 1 || after == kSum ? p : plan_product(M, N, K, after, false);
}

// Whether a linear layer is for the few-rows kernel, each of whose workgroups goes through all of K for its columns: long
// reductions are split over tiles instead, which takes a second launch.  Tiles | few rows, us on the device.  16 columns a
// workgroup, 97 | 1000 columns: 1 row, K = 8192 9.0 | 7.8, 9.9 | 8.1, K = 32768 12.7 | 18.7, 17.2 | 18.9; 16 rows,
// K = 4096 8.9 | 9.2, 9.9 | 9.4, K = 8192 9.6 | 13.4, 10.9 | 13.6; 32 rows, K = 2048 8.7 | 9.7, 9.5 | 10.0, K = 4096
// 9.1 | 14.2, 10.2 | 14.4; 64 rows, K = 1024 8.8 | 10.4, 9.8 | 10.8, K = 2048 8.8 | 12.8, 10.5 | 13.1 (the launch saved
// is worth 3 us to a host that waits for nothing else: 64 rows, K = 1024 13.1 | 10.0, K = 2048 12.8 | 12.5).  64 columns
// a workgroup, 4600 | 10000 | 14336 columns: 32 rows, K = 4096 13.8 | 15.8, 20.4 | 17.1, 24.4 | 20.3, K = 8192
// 19.0 | 27.7, 30.9 | 32.1, 39.5 | 37.4; 64 rows, K = 2048 13.4 | 12.1, 15.9 | 13.6, 16.0 | 13.7, K = 4096 15.3 | 20.5,
// 21.7 | 21.6, 25.6 | 23.2, K = 16384 30.9 | 68.2, 68.8 | 99.8, 106.6 | 116.6.
bool few_linear(int64_t M, int64_t N, int64_t K)
{
    if (M > kRowsMost)
        return false;
    if (rows_cols(N, M) == 16)
        return K * std::max<int64_t>(M, 4) <= 1 << 16;
    return K * std::max<int64_t>(M, 32) <= 1 << 17 || (N + 63) / 64 * 4 >= cus() * 3;
}

// The same for X (M, K) times Y (K, N), whose few rows have a tile of 32 rows, a workgroup for each CU as far as parts of
// four steps allow.  128 x 128 tiles by their plan | 32 rows, us: 1 | 32 rows of N = 1024, K = 512 7.1, 7.3 | 6.6, 7.3,
// K = 8192 9.7, 12.2 | 7.7, 10.4; N = 4096, K = 2048 10.0, 12.0 | 8.0, 10.4, K = 32000 45.2, 47.5 | 44.8, 46.7; N = 14336,
// K = 64 5.0, 5.3 | 4.0, 4.1, K = 512 7.7, 8.1 | 7.6, 9.5, K = 8192 40.7, 41.6 | 39.6, 40.2.  With 48 rows, two tiles of
// 32: N = 4096, K = 2048 12.5 | 14.0, K = 32000 48.2 | 52.7.  Parts of at least eight steps: K = 512 5.3, 5.4 instead of
// 6.6, 7.3 (one part, no join), K = 2048 7.7, 8.2 instead of 7.1, 7.8 at N = 1024.
Plan plan_nn(int64_t M, int64_t N, int64_t K)
{
    if (M > 32)
        return plan_product(M, N, K, kSum);
    Plan p;
    p.tile = kTile32;
    const int64_t steps = std::max<int64_t>(1, (K + 63) / 64);
    const int64_t parts = std::max<int64_t>(1, std::min(cus() / std::max<int64_t>(1, (N + 127) / 128), steps / 4));
    p.split_steps = (steps + parts - 1) / parts;
    p.splits = (int)((steps + p.split_steps - 1) / p.split_steps);
    return p;
}

TileArgs product(const void* A, int64_t lda, const void* B, int64_t ldb, int64_t M, int64_t N, int64_t K, void* C,
                 int64_t ldc)
{
    TileArgs a = {};
    a.A = static_cast<const __bf16*>(A);
    a.B = static_cast<const __bf16*>(B);
    a.lda = lda;
    a.ldb = ldb;
    a.M = M;
    a.N = N;
    a.K = K;
    a.k_valid = K;
    a.splits = 1;
    a.out.C = static_cast<__bf16*>(C);
    a.out.ldc = ldc;
    return a;
}

// Launches a product by its plan; a split one is joined through `part`.
template <typename Launch>
hipError_t run_product(Launch launch, const Plan& p, TileArgs a, void* part, hipStream_t s)
{
    if (p.splits > 1) {
        a.splits = p.splits;
        a.split_steps = p.split_steps;
        a.part = static_cast<float*>(part);
        a.ldp = up(a.N, 8);
    }
    hipError_t e = launch(p.tile, a, s);
    if (e == hipSuccess && p.splits > 1)
        e = launch_join(a.part, p.splits, a.M, a.N, a.ldp, a.out, s);
    return e;
}

hipError_t nt_linear(Tile t, const TileArgs& a, hipStream_t s) { return launch_nt(t, kEpiLinear, a, s); }

struct LinearBwd {
    bool own_d;              // d = dC act'(pre) is written to the workspace
    int64_t ldd;
    Plan da, db;
    int64_t d_bytes, sum_bytes, part_bytes;
    int64_t bytes() const { return d_bytes + sum_bytes + part_bytes; }
};

LinearBwd plan_linear_bwd(int64_t M, int64_t Nc, int64_t K, int act)
{
    LinearBwd w;
    w.own_d = act != kActNone || Nc % 8 != 0;
    w.ldd = up(Nc, 8);
    w.da = plan_nn(M, K, w.ldd);
    w.db = plan_product(Nc, K, M, kSum);
    w.d_bytes = w.own_d ? region(M * w.ldd * 2) : 0;
    w.sum_bytes = colsum_rows(M) > 1 ? region(colsum_rows(M) * Nc * 4) : 0;
    w.part_bytes = std::max(w.da.part_bytes(M, K), w.db.part_bytes(Nc, K));
    return w;
}

// Whether the logits of T rows are for the few-rows kernel: up to kRowsMost always, and any number of them where there
// is at most one of its 64 x 64 tiles for a CU, or two in a reduction of up to 16 steps: two on a CU share its way to
// the caches.  128 x 128 | 64 x 64, us.  At most one, statistics and join: T = 384, V = 1003, K = 256 10.2 | 8.2,
// K = 4096 30.0 | 24.1; T = 2048, V = 500, K = 256 10.6 | 8.7, K = 4096 31.7 | 27.6; T = 16384, V = 64, K = 2048
// 23.4 | 21.9.  Two, loss and gradients: T = 200, V = 4427, K = 1024 49.0 | 45.8, K = 2048 63.7 | 69.8; T = 1024,
// V = 2048, K = 1024 56.5 | 53.6, K = 2048 69.9 | 72.1; T = 4096, V = 500, K = 512 60.6 | 56.3, K = 1024 66.1 | 69.2.
bool few_rows(int64_t T, int64_t V, int64_t K)
{
    if (T <= kRowsMost)
        return true;
    const int64_t tiles = (T + kRowsMost - 1) / kRowsMost * ((V + 63) / 64);
    return tiles <= (K <= 16 * 64 ? 2 : 1) * cus();
}

Tile xent_tile(int64_t T, int64_t V, int64_t K) { return plan_product(T, V, K, kStatistics, false).tile; }

int64_t stat_pairs(int64_t T, int64_t V, int64_t K)
{
    if (few_rows(T, V, K)) {
        const int cols = rows_cols(V, T);
        return (V + cols - 1) / cols;
    }
    return (V + kStatCols - 1) / kStatCols;
}

hipError_t launch_logits(Epi epi, const TileArgs& a, hipStream_t s)
{
    return few_rows(a.M, a.N, a.K) ? launch_rows(epi, a.M, a, s) : launch_nt(xent_tile(a.M, a.N, a.K), epi, a, s);
}

struct XentBwd {
    int64_t piece;           // columns of the vocabulary at a time, a multiple of 256
    int64_t pieces;
    Plan da;
    bool part;               // dA is summed in fp32 in the workspace
    int64_t part_bytes;
    int64_t bytes(int64_t T) const { return region(T * piece * 2) + part_bytes; }
};

XentBwd plan_xent_bwd(int64_t T, int64_t V, int64_t K, int64_t piece)
{
    XentBwd w;
    w.piece = piece;
    w.pieces = (V + piece - 1) / piece;
    w.da = plan_nn(T, K, std::min(up(V, 8), piece));
    w.part = w.pieces > 1 || w.da.splits > 1;
    w.part_bytes = w.part ? region((int64_t)w.da.splits * T * K * 4) : 0;
    return w;
}

// Equal pieces of at most kPieceBytes of d logits; fewer columns, down to 256, where the workspace is
// smaller than that.
XentBwd plan_xent_bwd_in(int64_t T, int64_t V, int64_t K, int64_t room)
{
    const int64_t most = std::max<int64_t>(256, kPieceBytes / std::max<int64_t>(1, T * 2) / 256 * 256);
    for (int64_t n = (V + most - 1) / most;; ++n) {
        const XentBwd w = plan_xent_bwd(T, V, K, up((V + n - 1) / n, 256));
        if (w.piece == 256 || w.bytes(T) <= room)
            return w;
    }
}

bool shapes_ok(int64_t M, int64_t Nc, int64_t K)
{
    return M >= 0 && Nc >= 0 && K >= 0 && K % 8 == 0;
}

bool too_large(int64_t M, int64_t Nc, int64_t K)
{
    // tiles are counted in 32 bits
    return K > kMaxDim || Nc > kMaxDim || M > kMaxRows || (M / 128 + 1) * (std::max(Nc, K) / 128 + 1) > (1 << 28);
}

}  // namespace
}  // namespace lm
}  // namespace ag

using namespace ag;
using namespace ag::lm;

extern "C" int64_t gemm_bias_act_workspace(int64_t M, int64_t Nc, int64_t K)
{
    if (!shapes_ok(M, Nc, K) || too_large(M, Nc, K))
        return 0;
    return few_linear(M, Nc, K) ? 0 : plan_linear(M, Nc, K, kSum).part_bytes(M, Nc);
}

extern "C" int gemm_bias_act(const void* A, const void* B, const void* bias, const void* residual, int64_t M, int64_t Nc,
                             int64_t K, int32_t act, void* C, void* pre, void* work, int64_t work_bytes, void* stream)
{
    if (!shapes_ok(M, Nc, K) || act < kActNone || act > kActGeluTanh)
        return AG_EINVAL;
    if (M == 0 || Nc == 0)
        return AG_OK;
    if (bad(A, K) || bad(B, K) || bad(C, 1) || !aligned(bias, 16) || !aligned(residual, 16) || !aligned(pre, 16))
        return AG_EINVAL;
    if (too_large(M, Nc, K))
        return AG_EUNSUPPORTED;
    const bool few = few_linear(M, Nc, K);
    const Plan p = few ? Plan()
                       : plan_linear(M, Nc, K, act != kActNone ? kActivation : bias || residual || pre ? kStatistics : kSum);
    const int64_t need = few ? 0 : p.part_bytes(M, Nc);
    if (work_bytes < need || bad(work, need))
        return AG_EINVAL;
    TileArgs a = product(A, K, B, K, M, Nc, K, C, Nc);
    a.out.bias = static_cast<const __bf16*>(bias);
    a.out.residual = static_cast<const __bf16*>(residual);
    a.out.pre = static_cast<__bf16*>(pre);
    a.out.act = act;
    hipStream_t s = static_cast<hipStream_t>(stream);
    LM_HIP(few ? launch_rows(kEpiLinear, M, a, s) : run_product(nt_linear, p, a, work, s), "launch gemm_bias_act");
    return AG_OK;
}

extern "C" int64_t gemm_bias_act_bwd_workspace(int64_t M, int64_t Nc, int64_t K, int32_t act)
{
    if (!shapes_ok(M, Nc, K) || too_large(M, Nc, K))
        return 0;
    return plan_linear_bwd(M, Nc, K, act).bytes();
}

extern "C" int gemm_bias_act_bwd(const void* dC, const void* A, const void* B, const void* pre, int64_t M, int64_t Nc,
                                 int64_t K, int32_t act, void* dA, void* dB, void* dbias, void* work, int64_t work_bytes,
                                 void* stream)
{
    if (!shapes_ok(M, Nc, K) || act < kActNone || act > kActGeluTanh)
        return AG_EINVAL;
    if (bad(dC, M * Nc) || (dB && bad(A, M * K)) || (dA && bad(B, Nc * K)) || (act != kActNone && bad(pre, M * Nc)) ||
        !aligned(dA, 16) || !aligned(dB, 16) || !aligned(dbias, 16) || !aligned(pre, 16))
        return AG_EINVAL;
    if (too_large(M, Nc, K))
        return AG_EUNSUPPORTED;
    const LinearBwd w = plan_linear_bwd(M, Nc, K, act);
    if (work_bytes < w.bytes() || bad(work, w.bytes()))
        return AG_EINVAL;
    hipStream_t s = static_cast<hipStream_t>(stream);
    char* ws = static_cast<char*>(work);
    const void* d = dC;
    float* sum = reinterpret_cast<float*>(ws + w.d_bytes);
    void* part = ws + w.d_bytes + w.sum_bytes;
    const bool want_d = w.own_d && (dA || dB);
    if (want_d)
        d = ws;
    if (want_d || dbias)
        LM_HIP(launch_act_bwd(static_cast<const __bf16*>(dC), static_cast<const __bf16*>(pre), act, M, Nc,
                              want_d ? reinterpret_cast<__bf16*>(ws) : nullptr, w.ldd, dbias ? sum : nullptr,
                              static_cast<__bf16*>(dbias), s),
               "launch act_bwd");
    if (dbias && colsum_rows(M) != 1)
        LM_HIP(launch_colsum_join(sum, colsum_rows(M), Nc, static_cast<__bf16*>(dbias), s), "launch colsum_join");
    if (dA) {
        TileArgs a = product(d, w.ldd, B, K, M, K, w.ldd, dA, K);
        a.k_valid = Nc;
        LM_HIP(run_product(launch_nn, w.da, a, part, s), "launch dA");
    }
    if (dB)
        LM_HIP(run_product(launch_tn, w.db, product(d, w.ldd, A, K, Nc, K, M, dB, K), part, s), "launch dB");
    return AG_OK;
}

static bool groups_ok(const void* ends, int32_t E, int64_t M, int64_t Nc, int64_t K)
{
    return shapes_ok(M, Nc, K) && Nc % 8 == 0 && E >= 1 && !bad(ends, 1, 4);
}

// Tile of the products whose rows are grouped, a quarter of a large tile for each group's end taken as empty (only the
// device knows the groups).  The large one from a round of it on: before that its halves, two of which make a unit,
// leave CUs empty (1041 rows in 4 groups, 3528 x 416: 19 us against 11).
static Tile group_tile(int64_t M, int64_t N, int64_t K, int32_t E)
{
    const int64_t rows = M + 64 * (int64_t)E;
    return rows / 256 * ((N + 255) / 256) < cus() ? kTile128 : plan_product(rows, N, K, kSum, false, true).tile;
}

// Whether products grouped by rows are for the few-rows kernel, by the groups' mean rows: only the device knows more.  Each
// of its workgroups goes over the groups' ends by itself, 64 at a time, and in a short reduction over many groups that
// takes more than the product.  Tiles | few rows, us, for rows spread evenly, by weights r^4 with r uniform, all in one
// group: 16 groups, K = 4096, N = 2048, 32 rows each 44 | 46, -, 32 | 23; 64, K = 2048, N = 768, 4 rows 42 | 36,
// 26 | 30, 19 | 11, 32 rows 44 | 44, 41 | 50, 24 | 26; 256, K = 4096, N = 1024, 4 rows 524 | 419, 232 | 238, 35 | 69.
// Above a mean of 32: 64, K = 2048, N = 1024, 48 rows 49 | 58, -, 22 | 34.  More groups than K / 8: 512, K = 1024, N = 512,
// 4 rows 112 | 135, 65 | 94, 20 | 72; 256, K = 512, N = 2048, 32 rows 131 | 196, 97 | 187, 31 | 168; up to 64 groups
// that does not show: K = 64, N = 512, 32 rows 8.0 | 7.8, 8.0 | 8.5, 8.1 | 7.7.
static bool few_groups(int64_t M, int64_t K, int32_t E) { return M / E <= 32 && E <= std::max<int64_t>(64, K / 8); }

extern "C" int gemm_grouped(const void* A, const void* B, const int32_t* ends, int32_t E, int64_t M, int64_t Nc, int64_t K,
                            void* C, void* stream)
{
    if (!groups_ok(ends, E, M, Nc, K))
        return AG_EINVAL;
    if (M == 0 || Nc == 0)
        return AG_OK;
    if (bad(A, K) || bad(B, K) || bad(C, 1))
        return AG_EINVAL;
    if (too_large(M, Nc, K) || E > kMaxGroups)
        return AG_EUNSUPPORTED;
    TileArgs a = product(A, K, B, K, M, Nc, K, C, Nc);
    a.ends = ends;
    a.E = E;
    a.group = kGroupRows;
    a.strideB = Nc * K;
    hipStream_t s = static_cast<hipStream_t>(stream);
    LM_HIP(few_groups(M, K, E) ? launch_rows(kEpiLinear, M / E, a, s) : launch_nt(group_tile(M, Nc, K, E), kEpiLinear, a, s),
           "launch gemm_grouped");
    return AG_OK;
}

extern "C" int gemm_grouped_bwd(const void* dC, const void* A, const void* B, const int32_t* ends, int32_t E, int64_t M,
                                int64_t Nc, int64_t K, void* dA, void* dB, void* stream)
{
    if (!groups_ok(ends, E, M, Nc, K))
        return AG_EINVAL;
    if (bad(dC, M * Nc) || (dB && bad(A, M * K)) || (dA && bad(B, Nc * K)) || !aligned(dA, 16) || !aligned(dB, 16))
        return AG_EINVAL;
    if (too_large(M, Nc, K) || E > kMaxGroups)
        return AG_EUNSUPPORTED;
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (dA && M > 0 && K > 0) {
        TileArgs a = product(dC, Nc, B, K, M, K, Nc, dA, K);
        a.ends = ends;
        a.E = E;
        a.group = kGroupRows;
        a.strideB = Nc * K;
        // tiles of 32 rows by the groups' mean (128 or 256 | 32 rows, us, even groups): 16 groups, 2048 to 4096, 32 rows
        // each 46.4 | 43.5, 48 rows 47.1 | 52.0; 256 groups, 512 to 1024, 32 rows 60 | 57, 48 rows 63 | 85; all in one of
        // 256 groups, 8 rows 13.8 | 13.8, 32 rows 19 | 39
        LM_HIP(launch_nn(M / E <= 32 ? kTile32 : group_tile(M, K, Nc, E), a, s), "launch dA");
    }
    if (dB && Nc > 0 && K > 0) {
        TileArgs a = product(dC, Nc, A, K, Nc, K, M, dB, K);
        a.ends = ends;
        a.E = E;
        a.group = kGroupK;
        // 256 x 256 tiles from a round of them on, by both sides (128 x 128 | 256 x 256, us, uneven groups): 8 groups,
        // 1024 x 1024, half a round: 64 rows each 12 | 16, 1000 rows 25 | 45; 16 groups, a round: 19 | 16, 48 | 62;
        // 8 groups, 2048 x 2048, two rounds: 32 | 25, 88 | 69
        const int64_t tiles = (Nc + 255) / 256 * ((K + 255) / 256) * E;
        LM_HIP(launch_tn(tiles >= cus() ? kTile256 : kTile128, a, s), "launch dB");
    }
    return AG_OK;
}

static bool xent_shapes_ok(int64_t T, int64_t V, int64_t K) { return shapes_ok(T, V, K) && V >= 1; }

extern "C" int64_t gemm_xent_workspace(int64_t T, int64_t V, int64_t K)
{
    if (!xent_shapes_ok(T, V, K) || too_large(T, V, K))
        return 0;
    return region(T * stat_pairs(T, V, K) * 8) + region(T * 4);
}

extern "C" int gemm_xent(const void* A, const void* B, const int64_t* targets, int64_t T, int64_t V, int64_t K, float* loss,
                         float* lse, void* work, int64_t work_bytes, void* stream)
{
    if (!xent_shapes_ok(T, V, K))
        return AG_EINVAL;
    if (T == 0)
        return AG_OK;
    if (bad(A, K) || bad(B, K) || bad(targets, 1, 8) || bad(loss, 1, 4) || bad(lse, 1, 4) || bad(work, 1))
        return AG_EINVAL;
    if (too_large(T, V, K))
        return AG_EUNSUPPORTED;
    if (work_bytes < gemm_xent_workspace(T, V, K))
        return AG_EINVAL;
    hipStream_t s = static_cast<hipStream_t>(stream);
    TileArgs a = product(A, K, B, K, T, V, K, nullptr, 0);
    a.stat_n = stat_pairs(T, V, K);
    a.stat = static_cast<float*>(work);
    a.hit = reinterpret_cast<float*>(static_cast<char*>(work) + region(T * a.stat_n * 8));
    a.targets = targets;
    LM_HIP(launch_logits(kEpiStat, a, s), "launch gemm_xent");
    LM_HIP(launch_xent_join(a.stat, a.stat_n, a.hit, targets, T, V, loss, lse, s), "launch xent_join");
    return AG_OK;
}

extern "C" int64_t gemm_xent_bwd_workspace(int64_t T, int64_t V, int64_t K)
{
    if (!xent_shapes_ok(T, V, K) || too_large(T, V, K))
        return 0;
    return plan_xent_bwd_in(T, V, K, INT64_MAX).bytes(T);
}

extern "C" int gemm_xent_bwd(const float* dloss, const void* A, const void* B, const int64_t* targets, const float* lse,
                             int64_t T, int64_t V, int64_t K, void* dA, void* dB, void* work, int64_t work_bytes,
                             void* stream)
{
    if (!xent_shapes_ok(T, V, K))
        return AG_EINVAL;
    if (bad(A, T * K) || bad(B, K) || bad(targets, T, 8) || bad(dloss, T, 4) || bad(lse, T, 4) || !aligned(dA, 16) ||
        !aligned(dB, 16))
        return AG_EINVAL;
    if (too_large(T, V, K))
        return AG_EUNSUPPORTED;
    if (K == 0 || (!dA && !dB))
        return AG_OK;
    const XentBwd w = plan_xent_bwd_in(T, V, K, work_bytes);
    if (work_bytes < w.bytes(T) || bad(work, w.bytes(T)))
        return AG_EINVAL;
    hipStream_t s = static_cast<hipStream_t>(stream);
    char* ws = static_cast<char*>(work);
    float* part = reinterpret_cast<float*>(ws + region(T * w.piece * 2));
    const int64_t ldd = w.piece;
    for (int64_t i = 0; i < w.pieces; ++i) {
        const int64_t v0 = i * w.piece, n = std::min(w.piece, V - v0);
        const char* Bp = static_cast<const char*>(B) + v0 * K * 2;
        TileArgs a = product(A, K, Bp, K, T, n, K, ws, ldd);
        a.targets = targets;
        a.lse = lse;
        a.dloss = dloss;
        a.dloss_rows = T;
        a.vocab = V;
        a.col0 = v0;
        LM_HIP(launch_logits(kEpiGrad, a, s), "launch d logits");
        if (dA) {
            a = product(ws, ldd, Bp, K, T, K, up(n, 8), dA, K);
            a.k_valid = n;
            a.dloss = dloss;
            a.dloss_rows = T;
            if (w.part) {
                a.splits = w.da.splits;
                a.split_steps = w.da.split_steps;
                a.part = part;
                a.ldp = K;
                a.accumulate = i > 0;
            }
            LM_HIP(launch_nn(w.da.tile, a, s), "launch dA");
        }
        if (dB) {
            a = product(ws, ldd, A, K, n, K, T, static_cast<char*>(dB) + v0 * K * 2, K);
            a.dloss = dloss;
            a.dloss_rows = T;
            const Plan p = plan_product(n, K, T, kSum, false);
            LM_HIP(launch_tn(p.tile, a, s), "launch dB");
        }
    }
    if (dA && w.part) {
        LinearOut out = {};
        out.C = static_cast<__bf16*>(dA);
        out.ldc = K;
        LM_HIP(launch_join(part, w.da.splits, T, K, K, out, s, dloss, T), "launch dA join");
    }
    return AG_OK;
}
