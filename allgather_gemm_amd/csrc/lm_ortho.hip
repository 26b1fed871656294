// lm_ortho.hip -- Newton-Schulz orthogonalisation of a matrix or a stack of them: kernels and entry points.
//
//   X = G / (|G| + eps), turned so that it is m x n with m <= n; for each (a, b, c):  A = X X^T,  B = a I + b A + c A A,
//   X = B X.
//
// Products by fp16 matrix instructions with fp32 sums: the iterates' singular values stay below a bound that the
// coefficients give (checked by the entry point), so fp16 with a scale known beforehand holds them, with three bits more than bf16.
// What a rounding of X does is not the same everywhere: an error among X's small left and right singular directions comes
// out multiplied by the remaining steps' a's (3.4445^4 after the first of five), any other by about one.  Through A, and
// through B's own rounding, what is off reaches those directions only times X, which is small there; a rounding of X is in
// them as it is.  So the iterates are kept as two fp16, value and remainder, while the remaining gain is above 8: the products
// take the value alone, and a times the remainder is added to B X (B times it, but for what does not grow).  Error of the
// result's norm for a 4096 x 4096 momentum of shared directions and noise: 6.5e-3 without remainders, 1.96e-3 with them down to
// a gain of 16, 1.77e-3 to 8, 1.74e-3 to 3, of which 1.66e-3 is the result's own rounding to bf16; they take 2.5 % of the time.
//
// A and A A are symmetric: their tiles at and below the diagonal are computed, and each is stored on both sides of it.  All
// extents are padded to whole tiles of 128 with zeros, which the steps keep.
//
// Five steps of 4096 x 4096 take 1.34 to 1.40 ms, 1.0 PFLOP/s of the products that are computed, of 14336 x 4096 3.6 to 3.85 ms, 1.06.
// Matrix instructions run in 0.50-0.54 of the cycles in A A and X X^T, 0.57-0.60 in B X, 0.69 in the longer X X^T, at 1.8 to 1.9 GHz;
// in the rest the one wave of a SIMD waits (0.17-0.24 of its cycles), reads fragments, starts a tile or stores one.  Small matrices
// wait for their launches, two or three a step of 5 to 10 us.
#include "../../include/aggemm.h"
#include "ag_internal.hpp"
#include "lm_tile.hpp"

#include <algorithm>
#include <cmath>

namespace ag {
namespace lm {

struct OrthoArgs : TileArgs {
    float alpha, beta;       // out = alpha sums + beta addend, plus `unit` on the diagonal (kEpiSquare)
    float unit;
    float square_alpha, square_beta;   // B out of A A and A, where X = B X forms it (ortho_thin_kernel)
    const float* scale;      // for each matrix what X is stored in, see in_units()
    float now, next;         // X comes in units of min(1, scale now), or (0) of scale; it goes in those of `next`, or (0) of 1
    const _Float16* add;     // addend: A (kEpiSquare); X's remainder, or null (kEpiUpdate)
    _Float16 *hi, *lo;       // the result and (unless null) its remainder
    int64_t ldo, stride;     // of addend and result: rows, matrices
    // the last step's result, m x n unpadded (null: hi), or its transpose
    __bf16* last;
    int64_t m, n;
    bool turned;
    int tiles_m;
    int cut;                 // of the tiles, those that go in quarters
    // X X^T of a long reduction over few tiles: `splits` workgroups for each, whose fp32 sums go here, 4096 for each, and a
    // count for each tile of those that are done, zero before and after
    float* sums;
    uint32_t* done;
};

namespace {

constexpr float kScaleX = 4096.0f, kScaleA = 4096.0f;   // stored = true x this; B: scale_b()
constexpr int PAD = 128;

// X is stored in units of f: at the start of scale = 2^k / (|G| + eps) <= 2 with |G| in [1/2, 1) 2^k, after a step of
// min(1, scale g) with g the most that the steps so far can have multiplied a singular value by.  Where eps does not count that is
// 1, X itself; where |G| is far below eps, X keeps its bits so (as X itself G of 1e-8 eps came out off by 0.4, of 1e-9 as
// zeros).  A is always that of X itself: where f is small, next to nothing beside a I.  A scale of NaN stays one.
__device__ __forceinline__ float in_units(float scale, float g)
{
    const float f = scale * g;
    return f > 1.0f ? 1.0f : f;
}

// A wave's block of 32 rows and FN * 32 columns of 16 bits in its LDS slab, laid out as half_slab_at() has it; three blocks
// side by side take rows of four, of which `units` 16-byte units are there.
template <int FN>
struct Slab {
    static constexpr int L = FN == 3 ? 4 : FN;
    static constexpr uint32_t RB = L * 64, UN = RB / 16;           // bytes and 16-byte units of a row
    static constexpr int RPI = 64 / UN, ITS = 32 / RPI;            // rows at a time, times
    static constexpr int BYTES = 32 * RB;

    // 16-byte unit u of row it * RPI + r0, the halves of the lower rows' units the other way round
    static __device__ __forceinline__ i32x4* unit(char* slab, int it, uint32_t r0, uint32_t u)
    {
        const uint32_t r = it * RPI + r0;
        return reinterpret_cast<i32x4*>(slab + r * RB + ((u ^ (r & (UN - 1))) * 16));
    }
    static __device__ __forceinline__ i32x4 halves(int it, i32x4 x)
    {
        return it * RPI >= 16 ? i32x4{x[2], x[3], x[0], x[1]} : x;
    }

    // a block on its way from memory
    struct Ahead {
        i32x4 x[ITS];
    };
    static __device__ __forceinline__ void fetch(Ahead& p, const _Float16* from, int64_t ld, uint32_t units, int lane)
    {
        const uint32_t u = lane % UN, r0 = lane / UN;
        if (FN != 3 || u < units) {
            from += r0 * ld + u * 8;
#pragma unroll
            for (int it = 0; it < ITS; ++it)
                p.x[it] = *reinterpret_cast<const i32x4*>(from + it * RPI * ld);
        }
    }
    static __device__ __forceinline__ void put(char* slab, const Ahead& p, int lane)
    {
        const uint32_t u = lane % UN, r0 = lane / UN;
#pragma unroll
        for (int it = 0; it < ITS; ++it)
            *unit(slab, it, r0, u) = halves(it, p.x[it]);
    }
    static __device__ __forceinline__ void out(char* slab, _Float16* to, int64_t ld, uint32_t units, int lane)
    {
        const uint32_t u = lane % UN, r0 = lane / UN;
        settle();
        to += r0 * ld + u * 8;
#pragma unroll
        for (int it = 0; it < ITS; ++it) {
            const i32x4 y = halves(it, *unit(slab, it, r0, u));
            if (FN != 3 || u < units)
                *reinterpret_cast<i32x4*>(to + it * RPI * ld) = y;
        }
        settle();
    }
    // this wave's LDS reads and writes are done
    static __device__ __forceinline__ void settle()
    {
        __builtin_amdgcn_s_waitcnt(0xC07F);   // lgkmcnt(0)
        __builtin_amdgcn_wave_barrier();
    }
};

// The slab's transpose to memory: the transposing LDS reads give a lane eight rows of its column.  p: where the block's first
// element goes, cols: valid columns of the block (rows there), rows: valid rows.
template <int FN>
__device__ __forceinline__ void half_slab_turned(const char* slab, __bf16* p, int64_t ld, int64_t rows, int64_t cols, int lane)
{
    constexpr uint32_t RB = Slab<FN>::RB, UN = Slab<FN>::UN;
    const uint32_t g = lane >> 4, i = lane & 15;
    const int n = (int)min((int64_t)8, rows - (int64_t)g * 8);
    __builtin_amdgcn_s_waitcnt(0xC07F);   // lgkmcnt(0): this wave's slab is written
    __builtin_amdgcn_wave_barrier();
    auto four = [&](uint32_t r, uint32_t cb) {
        const uint32_t piece = cb * 4 + (i & 3);
        const char* at = slab + r * RB + (((piece & 1) ^ (r >> 4)) * 8) + (((piece >> 1) ^ (r & (UN - 1))) * 16);
        return __builtin_bit_cast(bf16x4, __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_bf16x4*)const_cast<char*>(at)));
    };
#pragma unroll
    for (int cb = 0; cb < FN * 2; ++cb) {
        const bf16x4 lo = four(g * 8 + (i >> 2), cb), hi = four(g * 8 + 4 + (i >> 2), cb);
        const bf16x8 y = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
        const int64_t row = cb * 16 + i;
        __bf16* const out = p + row * ld + g * 8;
        if (row < cols) {
            if (n >= 8)
                *reinterpret_cast<bf16x8_any*>(out) = y;
            else
#pragma unroll
                for (int e = 0; e < 7; ++e)
                    if (e < n)
                        out[e] = y[e];
        }
    }
    __builtin_amdgcn_s_waitcnt(0xC07F);   // reads done before the slab is rewritten
    __builtin_amdgcn_wave_barrier();
}

}  // namespace

// What follows the sums of a wave's FM blocks of 32 rows, WM * 32 rows apart from row0 on, and 32 FN columns from col0 on.
template <int EPI, int FM, int FN, int WM, typename Acc>
__device__ __forceinline__ void after_sums(const OrthoArgs& a, const Where& w, Acc acc, char* slab, int64_t row0, int64_t col0,
                                           int lane)
{
    typedef Slab<FN> S;
    const uint32_t fr = lane & 31, fh = lane >> 5;
    const float f = EPI == kEpiSquare ? 1.0f : a.now == 0.0f ? w.scale : in_units(w.scale, a.now);
    const float r = EPI == kEpiGram ? f * f : EPI == kEpiUpdate && a.next != 0.0f ? f / in_units(w.scale, a.next) : f;
    const float alpha = a.alpha * r, beta = a.beta * (EPI == kEpiUpdate ? r : 1.0f);
    const bool keep = EPI == kEpiUpdate && a.lo, add = EPI == kEpiSquare || (EPI == kEpiUpdate && a.add);
    if (col0 >= a.N)
        return;
    // extents are multiples of 128, a wave's columns of a 192 x 192 tile are not
    const uint32_t units = (uint32_t)min((int64_t)FN * 4, (a.N - col0) / 8);
    const int64_t first = w.g * a.stride + row0 * a.ldo + col0;
    typename S::Ahead ahead;
    if (add && row0 < w.M)
        S::fetch(ahead, a.add + first, a.ldo, units, lane);
#pragma unroll
    for (int i = 0; i < FM; ++i) {
        const f32x16* const x = acc(i);
        const int64_t row = row0 + i * WM * 32;
        if (row >= w.M)
            break;
        const int64_t at = first + i * WM * 32 * a.ldo;
        if (add) {
            S::put(slab, ahead, lane);
            if (i + 1 < FM && row + WM * 32 < w.M)
                S::fetch(ahead, a.add + at + WM * 32 * a.ldo, a.ldo, units, lane);
            S::settle();
        }
        const int diagonal = (int)(row - col0) + (int)fr - (int)fh * 4;      // the lane's columns count from fh * 4
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                f16x4* const p = reinterpret_cast<f16x4*>(half_slab_at<S::L>(slab, j, q, fr, fh));
                float v[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    v[e] = alpha * x[j][q * 4 + e];
                if (add) {
                    const f16x4 y = *p;
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        v[e] = fmaf(beta, (float)y[e], v[e]);
                }
                if constexpr (EPI == kEpiSquare) {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        v[e] += diagonal == j * 32 + q * 8 + e ? a.unit : 0.0f;
                }
                if (EPI == kEpiUpdate && a.last) {
                    *reinterpret_cast<bf16x4*>(p) = bf16x4{(__bf16)v[0], (__bf16)v[1], (__bf16)v[2], (__bf16)v[3]};
                    continue;
                }
                const f16x4 h = {(_Float16)v[0], (_Float16)v[1], (_Float16)v[2], (_Float16)v[3]};
                *p = h;
                if (keep)
                    *reinterpret_cast<f16x4*>(half_slab_at<S::L>(slab + S::BYTES, j, q, fr, fh)) =
                        f16x4{(_Float16)(v[0] - (float)h[0]), (_Float16)(v[1] - (float)h[1]), (_Float16)(v[2] - (float)h[2]),
                              (_Float16)(v[3] - (float)h[3])};
            }
        if constexpr (EPI == kEpiUpdate) {
            if (a.last) {
                __bf16* const out = a.last + w.g * a.m * a.n;
                if (a.turned)
                    half_slab_turned<FN>(slab, out + col0 * a.m + row, a.m, a.m - row, a.n - col0, lane);
                else
                    half_slab_out<FN, true>(slab, out + row * a.n + col0, a.n, a.m - row, a.n - col0, lane);
                continue;
            }
        }
        S::out(slab, a.hi + at, a.ldo, units, lane);
        if (keep)
            S::out(slab + S::BYTES, a.lo + at, a.ldo, units, lane);
        if (EPI != kEpiUpdate && w.m0 > w.n0)  // a tile below the diagonal
            half_slab_turned<FN>(slab, reinterpret_cast<__bf16*>(a.hi + w.g * a.stride + col0 * a.ldo + row), a.ldo, 32, units * 8,
                                 lane);
    }
}

namespace {

// Tile t at or below the diagonal of rows x rows tiles: GROUP_M tile rows at a time, column by column, so that the tiles in
// flight share rows in the caches.
__device__ __forceinline__ void lower_tile(int t, int rows, int& m, int& n)
{
    int first = 0;
    while (true) {
        const int h = min(rows - first, GROUP_M), here = h * first + h * (h + 1) / 2;
        if (t < here) {
            if (t < h * first) {
                n = t / h;
                m = first + t - n * h;
            } else {
                t -= h * first;
                int r = 0;
                while (t > r)
                    t -= ++r;
                m = first + r;
                n = first + t;
            }
            return;
        }
        t -= here;
        first += h;
    }
}

// A launch's tiles: BM x BM ones, then (256 and 128) the last `cut` of them in quarters.
template <int BM, int S, int EPI>
__device__ __forceinline__ void ortho_body(const OrthoArgs& a)
{
    constexpr bool TB = EPI == kEpiUpdate, LARGE = BM == 256, QUARTERS = LARGE || BM == 128;
    constexpr int BYTES = BM * BK * 2;
    static_assert(S == 2 ? LARGE : S == 3 || S == 4, "stages");
    __shared__ __attribute__((aligned(1024))) char sA0[LARGE ? BYTES / 2 : BYTES], sU0[LARGE ? BYTES / 2 : 16];
    __shared__ __attribute__((aligned(1024))) char sB0[BYTES], sA1[BYTES], sB1[BYTES];
    __shared__ __attribute__((aligned(1024))) char sA2[S > 2 ? BYTES : 16], sB2[S > 2 ? BYTES : 16];
    __shared__ __attribute__((aligned(1024))) char sA3[S > 3 ? BYTES : 16], sB3[S > 3 ? BYTES : 16];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    Stages<S> l;
    l.a[0] = {sA0, LARGE ? sU0 : sA0};
    l.b[0] = {sB0, sB0 + BYTES / 2};
    l.a[1] = {sA1, sA1 + BYTES / 2};
    l.b[1] = {sB1, sB1 + BYTES / 2};
    if constexpr (S > 2) {
        l.a[2].lo = sA2;
        l.b[2].lo = sB2;
    }
    if constexpr (S > 3) {
        l.a[3].lo = sA3;
        l.b[3].lo = sB3;
    }
    // two slabs a wave where a remainder is kept beside the result
    constexpr int SLABS = (EPI == kEpiUpdate ? 2 : 1) * Slab<BM / 64>::BYTES;
    if constexpr (LARGE)
        l.slab = (wave == 0 ? sA0 : wave == 1 ? sU0 : sB0 + (wave - 2) * SLABS);
    else
        l.slab = (wave < 2 ? sA0 : sB0) + (wave & 1) * SLABS;
    static_assert((LARGE ? 1 : 2) * SLABS <= (int)sizeof(sA0) && 2 * SLABS <= BYTES, "slabs in the first stage");
    Stages<4> lq;
    if constexpr (BM == 128) {
        lq = l;
    } else if constexpr (LARGE) {
        lq.a[0].lo = sA0;
        lq.b[0].lo = sU0;
        lq.a[1].lo = sB0;
        lq.b[1].lo = sB0 + 16384;
        lq.a[2].lo = sA1;
        lq.b[2].lo = sA1 + 16384;
        lq.a[3].lo = sB1;
        lq.b[3].lo = sB1 + 16384;
        lq.slab = l.slab;
    }
    const int G = gridDim.x, rows = a.tiles_m, cols = (int)a.tiles_n;
    // workgroups are dispatched round-robin over the 8 XCDs: each XCD takes a contiguous run of tiles
    const int vid = (G % 8 == 0) ? (int)(blockIdx.x % 8) * (G / 8) + (int)(blockIdx.x / 8) : (int)blockIdx.x;
    const int per = EPI == kEpiUpdate ? rows * cols : rows * (rows + 1) / 2, all = per * a.E, whole = all - a.cut;
    auto tile = [&](int t, int& e, int& tm, int& tn) {
        e = t / per;
        if (EPI == kEpiUpdate)
            tile_of(t - e * per, rows, cols, tm, tn);
        else
            lower_tile(t - e * per, rows, tm, tn);
    };
    for (int t = vid; t < whole; t += G) {
        int e, tm, tn;
        tile(t, e, tm, tn);
        const Where w = {(int64_t)tm * BM, (int64_t)tn * BM, a.M, a.K, 0, e * a.M, tn, e, 0, false, EPI == kEpiSquare ? 1.0f : a.scale[e]};
        product_tile<BM, BM, 2, 2, S, false, TB, EPI>(a, l, w);
    }
    if constexpr (QUARTERS) {
        for (int t = vid; t < 4 * a.cut; t += G) {
            int e, tm, tn;
            tile(whole + t / 4, e, tm, tn);
            const int64_t m0 = (int64_t)tm * BM + (t >> 1 & 1) * (BM / 2), n0 = (int64_t)tn * BM + (t & 1) * (BM / 2);
            if (m0 >= a.M || n0 >= a.N || (EPI != kEpiUpdate && n0 > m0))
                continue;
            const Where w = {m0, n0, a.M, a.K, 0, e * a.M, tn, e, 0, false, EPI == kEpiSquare ? 1.0f : a.scale[e]};
            product_tile<BM / 2, BM / 2, 2, 2, 4, false, TB, EPI>(a, lq, w);
        }
    }
}

template <int EPI>
__global__ __launch_bounds__(NT, 1) void ortho256_kernel(OrthoArgs a)
{
    ortho_body<256, 2, EPI>(a);
}

template <int EPI>
__global__ __launch_bounds__(NT, 1) void ortho192_kernel(OrthoArgs a)
{
    ortho_body<192, 3, EPI>(a);
}

template <int EPI>
__global__ __launch_bounds__(NT, 1) void ortho128_kernel(OrthoArgs a)
{
    ortho_body<128, 4, EPI>(a);
}

// The parts of a 64 x 64 tile's reduction: each workgroup leaves its sums in memory and counts itself; the last one adds
// them all up, in the parts' order whoever came last, and has the tile from there on (true).  Nobody waits.  The sums are
// stored through the caches and counted when they have arrived, so no cache has to be written back (a release fence
// does that with the whole L2: X X^T of 512 x 4096 in six parts took 25 us with it, 15 without, as long as in one part).
__device__ __forceinline__ bool join_parts(const OrthoArgs& a, int64_t tile, int part, f32x16& x)
{
    constexpr int kWriteThrough = 1 | 16;              // cache policy bits sc0 | sc1
    __shared__ uint32_t s_before;
    f32x4* const sums = reinterpret_cast<f32x4*>(a.sums) + tile * a.splits * 1024;
    const __amdgpu_buffer_rsrc_t to = make_rsrc(sums + part * 1024, 16384);
#pragma unroll
    for (int q = 0; q < 4; ++q)
        __builtin_amdgcn_raw_buffer_store_b128(
            __builtin_bit_cast(i32x4, f32x4{x[q * 4], x[q * 4 + 1], x[q * 4 + 2], x[q * 4 + 3]}), to,
            (q * 256 + threadIdx.x) * 16, 0, kWriteThrough);
    wait_vmcnt0();
    __syncthreads();
    if (threadIdx.x < 64) {
        const uint32_t before = wave_fetch_add(a.done + tile, 1);
        if (is_lane0())
            s_before = before;
    }
    barrier_after_lds_write();
    if ((int)__builtin_amdgcn_readfirstlane(s_before) != a.splits - 1)
        return false;
    acquire_agent();
    if (threadIdx.x < 64)
        wave_exchange(a.done + tile, 0);
    x = f32x16{};
#pragma unroll 4
    for (int s = 0; s < a.splits; ++s) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const f32x4 y = sums[s * 1024 + q * 256 + threadIdx.x];
#pragma unroll
            for (int e = 0; e < 4; ++e)
                x[q * 4 + e] += y[e];
        }
    }
    return true;
}

// 64 x 64 tiles, a workgroup for each, of matrices so small that a launch mostly waits: for its code, its first loads, LDS.
// Everything about where a tile lies is one workgroup index each and 32 bits; a step's fragments are all read while the
// step before multiplies; four steps are on their way.  H = 2: steps of 128, one workgroup a CU; H = 1: of 64, two.
// PARTS: of a tile's reduction.  X X^T of 1024 x 1024 7.4 us, of 1024 x 8192 26.5 (0.165 a step of 64); as product_tile() has
// it, with the tiles' general order, 11.9 and 34.3.
template <int EPI, int H, bool PARTS>
__global__ __launch_bounds__(NT, H == 1 ? 2 : 1) void ortho64_kernel(OrthoArgs a)
{
    constexpr bool TB = EPI == kEpiUpdate;
    constexpr int HALF = H * 8192, OPS = H * 4;        // bytes of a step's A, loads of a step
    __shared__ __attribute__((aligned(1024))) char s0[2 * HALF], s1[2 * HALF], s2[2 * HALF], s3[2 * HALF];
    int tn = blockIdx.x, tm = blockIdx.y, part = 0;
    const int e = blockIdx.z;
    if constexpr (PARTS) {         // parts come first: a multiple of 8, so each XCD has its own columns of X in its cache
        part = blockIdx.x;
        tm = blockIdx.y / (uint32_t)a.tiles_n;
        tn = blockIdx.y - tm * (int)a.tiles_n;
    }
    if (!TB && tn > tm)
        return;
    const float scale = EPI == kEpiSquare ? 1.0f : a.scale[e];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), wm = wave >> 1, wn = wave & 1;
    const uint32_t lda = (uint32_t)a.lda * 2, ldb = (uint32_t)a.ldb * 2, r = tid >> 3, p = tid & 7;
    const uint32_t va = r * lda + ((p ^ swz(r)) * 16);
    const uint32_t vb = TB ? r * ldb + (((p >> 2) ^ Side<64, true>::ksw(r)) * 4 + (p & 3)) * 16 : r * ldb + ((p ^ swz(r)) * 16);
    const __amdgpu_buffer_rsrc_t ra = make_rsrc(a.A + (e * a.M + tm * 64) * a.lda, 64 * lda);
    const __amdgpu_buffer_rsrc_t rb = TB ? make_rsrc(a.B + e * a.strideB + tn * 64, (uint32_t)a.K * ldb - tn * 128)
                                         : make_rsrc(a.B + e * a.strideB + (int64_t)tn * 64 * a.ldb, 64 * ldb);
    const int all = (int)a.K / (H * 64), begin = PARTS ? min(part * (int)a.split_steps, all) : 0;
    const int end = PARTS ? min(begin + (int)a.split_steps, all) : all, steps = end - begin, last = max(end - 1, 0);
    int at = min(begin, last);                         // of the next loads; past the last step that one again
    auto issue = [&](char* s) {
        const uint32_t ka = at * H * 128, kb = TB ? at * H * 64 * ldb : ka;
        at = min(at + 1, last);
        char* const to = s + wave * 1024;
#pragma unroll
        for (int h = 0; h < H; ++h)
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (lds_void*)(to + h * 8192 + q * 4096), 16, (int)(va + q * 32 * lda),
                                                         (int)(ka + h * 128), 0, 0);
                __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, (lds_void*)(to + HALF + h * 8192 + q * 4096), 16,
                                                         (int)(vb + q * 32 * ldb), (int)(kb + h * (TB ? 64 * ldb : 128)), 0, 0);
            }
    };
    issue(s0);
    issue(s1);
    issue(s2);
    issue(s3);
    Frag<64, false, 1, true> fa;
    Frag<64, TB, 1, false> fb;
    fa.init(lane, wm);
    fb.init(lane, wn);
    bf16x8 af[2][4 * H], bf[2][4 * H];
    auto read = [&](int set, char* s) {
#pragma unroll
        for (int kk = 0; kk < 4 * H; ++kk) {
            af[set][kk] = fa.read(Part{s + (kk >> 2) * 8192, nullptr}, kk & 3, 0);
            bf[set][kk] = fb.read(Part{s + HALF + (kk >> 2) * 8192, nullptr}, kk & 3, 0);
        }
    };
    f32x16 acc = {};
    // the next step's loads are there, everyone has read this one's stage
    auto step = [&](int set, char* s, char* next) {
        wait_vmcnt<2 * OPS>();
        stage_barrier();
        issue(s);
        read(set ^ 1, next);
#pragma unroll
        for (int kk = 0; kk < 4 * H; ++kk)
            acc = __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, bf[set][kk]), __builtin_bit_cast(f16x8, af[set][kk]),
                                                         acc, 0, 0, 0);
    };
    wait_vmcnt<3 * OPS>();
    stage_barrier();
    read(0, s0);
    int k = 0;
    for (; k + 4 <= steps; k += 4) {
        step(0, s0, s1);
        step(1, s1, s2);
        step(0, s2, s3);
        step(1, s3, s0);
    }
    if (k < steps) {
        step(0, s0, s1);
        if (k + 1 < steps) {
            step(1, s1, s2);
            if (k + 2 < steps)
                step(0, s2, s3);
        }
    }
    wait_vmcnt0();
    stage_barrier();
    if constexpr (PARTS)
        if (!join_parts(a, ((int64_t)e * a.tiles_m + tm) * a.tiles_n + tn, part, acc))
            return;
    const Where w = {tm * 64, tn * 64, a.M, a.K, 0, 0, tn, e, 0, false, scale};
    after_sums<EPI, 1, 1, 2>(a, w, [&](int) { return &acc; }, s0 + wave * 2 * Slab<1>::BYTES, tm * 64 + wm * 32, tn * 64 + wn * 32, lane);
}

// ------------------------------------------------------------------------------------------- few rows
// X = B X with B = a I + b A + c A A formed on the way, for MP = 128 or 256 rows (padded), whose products take less than a
// launch: a workgroup holds all of A in LDS, makes 64 rows of B out of it and multiplies them with blocks of 64 columns of X,
// the next block on its way meanwhile.  What every workgroup of the same 64 rows does again is 64 MP MP products.  Five steps
// so | by a launch for B, us: 64 x 64 49 | 66, 128 x 512 59 | 72, 128 x 4096 80 | 95, 256 x 512 72 | 79, 256 x 8192 121 | 121,
// 25 of 72 x 5440 254 | 300.
template <int MP>
__global__ __launch_bounds__(NT, MP == 256 ? 1 : 2) void ortho_thin_kernel(OrthoArgs a)
{
    constexpr int KS = MP / 64, F = MP / 128, XOPS = 2 * KS;      // steps of 64; a wave's blocks of 32 columns of B
    // A by steps of 64 columns, MP rows of 128 bytes each; then B's rows, the slabs and a second block of X
    __shared__ __attribute__((aligned(1024))) char sT0[MP * 128];
    __shared__ __attribute__((aligned(1024))) char sT1[MP * 128];
    __shared__ __attribute__((aligned(1024))) char sT2[MP * 128];
    __shared__ __attribute__((aligned(1024))) char sT3[KS > 2 ? MP * 128 : 16];
    __shared__ __attribute__((aligned(1024))) char sX[MP * 128];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave >> 1, wn = wave & 1;
    const uint32_t fr = lane & 31, fh = lane >> 5, wave_off = wave * 1024;
    const int blocks = (int)(a.N / 64), sharers = (int)(gridDim.x / (a.E * KS));      // workgroups of the same rows
    const int first = (int)blockIdx.x % sharers, rb = (int)blockIdx.x / sharers % KS, e = (int)blockIdx.x / sharers / KS;
    const float scale = a.scale[e];
    char* const stage[4] = {sT0, sT1, KS > 2 ? sT2 : sT0, KS > 2 ? sT3 : sT1};

    Side<MP, false> sa;
    sa.init(tid, a.lda);
    sa.start(a.A + (int64_t)e * MP * MP, MP, MP, 0, 0, MP);
    each<KS>([&](auto kb) {
        const __amdgpu_buffer_rsrc_t r = sa.rsrc();
        const Part p = {stage[kb], stage[kb] + 16384};
#pragma unroll
        for (int q = 0; q < MP / 32; ++q)
            sa.load(r, p, wave_off, sa.offset(), sa.op_stride, q);
        sa.advance();
    });
    Side<64, true> sx;
    sx.init(tid, a.ldb);
    auto fetch_x = [&](char* to, int block) {
        sx.start(a.B + e * a.strideB + block * 64, 64, MP, block * 64, 0, MP);
#pragma unroll
        for (int kb = 0; kb < KS; ++kb) {
            const __amdgpu_buffer_rsrc_t r = sx.rsrc();
            const Part p = {to + kb * 8192, nullptr};
            sx.load(r, p, wave_off, sx.offset(), sx.op_stride, 0);
            sx.load(r, p, wave_off, sx.offset(), sx.op_stride, 1);
            sx.advance();
        }
    };
    fetch_x(sX, first);

    // 64 rows of A A: a wave's MP / 4 columns
    {
        Frag<64, false, 2, false> fa;
        Frag<64, false, F, false> fb;
        fa.init(lane, 0);
        fb.init(lane, 0);
        f32x16 acc[2][F] = {};
        each<KS>([&](auto kb) {
            wait_vmcnt<(KS - 1 - decltype(kb)::value) * (MP / 32) + XOPS>();
            stage_barrier();
            const Part pa = {stage[kb] + rb * 8192, nullptr}, pb = {stage[kb] + wave * F * 4096, nullptr};
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
                bf16x8 af[2], bf[F];
#pragma unroll
                for (int j = 0; j < F; ++j)
                    bf[j] = fb.read(pb, kk, j);
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    af[i] = fa.read(pa, kk, i);
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int j = 0; j < F; ++j)
                        acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, bf[j]),
                                                                           __builtin_bit_cast(f16x8, af[i]), acc[i][j], 0, 0, 0);
            }
        });
        const int kb = wave * F / 2;                   // the step in which the wave's columns are
        const char* const from = KS == 2 ? (kb ? sT1 : sT0) : kb < 2 ? (kb ? sT1 : sT0) : (kb == 2 ? sT2 : sT3);
        const uint32_t sw = swz(fr & 15);
        auto place = [&](int i, int j, int q) {        // of four columns in a step's row
            const uint32_t chunk = ((wave * F + j) & 1) * 4 + q;
            return (uint32_t)(i * 32 + fr) * 128 + ((chunk ^ sw) * 16) + fh * 8;
        };
        f16x4 h[2][F][4];
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < F; ++j) {
                const int diagonal = rb * 64 + i * 32 + (int)fr - ((wave * F + j) * 32 + (int)fh * 4);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const f16x4 y = *reinterpret_cast<const f16x4*>(from + rb * 8192 + place(i, j, q));
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        h[i][j][q][c] = (_Float16)(fmaf(a.square_beta, (float)y[c], a.square_alpha * acc[i][j][q * 4 + c]) +
                                                   (diagonal == q * 8 + c ? a.unit : 0.0f));
                }
            }
        stage_barrier();                               // A is read
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < F; ++j)
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    *reinterpret_cast<f16x4*>(sT0 + kb * 8192 + place(i, j, q)) = h[i][j][q];
    }

    Frag<64, false, 1, true> fa;
    Frag<64, true, 1, false> fb;
    fa.init(lane, wm);
    fb.init(lane, wn);
    char* const slab = sT1 + wave * 2 * Slab<1>::BYTES;
    auto block = [&](const char* x, char* other, int b) {
        const int next = b + sharers;
        if (next < blocks)
            fetch_x(other, next);
        if (next < blocks)
            wait_vmcnt<XOPS>();
        else
            wait_vmcnt0();
        stage_barrier();                               // B's rows are written, this block of X is there
        f32x16 acc = {};
#pragma unroll
        for (int kb = 0; kb < KS; ++kb)
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
                const bf16x8 bf = fb.read(Part{const_cast<char*>(x) + kb * 8192, nullptr}, kk, 0);
                const bf16x8 af = fa.read(Part{sT0 + kb * 8192, nullptr}, kk, 0);
                acc = __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, bf), __builtin_bit_cast(f16x8, af), acc, 0, 0, 0);
            }
        stage_barrier();                               // read: the block after the next may come there
        const Where w = {rb * 64, b * 64, a.M, a.K, 0, 0, 0, e, 0, false, scale};
        after_sums<kEpiUpdate, 1, 1, 2>(a, w, [&](int) { return &acc; }, slab, rb * 64 + wm * 32, (int64_t)b * 64 + wn * 32, lane);
    };
    for (int b = first; b < blocks; b += 2 * sharers) {
        block(sX, sT2, b);
        if (b + sharers < blocks)
            block(sT2, sX, b + sharers);
    }
}

// ------------------------------------------------------------------------------------------- what comes first
// Sums of squares in fp64: squares of any fp32 neither overflow nor vanish there.
template <typename T>
__global__ __launch_bounds__(256) void ortho_norm_kernel(const T* G, int64_t elements, double* part)
{
    __shared__ double s_sum[4];
    const T* p = G + blockIdx.y * elements;
    double sum = 0.0;
    typedef T vec __attribute__((ext_vector_type(8)));
    typedef vec vec_any __attribute__((aligned(sizeof(T))));
    for (int64_t i = (blockIdx.x * 256 + threadIdx.x) * (int64_t)8; i < elements; i += gridDim.x * (int64_t)2048) {
        if (i + 8 <= elements) {
            const vec v = *reinterpret_cast<const vec_any*>(p + i);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                sum = fma((double)(float)v[e], (double)(float)v[e], sum);
        } else {
            for (int e = 0; e < 8; ++e)
                if (i + e < elements)
                    sum = fma((double)(float)p[i + e], (double)(float)p[i + e], sum);
        }
    }
#pragma unroll
    for (int s = 1; s < 64; s <<= 1)
        sum += __shfl_xor(sum, s);
    if ((threadIdx.x & 63) == 0)
        s_sum[threadIdx.x >> 6] = sum;
    barrier_after_lds_write();
    if (threadIdx.x == 0)
        part[blockIdx.y * (int64_t)gridDim.x + blockIdx.x] = (s_sum[0] + s_sum[1]) + (s_sum[2] + s_sum[3]);
}

struct StartArgs {
    int64_t R, C;            // extents of G
    int64_t mp, np;          // padded extents of X
    int parts;               // sums of squares for each matrix
    float eps;
    const double* part;
    float* scale;
    uint32_t* done;          // counts to be zero
    int64_t counts;
    _Float16 *hi, *lo;       // lo may be null
};

// X from G, 64 x 64 elements a workgroup: scaled by a power of two, which rounds nothing in a bf16 G but elements below 2^-28 of
// its norm (fp16's subnormals: by 2^-37 of the norm at most).  `scale` gets what is left of 1 / (|G| + eps).
template <typename T, bool TURN>
__global__ __launch_bounds__(256) void ortho_start_kernel(const T* G, StartArgs a)
{
    __shared__ double s_sum[4];
    __shared__ float s_tile[TURN ? 64 : 1][65];
    const int64_t e = blockIdx.y;
    double sum = 0.0;
    for (int i = threadIdx.x; i < a.parts; i += 256)
        sum += a.part[e * a.parts + i];
#pragma unroll
    for (int s = 1; s < 64; s <<= 1)
        sum += __shfl_xor(sum, s);
    if ((threadIdx.x & 63) == 0)
        s_sum[threadIdx.x >> 6] = sum;
    barrier_after_lds_write();
    const double size = sqrt((s_sum[0] + s_sum[1]) + (s_sum[2] + s_sum[3])), norm = size + (double)a.eps;
    const bool fine = norm > 0.0 && norm < (double)INFINITY;
    int k = 0;
    if (fine)
        frexp(size > 0.0 ? size : norm, &k);
    const int tiles = (int)(a.np / 64);
    const int64_t i0 = blockIdx.x / tiles * 64, j0 = (int64_t)(blockIdx.x % tiles) * 64;
    if (blockIdx.x == 0 && threadIdx.x == 0)
        a.scale[e] = fine ? fmaxf((float)ldexp(1.0 / norm, k), 0x1p-149f) : NAN;
    if (blockIdx.x == 0 && e == 0)
        for (int64_t i = threadIdx.x; i < a.counts; i += 256)
            a.done[i] = 0;
    const int64_t g0 = TURN ? j0 : i0, h0 = TURN ? i0 : j0;             // the tile's first row and column in G
    const T* p = G + e * a.R * a.C;
    const int rl = threadIdx.x >> 2, cl = (threadIdx.x & 3) * 16;
    float x[16];
    {
        const int64_t row = g0 + rl;
        const int n = row < a.R && fine ? (int)max((int64_t)0, min((int64_t)16, a.C - h0 - cl)) : 0;
        typedef T vec __attribute__((ext_vector_type(8)));
        typedef vec vec_any __attribute__((aligned(sizeof(T))));
        const T* q = p + row * a.C + h0 + cl;
#pragma unroll
        for (int c = 0; c < 16; c += 8) {
            if (c + 8 <= n) {
                const vec v = *reinterpret_cast<const vec_any*>(q + c);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    x[c + i] = ldexpf((float)v[i], 12 - k);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    x[c + i] = c + i < n ? ldexpf((float)q[c + i], 12 - k) : 0.0f;
            }
        }
    }
    if constexpr (TURN) {
#pragma unroll
        for (int i = 0; i < 16; ++i)
            s_tile[rl][cl + i] = x[i];
        barrier_after_lds_write();
#pragma unroll
        for (int i = 0; i < 16; ++i)
            x[i] = s_tile[cl + i][rl];
    }
    const int64_t at = (e * a.mp + i0 + rl) * a.np + j0 + cl;
#pragma unroll
    for (int c = 0; c < 16; c += 8) {
        f16x8 h, r;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            h[i] = (_Float16)x[c + i];
            r[i] = (_Float16)(x[c + i] - (float)h[i]);
        }
        *reinterpret_cast<f16x8*>(a.hi + at + c) = h;
        if (a.lo)
            *reinterpret_cast<f16x8*>(a.lo + at + c) = r;
    }
}

// --------------------------------------------------------------------------------------------- host
int64_t up(int64_t x, int64_t n) { return (x + n - 1) / n * n; }

struct Ortho {
    int64_t m, n, mp, np;
    int parts;
    int64_t part, scale, sums, done, x0, x1, lo, a, b, bytes;      // offsets in the workspace
    int64_t counts;          // of tiles in parts
};

// Workgroups of a launch: 64 x 64 elements each at the start, tiles of 128 x 128 and their quarters in 32 bits.
bool ortho_too_large(int64_t E, int64_t R, int64_t C)
{
    const int64_t n = std::max(R, C), tiles = ((R + 127) / 128) * ((C + 127) / 128);
    return n > 1 << 20 || E > 65535 || tiles > 1 << 21 || E * tiles > 1 << 26;
}

// The largest |s (a + b t + c t^2)| and |a + b t + c t^2| for t = s^2, s in [0, top] and a hundredth beyond, which covers
// what the roundings add to a singular value.
void bounds(const float* q, double top, double* x, double* b)
{
    const double A = q[0], B = q[1], C = q[2], T = 1.01 * top * (1.01 * top);
    double t[4] = {0.0, T, T, T};
    int n = 2;
    const double disc = 9 * B * B - 20 * A * C;                          // a + 3 b t + 5 c t^2 = 0
    if (C != 0 && disc >= 0) {
        t[n++] = (-3 * B + std::sqrt(disc)) / (10 * C);
        t[n++] = (-3 * B - std::sqrt(disc)) / (10 * C);
    } else if (C == 0 && B != 0) {
        t[n++] = -A / (3 * B);
    }
    *x = 0;
    for (int i = 0; i < n; ++i)
        if (t[i] >= 0 && t[i] <= T)
            *x = std::max(*x, std::fabs(std::sqrt(t[i]) * (A + B * t[i] + C * t[i] * t[i])));
    *b = std::max(std::fabs(A), std::fabs(A + B * T + C * T * T));
    if (C != 0 && -B / (2 * C) > 0 && -B / (2 * C) < T)
        *b = std::max(*b, std::fabs(A - B * B / (4 * C)));
}

// What B is stored times: 2048, or more where B is small (a last step that only scales: as 2048 times itself it came out off by
// 1e-2 for a = 1e-9, as zeros for 1e-11).
float scale_b(double most)
{
    float s = 2048.0f;
    while (most * s < 1024.0 && s < 0x1p110f)
        s *= 2.0f;
    return s;
}

// Whether a step that hardly scales X, where a is next to nothing, leaves X, A and B bits enough in fp16.  For m equal singular
// values of norm `low` in all, t = low^2 / m: A and B are off by 2^-25 in each entry where these are small (2 sqrt(m) of that in a
// matrix of m rows), so A of 2^-36 sqrt(m) and B of 2^-24 sqrt(m) / by; X of 2^-37 in each of m n entries.  At most 2^-7 of what
// they are part of is taken, of which about half is in the result's norm.  (0, 1, 0) twice, taken for up to 227 rows, comes out off by
// 5e-4 for 64, 4e-4 for 256, 1e-2 for 1024 and 0.5 for 2048 x 4096; (1/8, 1/2, 0) twice and (0, 1, 0), just taken for 2048 x 4096,
// by 2.6e-3.  The largest of the three terms stands for their sum, so that a polynomial may cross zero.  most: bound of B; `low`
// becomes what it is after the step.
bool leaves_bits(const float* q, double most, double m, double n, double* low)
{
    const double t = *low * *low / m, b = std::fabs((double)q[1]), c = std::fabs((double)q[2]);
    const double size = std::max(std::fabs((double)q[0]), std::max(b * t, c * t * t)), by = scale_b(most);
    if (size > 0 && (size < std::sqrt(m) * (0x1p-29 * (b + 2 * c * t) + 0x1p-17 / by) || *low < std::sqrt(m * n) * 0x1p-30))
        return false;
    *low = std::min(1.0, *low * size);
    return true;
}

// A launch: its tiles, and how many of the last ones go in quarters.  The least by a model of their times: rounds of a tile on
// each CU, whose time is (step + crowd * share of the CUs that have one) for 64 of the reduction, plus a start.  Quarters are
// tiles of half the width, one a CU as well (the workgroup keeps its LDS), so they pay up to a round or two of them; 64 x 64 tiles
// go two a CU and one after the other.  Constants from a sweep of 50 stacks, which they meet to 5 %; what is chosen is within 1 %
// of the best on average.  64 | 128 | 192 | 256 wide, q: the last ones in quarters, us:
//   X X^T  1024 x 4096 16 | 28 | 46 | 77,  2048 x 2048 26 | 20 | 30 | 44,  3200 x 3200 - | 61, q 57 | 47 | 67,  3840 x 3840 - | 71,
//          q 103 | 61 | 82,  4096 x 4096 - | 96, q 93 | 71 | 91,  4608 x 4608 - | 122, q 140 | 138 | 104,  5760 x 5760 - | 221,
//          q 220 | 188 | 253, q 198,  6400 x 6400 - | 288, q 345 | 301 | 339, q 259,  7168 x 7168 - | 433, q 422 | 339 | 375, q 363,
//          8192 x 8192 - | 587, q 578 | 508 | 553, q 487;  16 of 1024 x 2048 102 | 62, q 55 | 72 | 57,  28 of 512 x 512 22 | 20, q 17 | - | 21
//   A A    16 of 1024 x 1024 - | 44, q 38 | 51 | 40,  else like X X^T of a square
//   B X    1024 x 4096 20 | 16 | - | 33,  2048 x 5632 84 | 66, q 79 | - | 58,  3200 x 3200 - | 92, q 96 | - | 79,  4096 x 4096
//          226 | 148 | - | 119,  4608 x 4608 - | 223, q 223 | - | 253, q 195,  6400 x 6400 - | 549, q 585 | - | 513, q 455,
//          8192 x 8192 - | 1110 | - | 862;  16 of 1024 x 2048 134 | 114 | - | 84,  8 of 512 x 512 10 | 11 | - | 23
// (192 x 192 is 253 tiles of 4096 x 4096, a round; a column operand's swizzle has no such width.)  In parts | in one, five steps:
// 100 x 5440 84 | 129, 250 x 8000 121 | 188, 640 x 8192 215 | 250; 512 x 4096, in one, 149.
struct OrthoTiles {
    int size;
    int64_t rows, cols, all, cut;
    int splits, split_steps;         // workgroups of a tile, steps of 128 that each takes
};

struct TilePrice {
    double step, crowd, start;
};

OrthoTiles plan_tiles(int epi, int64_t E, int64_t M, int64_t N, int64_t K)
{
    constexpr TilePrice k128 = {0.28, 0.22, 6.5}, k192 = {0.32, 0.58, 17}, k256 = {0.86, 0.74, 15.5};
    constexpr TilePrice kQuarter128 = {0.11, 0.11, 3}, kQuarter256 = {0.26, 0.24, 3.5};
    const bool lower = epi != kEpiUpdate;
    int cus = 0;
    if (device_cus(&cus) != hipSuccess || cus <= 0)
        cus = 256;
    const double steps = (double)(K / 64);
    OrthoTiles best = {};
    double least = 1e30;
    // inside: how much of the tiles is
    auto rounds = [&](const TilePrice& p, int64_t tiles, double inside) {
        const int64_t rest = tiles % cus;
        return tiles / cus * ((p.step + p.crowd) * steps + p.start) +
               (rest ? (p.step + p.crowd * inside * rest / cus) * steps + p.start : 0);
    };
    for (const int size : {64, 128, 192, 256}) {
        if (size == 192 && !lower)
            continue;
        OrthoTiles t = {size, (M + size - 1) / size, (N + size - 1) / size, 0, 0, 1, 0};
        t.all = E * (lower ? t.rows * (t.rows + 1) / 2 : t.rows * t.cols);
        if (size == 64 && t.all > 8 * cus)             // (offsets of 32 bits)
            continue;
        const TilePrice& price = size == 128 ? k128 : size == 192 ? k192 : k256;
        const double launch = size == 128 ? 1 : 0;
        double us;
        if (size == 64) {
            const double pairs = (double)t.all / (2 * cus);
            us = t.all <= cus ? 0.16 * steps + 5.5 : lower ? 3 + pairs * (0.31 * steps + 8) : 3.5 + pairs * (0.39 * steps + 3.7);
            if (epi == kEpiGram)                       // what the tiles read between them
                us = std::max(us, 5.5 + 256.0 * t.all * K / 18e6);
        } else {
            const double area = E * (lower ? M * (M + (double)size) / 2 : (double)M * N) / (size * size);
            us = launch + rounds(price, t.all, std::min(1.0, area / t.all));
        }
        const int64_t rest = t.all % cus;
        if ((size == 128 || size == 256) && t.all > cus && rest) {
            const double cut = launch + rounds(price, t.all - rest, 1) + rounds(size == 128 ? kQuarter128 : kQuarter256, 4 * rest, 1);
            if (cut < us) {
                us = cut;
                t.cut = rest;
            }
        }
        if (us < least) {
            least = us;
            best = t;
        }
        // parts of a long reduction
        for (int64_t parts = 8; epi == kEpiGram && size == 64 && parts <= 32 && parts * t.all <= 2 * cus; parts += 8) {
            const int64_t each = (K / 128 + parts - 1) / parts;
            us = (parts * t.all > cus ? 0.72 : 0.33) * each + 8.5 + 0.018 * parts * t.all;
            if (us < least) {
                least = us;
                best = t;
                best.splits = (int)parts;
                best.split_steps = (int)each;
            }
        }
    }
    return best;
}

Ortho plan_ortho(int64_t E, int64_t R, int64_t C)
{
    Ortho o;
    o.m = std::min(R, C);
    o.n = std::max(R, C);
    o.mp = up(o.m, PAD);
    o.np = up(o.n, PAD);
    o.parts = (int)std::max<int64_t>(1, std::min<int64_t>(1024, R * C / 8192));
    int64_t at = 0;
    auto region = [&](int64_t bytes) {
        const int64_t here = at;
        at += up(bytes, 256);
        return here;
    };
    o.part = region(E * o.parts * 8);
    o.scale = region(E * 4);
    const OrthoTiles gram = plan_tiles(kEpiGram, E, o.mp, o.mp, o.np);
    o.counts = gram.splits > 1 ? E * gram.rows * gram.cols : 0;
    o.sums = region(o.counts * gram.splits * 16384);
    o.done = region(o.counts * 4);
    o.x0 = region(E * o.mp * o.np * 2);
    o.x1 = region(E * o.mp * o.np * 2);
    o.lo = region(E * o.mp * o.np * 2);                // (whether a remainder is kept the coefficients say, which are not known here)
    o.a = region(E * o.mp * o.mp * 2);
    o.b = region(E * o.mp * o.mp * 2);
    o.bytes = at;
    return o;
}

// kEpiGram, kEpiSquare: tiles at and below the diagonal; kEpiUpdate: all of them.
template <int EPI>
hipError_t launch_ortho(OrthoArgs a, hipStream_t s)
{
    int cus = 0;
    const hipError_t e = device_cus(&cus);
    if (e != hipSuccess)
        return e;
    const OrthoTiles t = plan_tiles(EPI, a.E, a.M, a.N, a.K);
    a.splits = t.splits;
    a.split_steps = t.split_steps;
    a.tiles_m = (int)t.rows;
    a.tiles_n = t.cols;
    a.cut = (int)t.cut;
    if (t.size == 64) {
        const dim3 tiles((unsigned)t.cols, (unsigned)t.rows, (unsigned)a.E);
        if constexpr (EPI == kEpiGram) {
            if (t.splits > 1) {
                const dim3 parts((unsigned)t.splits, tiles.x * tiles.y, tiles.z);
                if (t.all * t.splits > cus) {
                    a.split_steps *= 2;                // of 64
                    ortho64_kernel<EPI, 1, true><<<parts, dim3(NT), 0, s>>>(a);
                } else {
                    ortho64_kernel<EPI, 2, true><<<parts, dim3(NT), 0, s>>>(a);
                }
                return hipGetLastError();
            }
        }
        if (t.all <= cus)
            ortho64_kernel<EPI, 2, false><<<tiles, dim3(NT), 0, s>>>(a);
        else
            ortho64_kernel<EPI, 1, false><<<tiles, dim3(NT), 0, s>>>(a);
        return hipGetLastError();
    }
    const dim3 grid((unsigned)std::min(t.all - t.cut + 4 * t.cut, (int64_t)cus));
    switch (t.size) {
    case 128: ortho128_kernel<EPI><<<grid, dim3(NT), 0, s>>>(a); break;
    case 192:
        if constexpr (EPI != kEpiUpdate)
            ortho192_kernel<EPI><<<grid, dim3(NT), 0, s>>>(a);
        break;
    default: ortho256_kernel<EPI><<<grid, dim3(NT), 0, s>>>(a);
    }
    return hipGetLastError();
}

hipError_t launch_thin(const OrthoArgs& a, hipStream_t s)
{
    int cus = 0;
    const hipError_t e = device_cus(&cus);
    if (e != hipSuccess)
        return e;
    const int64_t rows = a.E * (a.M / 64), sharers = std::max<int64_t>(1, std::min(a.N / 64, (a.M == 128 ? 2 : 1) * cus / rows));
    const dim3 grid((unsigned)(rows * sharers));
    if (a.M == 128)
        ortho_thin_kernel<128><<<grid, dim3(NT), 0, s>>>(a);
    else
        ortho_thin_kernel<256><<<grid, dim3(NT), 0, s>>>(a);
    return hipGetLastError();
}

template <typename T>
void launch_start(const void* G, const Ortho& o, const StartArgs& a, int64_t E, hipStream_t s)
{
    const T* g = static_cast<const T*>(G);
    ortho_norm_kernel<T><<<dim3((unsigned)o.parts, (unsigned)E), dim3(256), 0, s>>>(g, a.R * a.C, const_cast<double*>(a.part));
    const dim3 grid((unsigned)(o.mp / 64 * (o.np / 64)), (unsigned)E);
    if (a.R > a.C)
        ortho_start_kernel<T, true><<<grid, dim3(256), 0, s>>>(g, a);
    else
        ortho_start_kernel<T, false><<<grid, dim3(256), 0, s>>>(g, a);
}

}  // namespace
}  // namespace lm
}  // namespace ag

using namespace ag;
using namespace ag::lm;

#define ORTHO_HIP(call, what)           \
    do {                                \
        const hipError_t e_ = (call);   \
        if (e_ != hipSuccess)           \
            return hip_error(e_, what); \
    } while (0)

extern "C" int64_t newton_schulz_workspace(int64_t E, int64_t R, int64_t C)
{
    if (E <= 0 || R <= 0 || C <= 0 || ortho_too_large(E, R, C))
        return 0;
    return plan_ortho(E, R, C).bytes;
}

extern "C" int newton_schulz(const void* G, int32_t g_type, int64_t E, int64_t R, int64_t C, const float* coefficients,
                             int32_t steps, float eps, void* out, void* work, int64_t work_bytes, void* stream)
{
    if (E < 0 || R < 0 || C < 0 || steps < 1 || !coefficients || !(eps >= 0.0f) || std::isinf(eps) ||
        (g_type != AG_TYPE_BF16 && g_type != AG_TYPE_F32))
        return AG_EINVAL;
    for (int64_t i = 0; i < 3 * (int64_t)steps; ++i)
        if (!std::isfinite(coefficients[i]))
            return AG_EINVAL;
    if (E == 0 || R == 0 || C == 0)
        return AG_OK;
    const auto bad = [](const void* p) { return !p || (reinterpret_cast<uintptr_t>(p) & 15); };
    if (bad(G) || bad(out))
        return AG_EINVAL;
    if (ortho_too_large(E, R, C))
        return AG_EUNSUPPORTED;
    // stored values: X, A and B of every step within fp16, and not all of X down where it has few bits
    double top = 1.0, low = 1.0;
    for (int32_t i = 0; i < steps; ++i) {
        double x, b;
        bounds(coefficients + 3 * i, top, &x, &b);
        if (top > 3.5 || top < 0.015625 || b > 28.0 ||
            !leaves_bits(coefficients + 3 * i, b, (double)std::min(R, C), (double)std::max(R, C), &low))
            return AG_EUNSUPPORTED;
        top = x;
    }
    const Ortho o = plan_ortho(E, R, C);
    if (work_bytes < o.bytes || bad(work))
        return AG_EINVAL;
    char* const ws = static_cast<char*>(work);
    hipStream_t s = static_cast<hipStream_t>(stream);
    auto half = [&](int64_t at) { return reinterpret_cast<_Float16*>(ws + at); };
    // what the steps after each multiply a rounding of its result by, among small singular directions
    auto keeps = [&](int32_t step) {
        double gain = 1.0;
        for (int32_t i = step + 1; i < steps; ++i)
            gain *= std::fabs((double)coefficients[3 * i]);
        return gain > 8.0;
    };
    bool kept = g_type == AG_TYPE_F32 && keeps(-1);
    float* const scale = reinterpret_cast<float*>(ws + o.scale);
    const StartArgs st = {R, C, o.mp, o.np, o.parts, eps, reinterpret_cast<double*>(ws + o.part), scale,
                          reinterpret_cast<uint32_t*>(ws + o.done), o.counts, half(o.x0),
                          kept ? half(o.lo) : nullptr};
    if (g_type == AG_TYPE_F32)
        launch_start<float>(G, o, st, E, s);
    else
        launch_start<__bf16>(G, o, st, E, s);
    ORTHO_HIP(hipGetLastError(), "launch newton_schulz start");
    double grown = 0.0;
    top = 1.0;
    int64_t cur = o.x0, next = o.x1;
    const int64_t xs = o.mp * o.np, as = o.mp * o.mp;
    for (int32_t i = 0; i < steps; ++i) {
        const float a = coefficients[3 * i], b = coefficients[3 * i + 1], c = coefficients[3 * i + 2];
        const bool keep = i + 1 < steps && keeps(i);
        double most;
        bounds(coefficients + 3 * i, top, &top, &most);
        const float by = scale_b(most);
        auto product = [&](int64_t A, int64_t lda, int64_t B, int64_t ldb, int64_t M, int64_t N, int64_t K, int64_t strideB) {
            OrthoArgs p = {};
            p.A = reinterpret_cast<const __bf16*>(ws + A);
            p.B = reinterpret_cast<const __bf16*>(ws + B);
            p.lda = lda;
            p.ldb = ldb;
            p.M = M;
            p.N = N;
            p.K = p.k_valid = K;
            p.E = (int)E;
            p.splits = 1;
            p.strideB = strideB;
            p.ldo = N;
            p.stride = M * N;
            return p;
        };
        OrthoArgs p = product(cur, o.np, cur, o.np, o.mp, o.mp, o.np, xs);
        p.alpha = kScaleA / (kScaleX * kScaleX);
        p.scale = scale;
        p.now = (float)grown;
        p.hi = half(o.a);
        p.sums = reinterpret_cast<float*>(ws + o.sums);
        p.done = reinterpret_cast<uint32_t*>(ws + o.done);
        ORTHO_HIP(launch_ortho<kEpiGram>(p, s), "launch newton_schulz X X^T");
        const float square_alpha = c * (by / (kScaleA * kScaleA)), square_beta = b * (by / kScaleA);
        const bool thin = o.mp <= 256;
        if (!thin) {
            p = product(o.a, o.mp, o.a, o.mp, o.mp, o.mp, o.mp, as);
            p.alpha = square_alpha;
            p.beta = square_beta;
            p.unit = a * by;
            p.add = half(o.a);
            p.hi = half(o.b);
            ORTHO_HIP(launch_ortho<kEpiSquare>(p, s), "launch newton_schulz A A");
        }
        p = product(thin ? o.a : o.b, o.mp, cur, o.np, o.mp, o.np, o.mp, xs);
        p.square_alpha = square_alpha;
        p.square_beta = square_beta;
        p.unit = a * by;
        p.alpha = 1.0f / by;
        p.beta = a;
        p.scale = scale;
        p.now = (float)grown;
        grown = std::max(1.0, (i ? grown : 1.0) * most);
        if (grown > 0x1p127)                           // from here on X itself, whatever the scale
            grown = INFINITY;
        p.next = i + 1 < steps ? (float)grown : 0.0f;
        p.add = kept ? half(o.lo) : nullptr;
        p.hi = half(next);
        p.lo = keep ? half(o.lo) : nullptr;
        if (i + 1 == steps) {
            p.alpha /= kScaleX;
            p.beta /= kScaleX;
            p.last = static_cast<__bf16*>(out);
            p.m = o.m;
            p.n = o.n;
            p.turned = R > C;
        }
        ORTHO_HIP(thin ? launch_thin(p, s) : launch_ortho<kEpiUpdate>(p, s), "launch newton_schulz B X");
        kept = keep;
        std::swap(cur, next);
    }
    return AG_OK;
}
