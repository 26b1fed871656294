// lm_norm.hip -- layer norm over rows, with the residual stream added in front, and its gradients: kernels and entry
// points.  All of it is bound by the bytes it moves.
//
//   h = bf16(x + residual),  m = mean(h),  r = 1 / sqrt(mean((h - m)^2) + eps),  y = (h - m) r w + b
//   xh = (h - m) r,  g = dy w:   dx = r (g - mean(g) - xh mean(g xh)) + dh,  dw = sum dy xh,  db = sum dy
//
// A row stays in registers between its one read and its one write: TPR threads have it in C pieces of eight columns each,
// so mean and variance are two sums over the same values and the variance is that of differences from the mean.  Rows
// wider than that go through memory (the caches) once for each sum.
#include "../../include/aggemm.h"
#include "ag_internal.hpp"
#include "lm_tile.hpp"

#include <algorithm>
#include <cmath>

namespace ag {
namespace lm {
namespace {

constexpr int kNormWidest = 16384;     // columns of a row in registers

struct NormArgs {
    const __bf16 *x, *residual, *w, *b;
    int64_t rows;
    int width;
    float eps;
    __bf16 *y, *h;
    float *mean, *rstd;
};

struct NormBwdArgs {
    const __bf16 *dy, *h, *w, *dh;
    const float *mean, *rstd;
    int64_t rows;
    int width;
    __bf16* dx;
    __bf16 *dw, *db;         // written by the kernel itself where one workgroup (row of them) has all rows
    float* part;             // [2][parts][width]: partial sums of dw and db; null: neither is wanted
    int64_t parts;
};

// The eight columns of a thread's piece, which may start anywhere: their last n are loaded from `lo` on, so that what is read
// ends with the row, and moved down by the s = 8 - n others, which come out as zeros.  No lane takes a way of its own (eight
// loads of one element each were that, and the registers for them).
struct Piece {
    int lo, s;
    __device__ __forceinline__ Piece(int col, int width) : lo(min(col, width - 8)), s(min(col - lo, 8)) {}
    __device__ __forceinline__ int n() const { return 8 - s; }
    __device__ __forceinline__ i32x4 load(const __bf16* row) const { return *reinterpret_cast<const i32x4_any*>(row + lo); }
    __device__ __forceinline__ bf16x8 take(const __bf16* row) const 
    {
        return __builtin_bit_cast(bf16x8, fit(load(row)));
    }
    __device__ __forceinline__ i32x4 fit(i32x4 v) const
    {
        if (s & 8)
            v = i32x4{};
        if (s & 4)
            v = i32x4{v[2], v[3], 0, 0};
        if (s & 2)
            v = i32x4{v[1], v[2], v[3], 0};
        if (s & 1)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                v[i] = (int)((uint32_t)v[i] >> 16 | (i < 3 ? (uint32_t)v[i < 3 ? i + 1 : i] << 16 : 0u));
        return v;
    }
};

// Eight columns of rows of any length, zeros past the n that are valid.
__device__ __forceinline__ bf16x8 take8(const __bf16* p, int n)
{
    if (n >= 8)
        return *reinterpret_cast<const bf16x8_any*>(p);
    bf16x8 v = load8_few(p, n);
#pragma unroll
    for (int e = 0; e < 8; ++e)
        v[e] = e < n ? v[e] : (__bf16)0.0f;
    return v;
}

// The stores leave the L2 caches to what is read, us: forward 16384 x 4096 99.5 | 96.1 so, 16384 x 8192 194 | 189, gradients
// 8192 x 14336 151 | 148, 65536 x 200 28.7 | 25.5 (forward 19.2 | 19.4).
__device__ __forceinline__ void give8(__bf16* p, int n, bf16x8 v)
{
    if (n >= 8) {
        __builtin_nontemporal_store(v, reinterpret_cast<bf16x8_any*>(p));
        return;
    }
#pragma unroll
    for (int e = 0; e < 7; ++e)
        if (e < n)
            p[e] = v[e];
}

// Value e of eight.  (As vectors of bf16 what is kept between its uses takes twice the registers.)
__device__ __forceinline__ float value(const i32x4& v, int e)
{
    return __builtin_bit_cast(float, e & 1 ? (uint32_t)v[e >> 1] & 0xFFFF0000u : (uint32_t)v[e >> 1] << 16);
}

__device__ __forceinline__ bf16x8 ones()
{
    const __bf16 x = (__bf16)1.0f;
    return bf16x8{x, x, x, x, x, x, x, x};
}

// x summed over N = 16, 32 or 64 neighbouring lanes: within 16 by the arithmetic's own lane exchange (the neighbour, the other
// pair, the other four and the other eight mirrored), which needs no LDS.
template <int N>
__device__ __forceinline__ float lanes_sum(float x)
{
    auto with = [&](auto ctrl) {
        x += __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), decltype(ctrl)::value, 0xF, 0xF, true));
    };
    with(std::integral_constant<int, 0xB1>());       // quad_perm [1, 0, 3, 2]
    with(std::integral_constant<int, 0x4E>());       // quad_perm [2, 3, 0, 1]
    with(std::integral_constant<int, 0x141>());      // row_half_mirror
    with(std::integral_constant<int, 0x140>());      // row_mirror
    if (N > 16)
        x += __shfl_xor(x, 16);
    if (N > 32)
        x += __shfl_xor(x, 32);
    return x;
}

// (a, b) summed over the TPR threads of a row; every one of them gets the sums.  `turn` counts the sums taken: two
// buffers in turn need one barrier each, for whoever writes one again has passed the barrier behind its last reads.
template <int TPR>
__device__ __forceinline__ float2 row_sum(float a, float b, float2 (*s_sum)[16], int& turn)
{
    a = lanes_sum<TPR < 64 ? TPR : 64>(a);
    b = lanes_sum<TPR < 64 ? TPR : 64>(b);
    if constexpr (TPR > 64) {
        float2* const buf = s_sum[turn++ & 1];
        if ((threadIdx.x & 63) == 0)
            buf[threadIdx.x >> 6] = make_float2(a, b);
        barrier_after_lds_write();
        a = b = 0.0f;
#pragma unroll
        for (int i = 0; i < TPR / 64; ++i) {
            a += buf[i].x;
            b += buf[i].y;
        }
    }
    return make_float2(a, b);
}

template <int TPR>
constexpr int kThreads = TPR > 256 ? TPR : 256;

// ------------------------------------------------------------------------------------------ forward
template <int TPR, int C>
__global__ __launch_bounds__(kThreads<TPR>) void norm_kernel(NormArgs a)
{
    constexpr int RPW = kThreads<TPR> / TPR;            // rows of a workgroup at a time
    __shared__ float2 s_sum[2][16];
    int turn = 0;
    const int t = RPW == 1 ? threadIdx.x : threadIdx.x % TPR, rl = RPW == 1 ? 0 : threadIdx.x / TPR;
    bf16x8 w[C], b[C];
    auto piece = [&](int c) { return Piece((c * TPR + t) * 8, a.width); };
#pragma unroll
    for (int c = 0; c < C; ++c) {
        w[c] = a.w ? piece(c).take(a.w) : ones();
        b[c] = a.b ? piece(c).take(a.b) : bf16x8{};
    }
    const float count = (float)a.width;
    for (int64_t row = blockIdx.x * (int64_t)RPW + rl; row < a.rows; row += gridDim.x * (int64_t)RPW) {
        const int64_t at = row * a.width;
        bf16x8 v[C], r[C];
#pragma unroll
        for (int c = 0; c < C; ++c)
            v[c] = piece(c).take(a.x + at);
        if (a.residual) {
#pragma unroll
            for (int c = 0; c < C; ++c)
                r[c] = piece(c).take(a.residual + at);
#pragma unroll
            for (int c = 0; c < C; ++c)
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    v[c][e] = (__bf16)((float)v[c][e] + (float)r[c][e]);
            if (a.h) {
#pragma unroll
                for (int c = 0; c < C; ++c)
                    give8(a.h + at + (c * TPR + t) * 8, piece(c).n(), v[c]);
            }
        }
        float sum = 0.0f;
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int e = 0; e < 8; ++e)
                sum += (float)v[c][e];
        const float mean = row_sum<TPR>(sum, 0.0f, s_sum, turn).x / count;
        float sq = 0.0f;
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float d = e < piece(c).n() ? (float)v[c][e] - mean : 0.0f;
                sq = fmaf(d, d, sq);
            }
        const float rstd = 1.0f / sqrtf(row_sum<TPR>(sq, 0.0f, s_sum, turn).x / count + a.eps);
#pragma unroll
        for (int c = 0; c < C; ++c) {
            bf16x8 o;
#pragma unroll
            for (int e = 0; e < 8; ++e)
                o[e] = (__bf16)fmaf(((float)v[c][e] - mean) * rstd, (float)w[c][e], (float)b[c][e]);
            give8(a.y + at + (c * TPR + t) * 8, piece(c).n(), o);
        }
        if (t == 0) {
            if (a.mean)
                a.mean[row] = mean;
            if (a.rstd)
                a.rstd[row] = rstd;
        }
    }
}

// Rows wider than kNormWidest: a workgroup of 1024 threads a row, three times over it.  A thread sees the same columns each
// time, and where h is kept reads the sum back from there (h may be x's or residual's own buffer).  With residual and h, us, beside
// what a copy of as many bytes takes: 6554 x 20480 286 (216), 6500 x 20001 382 (209), 1024 x 131072 308 (216), 128 x 2^20, which half
// of the CUs have, 505 (216); gradients with dh 332, 468, 359 and 543.  (8192 x 16384 in registers: 193 and 211, 216.)  Rows of
// fewer than 8 columns come here too and keep one thread of the 1024 at work: right, and slow, 13.2 ms for 2^20 rows of 4 where 8
// columns take 0.09.  They wait for a kernel of their own.
__global__ __launch_bounds__(1024) void norm_wide_kernel(NormArgs a)
{
    constexpr int TPR = 1024;
    __shared__ float2 s_sum[2][16];
    int turn = 0;
    const float count = (float)a.width;
    const bool add = a.residual != nullptr, kept = add && a.h;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const int64_t at = row * a.width;
        auto sum_at = [&](int col, int n) {
            bf16x8 v = take8(a.x + at + col, n);
            if (add) {
                const bf16x8 r = take8(a.residual + at + col, n);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    v[e] = (__bf16)((float)v[e] + (float)r[e]);
            }
            return v;
        };
        auto again = [&](int col, int n) { return kept ? take8(a.h + at + col, n) : sum_at(col, n); };
        float sum = 0.0f;
        for (int col = threadIdx.x * 8; col < a.width; col += TPR * 8) {
            const int n = min(a.width - col, 8);
            const bf16x8 v = sum_at(col, n);
            if (kept)
                give8(a.h + at + col, n, v);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                sum += (float)v[e];
        }
        const float mean = row_sum<TPR>(sum, 0.0f, s_sum, turn).x / count;
        float sq = 0.0f;
        for (int col = threadIdx.x * 8; col < a.width; col += TPR * 8) {
            const int n = min(a.width - col, 8);
            const bf16x8 v = again(col, n);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float d = e < n ? (float)v[e] - mean : 0.0f;
                sq = fmaf(d, d, sq);
            }
        }
        const float rstd = 1.0f / sqrtf(row_sum<TPR>(sq, 0.0f, s_sum, turn).x / count + a.eps);
        for (int col = threadIdx.x * 8; col < a.width; col += TPR * 8) {
            const int n = min(a.width - col, 8);
            const bf16x8 v = again(col, n);
            float w[8], b[8] = {};
#pragma unroll
            for (int e = 0; e < 8; ++e)
                w[e] = 1.0f;
            if (a.w)
                load8(a.w + col, n, w);
            if (a.b)
                load8(a.b + col, n, b);
            bf16x8 o;
#pragma unroll
            for (int e = 0; e < 8; ++e)
                o[e] = (__bf16)fmaf(((float)v[e] - mean) * rstd, w[e], b[e]);
            give8(a.y + at + col, n, o);
        }
        if (threadIdx.x == 0) {
            if (a.mean)
                a.mean[row] = mean;
            if (a.rstd)
                a.rstd[row] = rstd;
        }
    }
}

// ----------------------------------------------------------------------------------------- gradients
// Sums of 256 columns (32 lanes of eight) over rows [r0, r1), a row for each 32 of the N threads at a time, U of them ahead:
// into row `y` of the partial sums, or, without those, as dw and db.  `load`: eight columns of a row.
template <int N, int U, typename Load>
__device__ __forceinline__ void column_sums(const NormBwdArgs& a, int64_t r0, int64_t r1, int x, int y, Load load)
{
    constexpr int R = N / 32;
    __shared__ float s_sum[R][256 + 8];
    const int cl = threadIdx.x & 31, rl = threadIdx.x >> 5;
    const int col = x * 256 + cl * 8;
    float dw[8] = {}, db[8] = {};
    if (col < a.width) {
#pragma unroll U
        for (int64_t row = r0 + rl; row < r1; row += R) {
            float d[8], h[8];
            load(a.dy + row * a.width, col, d);
            load(a.h + row * a.width, col, h);
            const float mean = a.mean[row], rstd = a.rstd[row];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                dw[e] = fmaf(d[e], (h[e] - mean) * rstd, dw[e]);
                db[e] += d[e];
            }
        }
    }
    const int mine = x * 256 + threadIdx.x;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            s_sum[rl][cl * 8 + e] = k ? db[e] : dw[e];
        barrier_after_lds_write();
        if (threadIdx.x < 256 && mine < a.width) {
            float s = 0.0f;
#pragma unroll
            for (int r = 0; r < R; ++r)
                s += s_sum[r][threadIdx.x];
            __bf16* const out = k ? a.db : a.dw;
            if (a.part)
                a.part[(k * a.parts + y) * a.width + mine] = s;
            else if (out)
                out[mine] = (__bf16)s;
        }
        barrier_after_lds_write();
    }
}

// A workgroup's rows, and its share of the column sums in registers; `part` gets one row of them for each workgroup.
// SUMS: false leaves the columns out.
template <int TPR, int C, bool DH, bool SUMS>
__device__ __forceinline__ void norm_bwd_rows(const NormBwdArgs& a, int64_t first, int64_t workgroups)
{
    constexpr int NTH = kThreads<TPR>, RPW = NTH / TPR;
    __shared__ float2 s_sum[2][16];
    int turn = 0;
    const int t = RPW == 1 ? threadIdx.x : threadIdx.x % TPR, rl = RPW == 1 ? 0 : threadIdx.x / TPR;
    i32x4 w[C];
    float dw[C][8], db[C][8];
    auto piece = [&](int c) { return Piece((c * TPR + t) * 8, a.width); };
#pragma unroll
    for (int c = 0; c < C; ++c) {
        w[c] = a.w ? piece(c).fit(piece(c).load(a.w)) : __builtin_bit_cast(i32x4, ones());
#pragma unroll
        for (int e = 0; e < 8; ++e)
            dw[c][e] = db[c][e] = 0.0f;
    }
    const float inv = 1.0f / (float)a.width;
    // A row's loads go out while the one before it is computed (dh's with the row's own computation: its use comes last).
    // Two rows in turn, and loads without a condition (past the last row that one again): a copy of a row, or a branch
    // around its loads, would wait for them.
    struct Row {
        i32x4 dy[C], h[C];
        float mean, rstd;
    };
    auto fetch = [&](Row& r, int64_t row) {
        row = min(row, a.rows - 1);
        const int64_t at = row * a.width;
#pragma unroll
        for (int c = 0; c < C; ++c)
            r.dy[c] = piece(c).load(a.dy + at);
#pragma unroll
        for (int c = 0; c < C; ++c)
            r.h[c] = piece(c).load(a.h + at);
        r.mean = a.mean[row];
        r.rstd = a.rstd[row];
    };
    const int64_t step = workgroups * RPW;
    constexpr bool AHEAD = TPR < 1024 || !DH;          // the others have no registers for a second row
    auto compute = [&](Row& r, Row& next, int64_t row) {
        if constexpr (!AHEAD)
            fetch(r, row);
        i32x4 more[DH ? C : 1];
        auto fetch_more = [&] {
            if constexpr (DH) {
#pragma unroll
                for (int c = 0; c < C; ++c)
                    more[c] = piece(c).load(a.dh + row * a.width);
            }
        };
        if constexpr (AHEAD)
            fetch_more();
        if constexpr (AHEAD)
            fetch(next, row + step);
        __builtin_amdgcn_sched_barrier(0);
        i32x4 dy[C], h[C];
        float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            asm volatile("" : "+v"(w[c]));            // not eight floats from one row to the next
            dy[c] = piece(c).fit(r.dy[c]);
            h[c] = piece(c).fit(r.h[c]);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float off = value(h[c], e) - r.mean, d = value(dy[c], e);
                const float g = d * value(w[c], e);
                s1 += g;
                s2 = fmaf(g, off, s2);                 // times rstd at the end: past the row g is 0, but mean rstd may be infinite
                if constexpr (SUMS) {
                    dw[c][e] = fmaf(d, off * r.rstd, dw[c][e]);
                    db[c][e] += d;
                    asm volatile("" : "+v"(dw[c][e]), "+v"(db[c][e]));   // added now, not behind the sums over the row
                }
            }
            __builtin_amdgcn_sched_barrier(0);         // one piece's temporaries at a time
        }
        if constexpr (!AHEAD)
            fetch_more();
        const float2 s = row_sum<TPR>(s1, s2, s_sum, turn);
        const float m1 = s.x * inv, m2 = s.y * inv * r.rstd;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            // g and xh again from what is packed: kept, they are sixteen registers for each piece
            asm volatile("" : "+v"(dy[c]), "+v"(h[c]), "+v"(w[c]));
            const i32x4 d = DH ? piece(c).fit(more[DH ? c : 0]) : i32x4{};
            bf16x8 o;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float xh = (value(h[c], e) - r.mean) * r.rstd, g = value(dy[c], e) * value(w[c], e);
                o[e] = (__bf16)fmaf(r.rstd, g - m1 - xh * m2, value(d, e));
            }
            if (a.dx)
                give8(a.dx + row * a.width + (c * TPR + t) * 8, piece(c).n(), o);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    int64_t row = first * RPW + rl;
    Row r0, r1;
    if constexpr (AHEAD)
        fetch(r0, row);
    while (row < a.rows) {
        compute(r0, r1, row);
        row += step;
        if constexpr (AHEAD) {
            if (row >= a.rows)
                break;
            compute(r1, r0, row);
            row += step;
        }
    }
    if (!SUMS || !a.part)
        return;
    float* const out = a.part + first * a.width;
    const int64_t second = a.parts * a.width;              // from dw's sums to db's
    if constexpr (TPR >= 256) {
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (e < piece(c).n()) {
                    const int col = (c * TPR + t) * 8 + e;
                    out[col] = dw[c][e];
                    out[second + col] = db[c][e];
                }
    } else {
        // rows that lanes of a wave have side by side, then those of the four waves
        __shared__ float s_col[4][TPR * C * 8];
        const int wave = threadIdx.x >> 6;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
#pragma unroll
            for (int c = 0; c < C; ++c)
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    float v = k ? db[c][e] : dw[c][e];
#pragma unroll
                    for (int s = TPR; s < 64; s <<= 1)
                        v += __shfl_xor(v, s);
                    if ((threadIdx.x & 63) < TPR)
                        s_col[wave][(c * TPR + t) * 8 + e] = v;
                }
            barrier_after_lds_write();
            for (int col = threadIdx.x; col < a.width; col += NTH)
                out[k * second + col] = (s_col[0][col] + s_col[1][col]) + (s_col[2][col] + s_col[3][col]);
            barrier_after_lds_write();
        }
    }
}

template <int TPR, int C, bool DH>
__global__ __launch_bounds__(kThreads<TPR>) void norm_bwd_kernel(NormBwdArgs a)
{
    norm_bwd_rows<TPR, C, DH, true>(a, blockIdx.x, gridDim.x);
}

// Few rows: workgroups for the rows and, after them, for the columns, which read the same again and leave no partial sums to
// be joined by another launch.
template <int TPR, int C, bool DH>
__global__ __launch_bounds__(kThreads<TPR>) void norm_bwd_few_kernel(NormBwdArgs a, int row_workgroups)
{
    if ((int)blockIdx.x < row_workgroups) {
        norm_bwd_rows<TPR, C, DH, false>(a, blockIdx.x, row_workgroups);
    } else {
        column_sums<kThreads<TPR>, 4>(a, 0, a.rows, blockIdx.x - row_workgroups, 0, [&](const __bf16* row, int col, float* x) {
            const i32x4 v = Piece(col, a.width).fit(Piece(col, a.width).load(row));
#pragma unroll
            for (int e = 0; e < 8; ++e)
                x[e] = value(v, e);
        });
    }
}

// Column sums of rows wider than kNormWidest, a chunk of them
__global__ __launch_bounds__(256) void norm_cols_kernel(NormBwdArgs a, int64_t chunk)
{
    const int64_t r0 = blockIdx.y * chunk;
    column_sums<256, 1>(a, r0, min(a.rows, r0 + chunk), blockIdx.x, blockIdx.y,
                [&](const __bf16* row, int col, float* x) { load8(row + col, min(a.width - col, 8), x); });
}

// dx of rows wider than kNormWidest
__global__ __launch_bounds__(1024) void norm_bwd_wide_kernel(NormBwdArgs a)
{
    constexpr int TPR = 1024;
    __shared__ float2 s_sum[2][16];
    int turn = 0;
    const float count = (float)a.width;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const int64_t at = row * a.width;
        const float mean = a.mean[row], rstd = a.rstd[row];
        auto values = [&](int col, int n, float* g, float* off) {
            float w[8];
#pragma unroll
            for (int e = 0; e < 8; ++e)
                w[e] = 1.0f;
            load8(a.dy + at + col, n, g);
            load8(a.h + at + col, n, off);
            if (a.w)
                load8(a.w + col, n, w);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                g[e] *= w[e];
                off[e] -= mean;
            }
        };
        float s1 = 0.0f, s2 = 0.0f;
        for (int col = threadIdx.x * 8; col < a.width; col += TPR * 8) {
            float g[8], off[8];
            values(col, min(a.width - col, 8), g, off);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                s1 += g[e];
                s2 = fmaf(g[e], off[e], s2);
            }
        }
        const float2 s = row_sum<TPR>(s1, s2, s_sum, turn);
        const float m1 = s.x / count, m2 = s.y / count * rstd;
        for (int col = threadIdx.x * 8; col < a.width; col += TPR * 8) {
            const int n = min(a.width - col, 8);
            float g[8], off[8], dh[8] = {};
            values(col, n, g, off);
            if (a.dh)
                load8(a.dh + at + col, n, dh);
            bf16x8 o;
#pragma unroll
            for (int e = 0; e < 8; ++e)
                o[e] = (__bf16)fmaf(rstd, g[e] - m1 - off[e] * rstd * m2, dh[e]);
            give8(a.dx + at + col, n, o);
        }
    }
}

// dw and db from their partial sums: 32 columns of a workgroup, each summed by eight threads.
__global__ __launch_bounds__(256) void norm_join_kernel(const float* part, int64_t parts, int width, __bf16* dw, __bf16* db)
{
    __shared__ float s_sum[8][32];
    const int cl = threadIdx.x & 31, rl = threadIdx.x >> 5;
    const int col = blockIdx.x * 32 + cl;
    __bf16* const out = blockIdx.y ? db : dw;
    if (!out)
        return;
    const float* p = part + blockIdx.y * parts * width + col;
    float s = 0.0f;
    if (col < width) {
#pragma unroll 8
        for (int64_t r = rl; r < parts; r += 8)
            s += p[r * width];
    }
    s_sum[rl][cl] = s;
    barrier_after_lds_write();
    if (rl == 0 && col < width) {
#pragma unroll
        for (int r = 1; r < 8; ++r)
            s += s_sum[r][cl];
        out[col] = (__bf16)s;
    }
}

// rows of less than one piece go the way of the widest ones
bool in_registers(int64_t width) { return width >= 8 && width <= kNormWidest; }

int64_t cus()
{
    int n = 0;
    if (device_cus(&n) != hipSuccess || n <= 0)
        n = 256;
    return n;
}

// f(TPR, C, workgroups a CU): the threads and pieces of rows of `width` <= kNormWidest columns.  As few threads as have
// columns each, pieces enough to be in flight, and no more workgroups than that takes: each walks through memory at a place
// of its own.  us for 65536 rows up to 2000 columns, 2^27 values beyond; the first is what is taken:
//    100 columns, 16 threads 11.9, 4 workgroups a CU 12.5, 64 threads 30;    200, 32 threads 19.0, 19.9, 64 threads 29
//    500, 64 threads 46.2, 4 a CU 46.1, 256 threads 102;    1000, 64 of two pieces 98.6, 8 a CU 110, 256 threads 123
//   2000, 256 threads 205, 8 a CU 217, 64 of four pieces 275;    4096, 256 of two 193, 8 a CU 211, 512 threads 200
//   8192, 512 of two 194, 4 a CU 214, 256 of four 193 at 4;    14336, 512 of four 208, 4 a CU 255, 1024 of two 218
template <typename F>
auto forward_by_width(int64_t width, F f)
{
    using std::integral_constant;
#define AG_NORM(TPR, C, PER) return f(integral_constant<int, TPR>(), integral_constant<int, C>(), PER)
    if (width <= 128)
        AG_NORM(16, 1, 8);
    if (width <= 256)
        AG_NORM(32, 1, 8);
    if (width <= 512)
        AG_NORM(64, 1, 8);
    if (width <= 1024)
        AG_NORM(64, 2, 4);
    if (width <= 2048)
        AG_NORM(256, 1, 4);
    if (width <= 4096)
        AG_NORM(256, 2, 4);
    if (width <= 8192)
        AG_NORM(512, 2, 2);
    AG_NORM(512, 4, 2);
}

// The same for the gradients, whose partial sums are a row for each workgroup.  us at 1 | 2 | 4 workgroups a CU, with dh; without:
//    100 columns 21 | 19 | 21; 19 | 18 | 19    500 62 | 50 | 52; 54 | 41 | 43    1000 107 | 108 | 116; 94 | 82 | 91
//   2000, 64 threads of four pieces 205 | 226 | 230; 150 | 166 | 174, 256 threads 297 | 215 | 235; 234 | 180 | 173
//   4096, 256 threads of two 207 | 216 | 228; 168 | 169 | 178, 512 threads 207 | 213 | 226; 188 | 164 | 181
//   8192, 512 of two 200 | 216 | 245; 157 | 173 | 192, 256 of four 205 | 222 | 255; 158 | 176 | 194
//  14336, 1024 of two 215 | 239 | 282; 173 | 195 | 240, 512 of four 223 | 248 | 293; 176 | 194 | 246
template <typename F>
auto backward_by_width(int64_t width, F f)
{
    using std::integral_constant;
    if (width <= 128)
        AG_NORM(16, 1, 2);
    if (width <= 256)
        AG_NORM(32, 1, 2);
    if (width <= 512)
        AG_NORM(64, 1, 2);
    if (width <= 1024)
        AG_NORM(64, 2, 2);
    if (width <= 2048)
        AG_NORM(64, 4, 1);
    if (width <= 4096)
        AG_NORM(256, 2, 1);
    if (width <= 8192)
        AG_NORM(512, 2, 1);
    AG_NORM(1024, 2, 1);
#undef AG_NORM
}

int64_t row_workgroups(int64_t rows, int tpr, int per_cu)
{
    const int at_a_time = std::max(1, 256 / tpr);
    return std::min((rows + at_a_time - 1) / at_a_time, cus() * per_cu);
}

// Gradients for rows that few workgroups read twice rather than another launch join their sums.  With dh, us, in one launch | two,
// called one after the other from Python, where two launches cost the host 16:
//    256 columns  64 rows 11.8 | 16.1, 128 12.0 | 16.0, 256 13.6 | 16.1, 320 16.6 | 16.1;   1024, 256 rows 14.0 | 16.2, 320 16.8 | 16.2
//   4096, 256 rows 14.6 | 16.1, 320 17.5 | 16.2;   8192, 256 rows 11.8 | 24.2, 320 13.2 | 25.1;   14336, 320 rows 17.6 | 33.9
// The sides cross near 290 rows up to 4096 columns: the limit.  On the device alone (replayed in a graph) they cross earlier where
// rows are narrow and a column's sum, 32 rows at a time, is what takes long, and later where they are wide:
//    256 columns  64 rows 5.0 | 5.8, 128 8.1 | 6.0, 256 14.0 | 6.5;   1024, 64 rows 5.5 | 6.4, 256 14.2 | 6.4;   2000, 160 rows 9.8 | 10.0
//   4096, 256 rows 15.0 | 15.2;   8192, 384 rows 19.6 | 24.6;   14336, 256 rows 14.7 | 31.8, 448 23.1 | 35.3
// One rule serves both, for the sums' order is to be the shape's alone.  Rows past 8192 columns, where a kernel of 1024 threads would
// join in, go the other way, at the figures above.
bool few_rows(int64_t rows, int64_t width) { return in_registers(width) && width <= 8192 && rows <= 256; }

// rows of partial sums
int64_t bwd_parts(int64_t rows, int64_t width)
{
    if (rows <= 0 || width <= 0)
        return 0;
    // Eight threads have a column in each part.  Rows too wide for registers are few; of narrow ones there may be 2^30: then a
    // thread adds 2^17 of them up, as many as where rows of 8 columns are in registers (in 32 parts it was 2^22, and a dbias of
    // 2^27 gradients of one sign came out 0.8 % small).
    if (!in_registers(width))
        return std::min<int64_t>((rows + 31) / 32, width < 8 ? 1024 : 32);
    if (few_rows(rows, width))
        return 0;
    return backward_by_width(width, [&](auto tpr, auto, int per) { return row_workgroups(rows, decltype(tpr)::value, per); });
}

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
bool bad(const void* p, uintptr_t n) { return !p || !aligned(p, n); }

bool norm_too_large(int64_t rows, int64_t width) { return width > 1 << 21 || rows > (int64_t)1 << 30; }

}  // namespace
}  // namespace lm
}  // namespace ag

using namespace ag;
using namespace ag::lm;

#define NORM_HIP(what)                      \
    do {                                    \
        const hipError_t e_ = hipGetLastError(); \
        if (e_ != hipSuccess)               \
            return hip_error(e_, what);     \
    } while (0)

extern "C" int layer_norm(const void* x, const void* residual, const void* weight, const void* bias, int64_t rows,
                          int64_t width, float eps, void* y, void* h, float* mean, float* rstd, void* stream)
{
    if (rows < 0 || width < 0 || !(eps >= 0.0f) || std::isinf(eps))
        return AG_EINVAL;
    if (rows == 0 || width == 0)
        return AG_OK;
    if (bad(x, 16) || bad(y, 16) || !aligned(residual, 16) || !aligned(weight, 16) || !aligned(bias, 16) ||
        !aligned(h, 16) || !aligned(mean, 4) || !aligned(rstd, 4) || (h && !residual))
        return AG_EINVAL;
    if (norm_too_large(rows, width))
        return AG_EUNSUPPORTED;
    const NormArgs a = {static_cast<const __bf16*>(x), static_cast<const __bf16*>(residual),
                        static_cast<const __bf16*>(weight), static_cast<const __bf16*>(bias), rows, (int)width, eps,
                        static_cast<__bf16*>(y), static_cast<__bf16*>(h), mean, rstd};
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (!in_registers(width))
        norm_wide_kernel<<<dim3((unsigned)std::min(rows, cus() * 2)), dim3(1024), 0, s>>>(a);
    else
        forward_by_width(width, [&](auto tpr, auto c, int per) {
            constexpr int T = decltype(tpr)::value, C = decltype(c)::value;
            norm_kernel<T, C><<<dim3((unsigned)row_workgroups(rows, T, per)), dim3(kThreads<T>), 0, s>>>(a);
        });
    NORM_HIP("launch layer_norm");
    return AG_OK;
}

extern "C" int64_t layer_norm_bwd_workspace(int64_t rows, int64_t width)
{
    if (rows < 0 || width < 0 || norm_too_large(rows, width))
        return 0;
    return bwd_parts(rows, width) * width * 8;
}

extern "C" int layer_norm_bwd(const void* dy, const void* h, const float* mean, const float* rstd, const void* weight,
                              const void* dh, int64_t rows, int64_t width, void* dx, void* dweight, void* dbias, void* work,
                              int64_t work_bytes, void* stream)
{
    if (rows < 0 || width < 0)
        return AG_EINVAL;
    if (width == 0)
        return AG_OK;
    if ((rows > 0 && (bad(dy, 16) || bad(h, 16) || bad(mean, 4) || bad(rstd, 4))) || !aligned(weight, 16) ||
        !aligned(dh, 16) || !aligned(dx, 16) || !aligned(dweight, 16) || !aligned(dbias, 16))
        return AG_EINVAL;
    if (norm_too_large(rows, width))
        return AG_EUNSUPPORTED;
    const int64_t parts = bwd_parts(rows, width);
    const bool sums = dweight || dbias;
    if (sums && (work_bytes < parts * width * 8 || (parts > 0 && bad(work, 16))))
        return AG_EINVAL;
    if (!dx && !sums)
        return AG_OK;
    hipStream_t s = static_cast<hipStream_t>(stream);
    const NormBwdArgs a = {static_cast<const __bf16*>(dy), static_cast<const __bf16*>(h), static_cast<const __bf16*>(weight),
                           static_cast<const __bf16*>(dh), mean, rstd, rows, (int)width, static_cast<__bf16*>(dx),
                           static_cast<__bf16*>(dweight), static_cast<__bf16*>(dbias),
                           sums && parts > 0 ? static_cast<float*>(work) : nullptr, parts};
    if (rows > 0 && !in_registers(width)) {
        if (dx)
            norm_bwd_wide_kernel<<<dim3((unsigned)std::min(rows, cus() * 2)), dim3(1024), 0, s>>>(a);
        if (sums)
            norm_cols_kernel<<<dim3((unsigned)((width + 255) / 256), (unsigned)parts), dim3(256), 0, s>>>(
                a, (rows + parts - 1) / parts);
    } else if (few_rows(rows, width) && sums && rows > 0) {
        backward_by_width(width, [&](auto tpr, auto c, int) {
            constexpr int T = decltype(tpr)::value, C = decltype(c)::value;
            if constexpr (T < 1024) {
                const int row_wgs = dx ? (int)((rows * T + kThreads<T> - 1) / kThreads<T>) : 0;
                const dim3 grid((unsigned)(row_wgs + (width + 255) / 256)), block(kThreads<T>);
                if (dx && dh)
                    norm_bwd_few_kernel<T, C, true><<<grid, block, 0, s>>>(a, row_wgs);
                else
                    norm_bwd_few_kernel<T, C, false><<<grid, block, 0, s>>>(a, row_wgs);
            }
        });
        NORM_HIP("launch layer_norm_bwd");
        return AG_OK;
    } else if (rows > 0) {
        backward_by_width(width, [&](auto tpr, auto c, int per) {
            constexpr int T = decltype(tpr)::value, C = decltype(c)::value;
            const dim3 grid((unsigned)row_workgroups(rows, T, per)), block(kThreads<T>);
            if (dx && dh)
                norm_bwd_kernel<T, C, true><<<grid, block, 0, s>>>(a);
            else
                norm_bwd_kernel<T, C, false><<<grid, block, 0, s>>>(a);
        });
    }
    NORM_HIP("launch layer_norm_bwd");
    if (sums) {
        norm_join_kernel<<<dim3((unsigned)((width + 31) / 32), 2), dim3(256), 0, s>>>(
            static_cast<const float*>(work), parts, (int)width, static_cast<__bf16*>(dweight), static_cast<__bf16*>(dbias));
        NORM_HIP("launch layer_norm join");
    }
    return AG_OK;
}
