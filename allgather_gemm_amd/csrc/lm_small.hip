// lm_small.hip -- what runs before and after the tiled products of the language-model operators:
// joining a split reduction, the activation's slope with the bias gradient, the softmax statistics.
// All are bound by the bytes they move.
#include "ag_internal.hpp"
#include "lm_tile.hpp"

#include <algorithm>

namespace ag {
namespace lm {
namespace {

// Eight columns of one row per unit: the fp32 sums of the splits.  L threads share a unit where there are
// few units and many splits (thread l adds splits l, l + L, ... in that order, then the L sums are added in
// theirs), so that enough loads are in flight: 64 splits of 33 x 1024 took 20 us with L = 1.  u0: the launch's first unit.
template <int L>
__global__ __launch_bounds__(NT) void join_kernel(const float* part, int splits, int64_t M, int64_t N, int64_t ldp,
                                                  LinearOut out, int64_t u0, const float* dloss,
                                                  int64_t dloss_rows)
{
    const float unit = loss_unit(loss_sample(dloss, dloss_rows));
    constexpr int U = NT / L;                      // units of a workgroup
    __shared__ f32x4 s_sum[L > 1 ? L - 1 : 1][U][2];
    const int64_t units = ldp / 8;
    const int ul = threadIdx.x % U, sl = threadIdx.x / U;
    const int64_t u = u0 + blockIdx.x * (int64_t)U + ul;
    const bool there = u < M * units;
    const int64_t row = there ? u / units : 0, col = there ? (u - row * units) * 8 : 0;
    f32x4 s0 = {}, s1 = {};
    if (there) {
        const float* p = part + row * ldp + col;
#pragma unroll 4
        for (int s = sl; s < splits; s += L) {
            const f32x4* q = reinterpret_cast<const f32x4*>(p + s * M * ldp);
            s0 += q[0];
            s1 += q[1];
        }
    }
    if (L > 1) {
        if (sl > 0) {
            s_sum[sl - 1][ul][0] = s0;
            s_sum[sl - 1][ul][1] = s1;
        }
        __syncthreads();
        if (sl > 0)
            return;
#pragma unroll
        for (int l = 0; l < L - 1; ++l) {
            s0 += s_sum[l][ul][0];
            s1 += s_sum[l][ul][1];
        }
    }
    float x[8] = {s0[0] * unit, s0[1] * unit, s0[2] * unit, s0[3] * unit,
                  s1[0] * unit, s1[1] * unit, s1[2] * unit, s1[3] * unit};
    const int n = (int)min((int64_t)8, N - col);
    if (!there || n <= 0)
        return;
    linear8(out, row, col, n, x);
}

constexpr int COLS = 256;      // columns of a workgroup of act_bwd_kernel: 32 lanes of 8

// d = dC act'(pre), rounded to bf16 (at most 2^-8 of it) for the two products, whose matrix instructions take both
// factors so; its column sums from the unrounded values.  The gradients of 8192 x 8192 x 8192 with gelu are then 0.00233
// of their norm off, 0.00166 if d were not rounded; two bf16 parts of it would double the products.
template <int R>
__global__ __launch_bounds__(NT) void act_bwd_kernel(const __bf16* dC, const __bf16* pre, int act, int64_t M, int64_t N,
                                                     int64_t chunk, __bf16* d, int64_t ldd, float* colsum,
                                                     __bf16* dbias)
{
    __shared__ float s_sum[8][COLS + 8];
    const int cl = threadIdx.x & 31, rl = threadIdx.x >> 5;
    const int64_t col = blockIdx.x * (int64_t)COLS + cl * 8;
    const int64_t r0 = blockIdx.y * chunk, r1 = min(M, r0 + chunk);
    const int n = (int)max((int64_t)0, min((int64_t)8, N - col));
    float sum[8] = {};
    // R rows of a thread at a time, their loads ahead of what is computed of the first
    auto rows = [&](auto load) {
        for (int64_t row0 = r0 + rl; row0 < r1; row0 += 8 * R) {
            float x[R][8], z[R][8];
#pragma unroll
            for (int i = 0; i < R; ++i) {
                const int64_t row = min(row0 + i * 8, r1 - 1);
                load(dC + row * N + col, x[i]);
                if (act != kActNone)
                    load(pre + row * N + col, z[i]);
            }
#pragma unroll
            for (int i = 0; i < R; ++i) {
                const int64_t row = row0 + i * 8;
                if (row >= r1)
                    break;
                if (act != kActNone)
                    act_slope8(x[i], z[i], act);
                if (d && col < ldd) {
                    bf16x8 o;
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        o[e] = (__bf16)x[i][e];
                    *reinterpret_cast<bf16x8*>(d + row * ldd + col) = o;
                }
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    sum[e] += x[i][e];
            }
        }
    };
    if (n < 8)
        rows([&](const __bf16* p, float* x) { load8(p, n, x); });
    else
        rows([](const __bf16* p, float* x) { load8(p, 8, x); });
    if (!dbias)
        return;
#pragma unroll
    for (int e = 0; e < 8; ++e)
        s_sum[rl][cl * 8 + e] = sum[e];
    __syncthreads();
    const int64_t c = blockIdx.x * (int64_t)COLS + threadIdx.x;
    if (c < N) {
        float s = 0.0f;
#pragma unroll
        for (int r = 0; r < 8; ++r)
            s += s_sum[r][threadIdx.x];
        if (gridDim.y == 1)
            dbias[c] = (__bf16)s;
        else
            colsum[blockIdx.y * N + c] = s;
    }
}

// 64 columns of a workgroup, each summed by four threads (rows r, r + 4, ... of the partial sums).
__global__ __launch_bounds__(NT) void colsum_join_kernel(const float* colsum, int64_t rows, int64_t N, __bf16* out)
{
    __shared__ float s_sum[4][64];
    const int cl = threadIdx.x & 63, rl = threadIdx.x >> 6;
    const int64_t c = blockIdx.x * (int64_t)64 + cl;
    float s = 0.0f;
    if (c < N) {
#pragma unroll 8
        for (int64_t r = rl; r < rows; r += 4)
            s += colsum[r * N + c];
    }
    s_sum[rl][cl] = s;
    __syncthreads();
    if (rl == 0 && c < N)
        out[c] = (__bf16)((s_sum[0][cl] + s_sum[1][cl]) + (s_sum[2][cl] + s_sum[3][cl]));
}

// The pieces' (maximum, sum) pairs of a row under one maximum.  W waves share a row: one, or four where a
// row has so many pairs that one wave would read them in more than eight rounds.
template <int W>
__global__ __launch_bounds__(NT) void xent_join_kernel(const float* stat, int64_t stat_n, const float* hit,
                                                       const int64_t* targets, int64_t T, int64_t vocab, float* loss,
                                                       float* lse)
{
    __shared__ float s_red[2][4];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t row = W == 1 ? blockIdx.x * (int64_t)(NT / 64) + wave : blockIdx.x;
    if (row >= T)
        return;
    const float2* p = reinterpret_cast<const float2*>(stat) + row * stat_n;
    const int64_t i0 = W == 1 ? lane : threadIdx.x;
    float mx = -INFINITY;
#pragma unroll 4
    for (int64_t i = i0; i < stat_n; i += W * 64)
        mx = fmaxf(mx, p[i].x);
#pragma unroll
    for (int s = 1; s < 64; s <<= 1)
        mx = fmaxf(mx, __shfl_xor(mx, s));
    if (W > 1) {
        if (lane == 0)
            s_red[0][wave] = mx;
        __syncthreads();
        mx = fmaxf(fmaxf(s_red[0][0], s_red[0][1]), fmaxf(s_red[0][2], s_red[0][3]));
    }
    const float base = mx == -INFINITY ? 0.0f : mx;
    float sum = 0.0f;
#pragma unroll 4
    for (int64_t i = i0; i < stat_n; i += W * 64) {
        const float2 v = p[i];
        sum += v.y * (v.x == -INFINITY ? (v.y != v.y ? v.y : 0.0f) : fast_exp(v.x - base));
    }
#pragma unroll
    for (int s = 1; s < 64; s <<= 1)
        sum += __shfl_xor(sum, s);
    if (W > 1) {
        if (lane == 0)
            s_red[1][wave] = sum;
        __syncthreads();
        sum = (s_red[1][0] + s_red[1][1]) + (s_red[1][2] + s_red[1][3]);
    }
    if (i0 == 0) {
        const float l = base + logf(sum);
        const int64_t y = targets[row];
        lse[row] = l;
        loss[row] = (y >= 0 && y < vocab) ? l - hit[row] : 0.0f;
    }
}

}  // namespace

hipError_t launch_join(const float* part, int splits, int64_t M, int64_t N, int64_t ldp, const LinearOut& out,
                       hipStream_t stream, const float* dloss, int64_t dloss_rows)
{
    const int64_t units = M * (ldp / 8);
    if (units <= 0)
        return hipSuccess;
    // four threads a unit once that leaves the chip's CUs with less than four workgroups each, sixteen likewise
    const int L = splits >= 32 && units < 16384 ? 16 : splits >= 8 && units < 65536 ? 4 : 1;
    const int64_t groups = (units * L + NT - 1) / NT;
    for (int64_t g = 0; g < groups; g += kMostWorkgroups) {
        const dim3 grid((unsigned)std::min(groups - g, kMostWorkgroups));
        const int64_t u0 = g * (NT / L);
        if (L == 16)
            join_kernel<16><<<grid, dim3(NT), 0, stream>>>(part, splits, M, N, ldp, out, u0, dloss, dloss_rows);
        else if (L == 4)
            join_kernel<4><<<grid, dim3(NT), 0, stream>>>(part, splits, M, N, ldp, out, u0, dloss, dloss_rows);
        else
            join_kernel<1><<<grid, dim3(NT), 0, stream>>>(part, splits, M, N, ldp, out, u0, dloss, dloss_rows);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess)
            return e;
    }
    return hipSuccess;
}

// Rows of one workgroup: a multiple of its 8 row lanes, at most 128 workgroups down the rows.  (With one the sums need
// no joining.)
static int64_t act_chunk(int64_t M) { return std::max<int64_t>(32, ((M + 127) / 128 + 7) / 8 * 8); }

int64_t colsum_rows(int64_t M) { return (M + act_chunk(M) - 1) / act_chunk(M); }

hipError_t launch_act_bwd(const __bf16* dC, const __bf16* pre, int act, int64_t M, int64_t N, __bf16* d, int64_t ldd,
                          float* colsum, __bf16* dbias, hipStream_t stream)
{
    if (M <= 0 || N <= 0)
        return hipSuccess;
    const dim3 grid((unsigned)((N + COLS - 1) / COLS), (unsigned)colsum_rows(M));
    // rows in flight a thread, four | one, us: 8192 x 8192 gelu 75-80 | 82-86, 8192 x 14336 silu 121 | 129; where
    // rows do not start on 16 bytes, 8191 x 8191 gelu 130 | 112-117, 47 x 10749 relu 11-12 | 7.5
    if (N % 8 == 0)
        act_bwd_kernel<4><<<grid, dim3(NT), 0, stream>>>(dC, pre, act, M, N, act_chunk(M), d, ldd, colsum, dbias);
    else
        act_bwd_kernel<1><<<grid, dim3(NT), 0, stream>>>(dC, pre, act, M, N, act_chunk(M), d, ldd, colsum, dbias);
    return hipGetLastError();
}

hipError_t launch_colsum_join(const float* colsum, int64_t rows, int64_t N, __bf16* out, hipStream_t stream)
{
    if (N <= 0)
        return hipSuccess;
    colsum_join_kernel<<<dim3((unsigned)((N + 63) / 64)), dim3(NT), 0, stream>>>(colsum, rows, N, out);
    return hipGetLastError();
}

hipError_t launch_xent_join(const float* stat, int64_t stat_n, const float* hit, const int64_t* targets, int64_t T,
                            int64_t vocab, float* loss, float* lse, hipStream_t stream)
{
    const int64_t per = stat_n > 512 ? 1 : NT / 64;        // rows of a workgroup
    for (int64_t r = 0; r < T; r += kMostWorkgroups * per) {
        const int64_t rows = std::min(T - r, kMostWorkgroups * per);
        const dim3 grid((unsigned)((rows + per - 1) / per));
        if (per == 1)
            xent_join_kernel<4><<<grid, dim3(NT), 0, stream>>>(stat + r * stat_n * 2, stat_n, hit + r, targets + r, rows,
                                                               vocab, loss + r, lse + r);
        else
            xent_join_kernel<1><<<grid, dim3(NT), 0, stream>>>(stat + r * stat_n * 2, stat_n, hit + r, targets + r, rows,
                                                               vocab, loss + r, lse + r);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess)
            return e;
    }
    return hipSuccess;
}

}  // namespace lm
}  // namespace ag
