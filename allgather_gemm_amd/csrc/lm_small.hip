// lm_small.hip -- what runs before and after the tiled products of the language-model operators:
// joining a split reduction, the activation's slope with the bias gradient, the softmax statistics.
// All are bound by the bytes they move.
#include "ag_internal.hpp"
#include "lm_tile.hpp"

#include <algorithm>

namespace ag {
namespace lm {
namespace {

// Eight columns of one row per thread: the fp32 sums of the splits, added in the order of the splits.
__global__ __launch_bounds__(NT) void join_kernel(const float* part, int splits, int64_t M, int64_t N, int64_t ldp,
                                                  LinearOut out, bool vec)
{
    const int64_t units = ldp / 8;
    const int64_t u = blockIdx.x * (int64_t)NT + threadIdx.x;
    if (u >= M * units)
        return;
    const int64_t row = u / units, col = (u - row * units) * 8;
    const float* p = part + row * ldp + col;
    f32x4 s0 = reinterpret_cast<const f32x4*>(p)[0], s1 = reinterpret_cast<const f32x4*>(p)[1];
    for (int s = 1; s < splits; ++s) {
        const f32x4* q = reinterpret_cast<const f32x4*>(p + s * M * ldp);
        s0 += q[0];
        s1 += q[1];
    }
    float x[8] = {s0[0], s0[1], s0[2], s0[3], s1[0], s1[1], s1[2], s1[3]};
    const int n = (int)min((int64_t)8, N - col);
    if (n <= 0)
        return;
    float b[8] = {}, r[8] = {};
    if (out.bias)
        load8(out.bias + col, n, vec, b);
    if (out.residual)
        load8(out.residual + row * out.ldc + col, n, vec, r);
    linear8(out, row, col, n, vec, x, b, r);
}

constexpr int COLS = 256;      // columns of a workgroup of act_bwd_kernel: 32 lanes of 8

// d = dC act'(pre), rounded to bf16 for the two products; its column sums from the unrounded values.
__global__ __launch_bounds__(NT) void act_bwd_kernel(const __bf16* dC, const __bf16* pre, int act, int64_t M, int64_t N,
                                                     int64_t chunk, __bf16* d, int64_t ldd, float* colsum, bool vec)
{
    __shared__ float s_sum[8][COLS + 8];
    const int cl = threadIdx.x & 31, rl = threadIdx.x >> 5;
    const int64_t col = blockIdx.x * (int64_t)COLS + cl * 8;
    const int64_t r0 = blockIdx.y * chunk, r1 = min(M, r0 + chunk);
    const int n = (int)max((int64_t)0, min((int64_t)8, N - col));
    float sum[8] = {};
    for (int64_t row = r0 + rl; row < r1; row += 8) {
        float x[8];
        load8(dC + row * N + col, n, vec, x);
        if (act != kActNone) {
            float z[8];
            load8(pre + row * N + col, n, vec, z);
            act_slope8(x, z, act);
        }
        if (d && col < ldd) {
            bf16x8 o;
#pragma unroll
            for (int e = 0; e < 8; ++e)
                o[e] = (__bf16)x[e];
            *reinterpret_cast<bf16x8*>(d + row * ldd + col) = o;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e)
            sum[e] += x[e];
    }
    if (!colsum)
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
        colsum[blockIdx.y * N + c] = s;
    }
}

__global__ __launch_bounds__(NT) void colsum_join_kernel(const float* colsum, int64_t rows, int64_t N, __bf16* out)
{
    const int64_t c = blockIdx.x * (int64_t)NT + threadIdx.x;
    if (c >= N)
        return;
    float s = 0.0f;
    for (int64_t r = 0; r < rows; ++r)
        s += colsum[r * N + c];
    out[c] = (__bf16)s;
}

// One wave per row: the pieces' (maximum, sum) pairs under one maximum.
__global__ __launch_bounds__(NT) void xent_join_kernel(const float* stat, int64_t stat_n, const float* hit,
                                                       const int64_t* targets, int64_t T, int64_t vocab, float* loss,
                                                       float* lse)
{
    const int64_t row = blockIdx.x * (int64_t)(NT / 64) + (threadIdx.x >> 6);
    const int lane = threadIdx.x & 63;
    if (row >= T)
        return;
    const float2* p = reinterpret_cast<const float2*>(stat) + row * stat_n;
    float mx = -INFINITY;
    for (int64_t i = lane; i < stat_n; i += 64)
        mx = fmaxf(mx, p[i].x);
#pragma unroll
    for (int s = 1; s < 64; s <<= 1)
        mx = fmaxf(mx, __shfl_xor(mx, s));
    const float base = mx == -INFINITY ? 0.0f : mx;
    float sum = 0.0f;
    for (int64_t i = lane; i < stat_n; i += 64) {
        const float2 v = p[i];
        sum += v.y * (v.x == -INFINITY ? (v.y != v.y ? v.y : 0.0f) : fast_exp(v.x - base));
    }
#pragma unroll
    for (int s = 1; s < 64; s <<= 1)
        sum += __shfl_xor(sum, s);
    if (lane == 0) {
        const float l = base + logf(sum);
        const int64_t y = targets[row];
        lse[row] = l;
        loss[row] = (y >= 0 && y < vocab) ? l - hit[row] : 0.0f;
    }
}

}  // namespace

hipError_t launch_join(const float* part, int splits, int64_t M, int64_t N, int64_t ldp, const LinearOut& out, bool vec,
                       hipStream_t stream)
{
    const int64_t units = M * (ldp / 8);
    if (units <= 0)
        return hipSuccess;
    join_kernel<<<dim3((unsigned)((units + NT - 1) / NT)), dim3(NT), 0, stream>>>(part, splits, M, N, ldp, out, vec);
    return hipGetLastError();
}

// Rows of one workgroup: a multiple of its 8 row lanes, at most 128 workgroups down the rows.
static int64_t act_chunk(int64_t M) { return std::max<int64_t>(32, ((M + 127) / 128 + 7) / 8 * 8); }

int64_t colsum_rows(int64_t M) { return (M + act_chunk(M) - 1) / act_chunk(M); }

hipError_t launch_act_bwd(const __bf16* dC, const __bf16* pre, int act, int64_t M, int64_t N, __bf16* d, int64_t ldd,
                          float* colsum, hipStream_t stream)
{
    if (M <= 0 || N <= 0)
        return hipSuccess;
    const dim3 grid((unsigned)((N + COLS - 1) / COLS), (unsigned)colsum_rows(M));
    act_bwd_kernel<<<grid, dim3(NT), 0, stream>>>(dC, pre, act, M, N, act_chunk(M), d, ldd, colsum, N % 8 == 0);
    return hipGetLastError();
}

hipError_t launch_colsum_join(const float* colsum, int64_t rows, int64_t N, __bf16* out, hipStream_t stream)
{
    if (N <= 0)
        return hipSuccess;
    colsum_join_kernel<<<dim3((unsigned)((N + NT - 1) / NT)), dim3(NT), 0, stream>>>(colsum, rows, N, out);
    return hipGetLastError();
}

hipError_t launch_xent_join(const float* stat, int64_t stat_n, const float* hit, const int64_t* targets, int64_t T,
                            int64_t vocab, float* loss, float* lse, hipStream_t stream)
{
    if (T <= 0)
        return hipSuccess;
    const int per = NT / 64;
    xent_join_kernel<<<dim3((unsigned)((T + per - 1) / per)), dim3(NT), 0, stream>>>(stat, stat_n, hit, targets, T,
                                                                                     vocab, loss, lse);
    return hipGetLastError();
}

}  // namespace lm
}  // namespace ag
