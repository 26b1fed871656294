// lm_rows.hip -- X (M, K) times Y (N, K) for few rows of X: a decoding step's linear layers, experts and
// logits.  The time is that of reading Y once (4.8 TB/s at 32000 x 4096, as a bare reading kernel), so
// nothing but Y's bytes in flight counts:
//   * A workgroup owns its columns (rows of Y) and the whole reduction: nothing is split over workgroups, and
//     no second launch joins anything.
//   * Y comes by buffer_load ... lds in whole 128-byte lines, several steps ahead, and is read by one wave
//     only.  (Straight into the operands' registers the lines come in halves: 63 us instead of 56 for the
//     32000 columns, 10 instead of 8 for 4096.)
//   * Many columns: 64 a workgroup, X staged once for its four waves, two workgroups a CU (rows_wide_kernel).
//     Few columns: 16 a workgroup, whose eight waves take the steps of the reduction in turn, each with a ring
//     of stages and an accumulator of its own and X out of L2 in registers: no barrier until the accumulators
//     are added up in LDS (rows_kernel).
// Rows, columns and k beyond the end are held out of the buffers' range and read as zeros.
#include "lm_launch.hpp"

namespace ag {
namespace lm {
namespace {

// Group of tile row tr, for tile rows of bm rows within their groups: its number, its first row (of the
// tile) and the tile's valid rows; false past the last.  The same rules as group_scan: ends are held to
// [0, limit] and to what their predecessors leave, and group E has the rows that belong to none.  Every wave
// finds it by itself, 64 groups at a time.
__device__ bool find_rows(const int32_t* ends, int E, int64_t limit, int bm, int64_t tr, int& g, int64_t& row0, int& rows)
{
    const int lane = threadIdx.x & 63, lim = (int)limit;
    int end0 = 0;              // end of the last group before these 64
    int64_t tile0 = 0;         // tile rows before them
    for (int base = 0; base <= E; base += 64) {
        const int e = base + lane;
        int end = max(end0, e < E ? min(ends[e], lim) : lim);
#pragma unroll
        for (int s = 1; s < 64; s <<= 1) {
            const int o = __shfl_up(end, s);
            if (lane >= s)
                end = max(end, o);
        }
        int prev = __shfl_up(end, 1);
        if (lane == 0)
            prev = end0;
        const int tiles = e <= E ? (end - prev + bm - 1) / bm : 0;
        int upto = tiles;
#pragma unroll
        for (int s = 1; s < 64; s <<= 1) {
            const int o = __shfl_up(upto, s);
            if (lane >= s)
                upto += o;
        }
        const uint64_t past = __ballot(tile0 + upto > tr);
        if (past) {
            const int l = __builtin_ctzll(past);
            const int64_t first = tile0 + __builtin_amdgcn_readlane(upto, l) - __builtin_amdgcn_readlane(tiles, l);
            const int64_t at = __builtin_amdgcn_readlane(prev, l) + (tr - first) * bm;
            g = base + l;
            row0 = at;
            rows = (int)min((int64_t)bm, __builtin_amdgcn_readlane(end, l) - at);
            return true;
        }
        end0 = __builtin_amdgcn_readlane(end, 63);
        tile0 += __builtin_amdgcn_readlane(upto, 63);
    }
    return false;
}

// Eight columns of a row, summed: what follows the product.
template <int EPI, int LPR>
__device__ __forceinline__ void finish8(const TileArgs& a, int64_t mrow, bool valid, int64_t col, int64_t slot, int lane,
                                        float* x, float unit)
{
    const int n = (int)max((int64_t)0, min((int64_t)8, a.N - col));
    if constexpr (EPI == kEpiStat) {
        stat8<LPR>(a, mrow, a.M, col, n, slot, lane, x);
    } else if constexpr (EPI == kEpiGrad) {
        grad8(a, mrow, a.M, col, n, x, unit);
    } else if (valid && n > 0) {
        linear8(a.out, mrow, col, n, x);
    }
}

// FM x 16 rows, 16 columns; D steps of 64 k are loaded ahead.
constexpr int W = 8;                 // waves
template <int FM, int D, int EPI>
__global__ __launch_bounds__(W * 64, 1) void rows_kernel(TileArgs a)
{
    constexpr int BM = FM * 16, BN = 16, SLOT = BN * 128;    // bytes of a wave's stage
    constexpr int OPS = 2 + FM * 2;                          // loads of a step
    static_assert(FM <= 4 && D >= 4 && D <= 8 && OPS * (D - 1) < 64, "sums fit stages 0 to 3; vmcnt");
    // one array per stage: the compiler then sees that the loads in flight fill other stages than the one read
    __shared__ __attribute__((aligned(1024))) char s0[W * SLOT], s1[W * SLOT], s2[W * SLOT], s3[W * SLOT];
    __shared__ __attribute__((aligned(1024))) char s4[D > 4 ? W * SLOT : 16], s5[D > 5 ? W * SLOT : 16];
    __shared__ __attribute__((aligned(1024))) char s6[D > 6 ? W * SLOT : 16], s7[D > 7 ? W * SLOT : 16];
    auto stage = [&](int d) {
        return d == 0 ? s0 : d == 1 ? s1 : d == 2 ? s2 : d == 3 ? s3 : d == 4 ? s4 : d == 5 ? s5 : d == 6 ? s6 : s7;
    };
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);

    int64_t row0 = (int64_t)blockIdx.y * BM, K = a.K;
    int rows = (int)min((int64_t)BM, a.M - row0), g = 0;
    if (EPI == kEpiLinear && a.group == kGroupRows) {
        if (!find_rows(a.ends, a.E, a.M, BM, blockIdx.y, g, row0, rows))
            return;
        if (g == a.E)              // rows past the last group: zeros
            g = 0, K = 0;
    }
    const int64_t n0 = (int64_t)blockIdx.x * BN;
    const int cols = (int)min((int64_t)BN, a.N - n0);
    const int32_t lda2 = (int32_t)(a.lda * 2), ldb2 = (int32_t)(a.ldb * 2), K2 = (int32_t)(K * 2);
    const __amdgpu_buffer_rsrc_t ra = make_rsrc(a.A + row0 * a.lda, (uint32_t)((rows - 1) * lda2 + K2));
    const __amdgpu_buffer_rsrc_t rb = make_rsrc(a.B + g * a.strideB + n0 * a.ldb, (uint32_t)((cols - 1) * ldb2 + K2));
    const int32_t r16 = lane & 15, k16 = (lane >> 4) * 16;
    const int32_t va = r16 * lda2 + k16;
    // eight rows of 128 bytes a load, 16-byte chunks swizzled by the row
    const int32_t r8 = lane >> 3;
    const int steps = (int)((K + 63) / 64);
    const uint32_t frag = r16 * 128 + wave * SLOT, sw = swz(r16);

    const float sample = EPI == kEpiGrad ? loss_sample(a.dloss, a.dloss_rows) : 1.0f;
    i32x4 xa[D][FM][2];
    f32x4 acc[FM];
#pragma unroll
    for (int i = 0; i < FM; ++i)
        acc[i] = f32x4{};
    auto load = [&](int d, int step) {
        const int32_t at = step * 128;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const int32_t c16 = ((lane & 7) ^ (int32_t)swz(q * 8 + r8)) * 16;
            const int32_t off = at + c16 < K2 ? (q * 8 + r8) * ldb2 + at + c16 : (int32_t)0x80000000;
            dma16(rb, stage(d) + wave * SLOT + q * 1024, off);
        }
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const int32_t off = at + s * 64 + k16 < K2 ? va + at + s * 64 : (int32_t)0x80000000;
#pragma unroll
            for (int i = 0; i < FM; ++i)
                xa[d][i][s] =
                    __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(ra, off + i * 16 * lda2, 0, 0));
        }
    };
    auto compute = [&](int d) {
        const char* st = stage(d) + frag;
        bf16x8 y[2];
#pragma unroll
        for (int s = 0; s < 2; ++s)
            y[s] = *reinterpret_cast<const bf16x8*>(st + (((s * 4 + (lane >> 4)) ^ sw) * 16));
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int i = 0; i < FM; ++i)
                acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(y[s], __builtin_bit_cast(bf16x8, xa[d][i][s]), acc[i],
                                                                 0, 0, 0);
    };
#pragma unroll
    for (int d = 0; d < D; ++d) {
        load(d, wave + d * W);
        __builtin_amdgcn_sched_barrier(0);
    }
    for (int st = wave; st < steps; st += W * D) {
#pragma unroll
        for (int d = 0; d < D; ++d) {
            wait_vmcnt<OPS * (D - 1)>();
            asm volatile("" ::: "memory");
            __builtin_amdgcn_sched_barrier(0);
            compute(d);
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");     // read before the stage is filled again
            __builtin_amdgcn_sched_barrier(0);
            load(d, st + (D + d) * W);
            __builtin_amdgcn_sched_barrier(0);
        }
    }
    wait_vmcnt0();                   // loads past the last step have landed too
    asm volatile("" ::: "memory");

    const float counted = EPI == kEpiGrad ? loss_unit(sample) : 1.0f;
    // lane l has row l % 16 and four columns from 4 (l / 16) of each 16 x 16 block; block row i of a wave goes
    // to its part of stage i, 16-byte units swizzled by the row
    constexpr uint32_t UM = BN / 4 - 1;
    auto unit = [&](int w, int i, int r, int u) {
        return reinterpret_cast<f32x4*>(stage(i) + w * SLOT + r * (BN * 4) + ((u ^ (r & UM)) * 16));
    };
#pragma unroll
    for (int i = 0; i < FM; ++i)
        *unit(wave, i, r16, lane >> 4) = acc[i];
    barrier_after_lds_write();
    constexpr int LPR = BN / 8, UNITS = 16 * LPR;            // eight columns of a row each, 16 rows at a time
#pragma unroll
    for (int i = 0; i < FM; ++i) {
        if (wave != i || lane >= UNITS)
            continue;
        const int r = lane / LPR, c = (lane % LPR) * 2;
        f32x4 x0 = *unit(0, i, r, c), x1 = *unit(0, i, r, c + 1);
#pragma unroll
        for (int w = 1; w < W; ++w) {
            x0 += *unit(w, i, r, c);
            x1 += *unit(w, i, r, c + 1);
        }
        float x[8] = {x0[0], x0[1], x0[2], x0[3], x1[0], x1[1], x1[2], x1[3]};
        finish8<EPI, LPR>(a, row0 + i * 16 + r, i * 16 + r < rows, n0 + c * 4, blockIdx.x, lane, x, counted);
    }
}

// FM x 16 rows, 64 columns, the reduction in steps of 64 k through a ring of D stages that the four waves
// share: each has 16 columns, and X is staged once for all.
template <int FM, int EPI>
__global__ __launch_bounds__(NT, 2) void rows_wide_kernel(TileArgs a)
{
    constexpr int BM = FM * 16, SR = FM <= 2 ? 32 : 64, D = FM <= 2 ? 6 : 5;   // 72 or 80 KiB: two workgroups a CU
    constexpr int XB = SR * 128, STAGE = XB + 64 * 128, XO = SR / 32, OPS = XO + 2;
    __shared__ __attribute__((aligned(1024))) char s0[STAGE], s1[STAGE], s2[STAGE], s3[STAGE], s4[STAGE];
    __shared__ __attribute__((aligned(1024))) char s5[D > 5 ? STAGE : 16];
    auto stage = [&](int d) { return d == 0 ? s0 : d == 1 ? s1 : d == 2 ? s2 : d == 3 ? s3 : d == 4 ? s4 : s5; };
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);

    int64_t row0 = (int64_t)blockIdx.y * BM, K = a.K;
    int rows = (int)min((int64_t)BM, a.M - row0), g = 0;
    if (EPI == kEpiLinear && a.group == kGroupRows) {
        if (!find_rows(a.ends, a.E, a.M, BM, blockIdx.y, g, row0, rows))
            return;
        if (g == a.E)              // rows past the last group: zeros
            g = 0, K = 0;
    }
    const int64_t n0 = (int64_t)blockIdx.x * 64;
    const int cols = (int)min((int64_t)64, a.N - n0);
    const int32_t lda2 = (int32_t)(a.lda * 2), ldb2 = (int32_t)(a.ldb * 2), K2 = (int32_t)(K * 2);
    const __amdgpu_buffer_rsrc_t ra = make_rsrc(a.A + row0 * a.lda, (uint32_t)((rows - 1) * lda2 + K2));
    const __amdgpu_buffer_rsrc_t rb = make_rsrc(a.B + g * a.strideB + n0 * a.ldb, (uint32_t)((cols - 1) * ldb2 + K2));
    const int32_t r8 = wave * 8 + (lane >> 3), c16 = ((lane & 7) ^ (int32_t)swz(r8)) * 16;   // 32 rows a load of the four
    const int32_t va = r8 * lda2 + c16, vb = r8 * ldb2 + c16;
    const int steps = (int)((K + 63) / 64);
    const int32_t r16 = lane & 15;
    const uint32_t sw = swz(r16);

    const float sample = EPI == kEpiGrad ? loss_sample(a.dloss, a.dloss_rows) : 1.0f;
    f32x4 acc[FM];
#pragma unroll
    for (int i = 0; i < FM; ++i)
        acc[i] = f32x4{};
    auto load = [&](int d, int step) {
        const int32_t at = step * 128;
        const bool in = at + c16 < K2;
        const int32_t pa = in ? va + at : (int32_t)0x80000000, pb = in ? vb + at : (int32_t)0x80000000;
#pragma unroll
        for (int q = 0; q < 2; ++q)
            dma16(rb, stage(d) + XB + q * 4096 + wave * 1024, pb + q * 32 * ldb2);
#pragma unroll
        for (int q = 0; q < XO; ++q)
            dma16(ra, stage(d) + q * 4096 + wave * 1024, pa + q * 32 * lda2);
    };
#pragma unroll
    for (int d = 0; d < D - 1; ++d)
        load(d, d);
    for (int st = 0; st < steps; st += D) {
#pragma unroll
        for (int d = 0; d < D; ++d) {
            if (st + d >= steps)
                break;
            wait_vmcnt<OPS * (D - 2)>();
            stage_barrier();
            load((d + D - 1) % D, st + d + D - 1);
            __builtin_amdgcn_sched_barrier(0);
            const char* sx = stage(d) + r16 * 128;
            const char* sy = stage(d) + XB + wave * 2048 + r16 * 128;
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const uint32_t c = ((s * 4 + (lane >> 4)) ^ sw) * 16;
                const bf16x8 y = *reinterpret_cast<const bf16x8*>(sy + c);
#pragma unroll
                for (int i = 0; i < FM; ++i)
                    acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                        y, *reinterpret_cast<const bf16x8*>(sx + i * 2048 + c), acc[i], 0, 0, 0);
            }
        }
    }
    wait_vmcnt0();                   // loads past the last step have landed too
    barrier_after_lds_write();

    const float counted = EPI == kEpiGrad ? loss_unit(sample) : 1.0f;
    // 16 rows a stage, 16-byte units swizzled by the row
    auto unit = [&](int i, int r, int u) { return reinterpret_cast<f32x4*>(stage(i) + r * 256 + ((u ^ r) * 16)); };
#pragma unroll
    for (int i = 0; i < FM; ++i)
        *unit(i, r16, wave * 4 + (lane >> 4)) = acc[i];
    barrier_after_lds_write();
#pragma unroll
    for (int i = 0; i < FM; ++i) {
        if ((wave >> 1) != (i & 1))  // 128 threads for 16 rows
            continue;
        const int u = tid & 127, r = u >> 3, c = (u & 7) * 2;
        const f32x4 x0 = *unit(i, r, c), x1 = *unit(i, r, c + 1);
        float x[8] = {x0[0], x0[1], x0[2], x0[3], x1[0], x1[1], x1[2], x1[3]};
        finish8<EPI, 8>(a, row0 + i * 16 + r, i * 16 + r < rows, n0 + c * 4, blockIdx.x, lane, x, counted);
    }
}

// 64 columns a workgroup once there are enough of them to keep the memory busy, by the columns and rows of X
// (that narrow workgroups each read again).  Both sides, us, K = 4096, 16 | 64 columns: N = 4096: 1 row
// 12 | 20, 64 rows 25 | 27; N = 14336: 1 row 33 | 28, 48 rows 67 | 30; N = 32000: 1 row 63 | 56, 64 rows 171 | 57.
// More rows than a tile's are always for them.
bool rows_wide(int64_t N, int64_t rows, int groups)
{
    return rows > kRowsMost || (N + 63) / 64 * groups >= (rows <= 16 ? 128 : 72);
}

template <int FM, int EPI>
hipError_t launch(bool wide, const TileArgs& a, hipStream_t stream)
{
    constexpr int BM = FM * 16, D = FM > 2 ? 4 : FM == 2 ? 6 : 8;
    int cus = 0;
    hipError_t e = device_cus(&cus);
    if (e != hipSuccess)
        return e;
    const int bn = wide ? 64 : 16;
    const int64_t tiles_n = (a.N + bn - 1) / bn;
    int64_t tiles_m = (a.M + BM - 1) / BM;
    if (a.group == kGroupRows)
        tiles_m += a.E + 1;
    tiles_m = tiles_m < a.M ? tiles_m : a.M;     // a tile row has a row at least
    if (tiles_n <= 0 || tiles_m <= 0)
        return hipSuccess;
    const dim3 grid((unsigned)tiles_n, (unsigned)tiles_m);
    if (wide)
        rows_wide_kernel<FM, EPI><<<grid, dim3(NT), 0, stream>>>(a);
    else if (tiles_n * tiles_m <= cus)
        rows_kernel<FM, D, EPI><<<grid, dim3(W * 64), 0, stream>>>(a);
    else        // a ring of half a CU's LDS: the workgroups past the first round start with it, not after it
        rows_kernel<FM, 4, EPI><<<grid, dim3(W * 64), 0, stream>>>(a);
    return hipGetLastError();
}

template <int EPI>
hipError_t launch_fm(int64_t rows, const TileArgs& a, hipStream_t stream)
{
    const bool wide = rows_wide(a.N, rows, a.group == kGroupRows ? a.E : 1);
    switch (rows <= 16 ? 1 : rows <= 32 ? 2 : rows <= 48 ? 3 : 4) {
    case 1: return launch<1, EPI>(wide, a, stream);
    case 2: return launch<2, EPI>(wide, a, stream);
    case 3: return launch<3, EPI>(wide, a, stream);
    default: return launch<4, EPI>(wide, a, stream);
    }
}

}  // namespace

int rows_cols(int64_t N, int64_t rows) { return rows_wide(N, rows, 1) ? 64 : 16; }

hipError_t launch_rows(Epi epi, int64_t rows, TileArgs a, hipStream_t stream)
{
    switch (epi) {
    case kEpiStat:
        a.stat_n = (a.N + rows_cols(a.N, rows) - 1) / rows_cols(a.N, rows);
        return launch_fm<kEpiStat>(rows, a, stream);
    case kEpiGrad: return launch_fm<kEpiGrad>(rows, a, stream);
    default: return launch_fm<kEpiLinear>(rows, a, stream);
    }
}

}  // namespace lm
}  // namespace ag
