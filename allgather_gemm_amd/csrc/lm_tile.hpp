// lm_tile.hpp -- the tiled matrix product behind the language-model operators (gemm_bias_act,
// gemm_grouped, gemm_xent and their gradients; newton_schulz), with what follows the product in its epilogue.
//
// One kernel template computes out = X * Y^T tile by tile with v_mfma_f32_32x32x16_bf16 and fp32
// sums, where each operand lies in memory in one of two ways:
//   * rows of the reduction ("row operand"): X (M, K), Y (N, K).  A K step of 64 is one 128-byte
//     LDS row per operand row, 16-byte chunks XOR-swizzled so the ds_read_b128 fragment loads are
//     free of bank conflicts.
//   * the reduction across rows ("column operand"): X (K, M), Y (K, N), which the gradients need:
//     dA = dC B reads B across its rows, dB = dC^T A reads both.  The K step's 64 rows land in LDS as
//     they are, and ds_read_b64_tr_b16 turns them: 16 lanes read four k rows of 16 columns and each
//     gets its column's four k values, so a fragment is two such reads and no operand is ever
//     transposed in memory.  Here 64-byte groups are swizzled by k, and the four k rows that a half
//     wave reads fall into distinct banks.
// Both arrive by buffer_load ... lds with the buffer's bounds set to the operand's last valid byte,
// so rows, columns and k beyond the end read zeros without a branch.
#pragma once

#include "ag_device.hpp"
#include "lm_internal.hpp"

#include <type_traits>

namespace ag {
namespace lm {

constexpr int NT = 256;        // threads per workgroup
constexpr int BK = 64;         // reduction elements per step
constexpr int GROUP_M = 8;     // tile rows per group of the grouped tile order

__device__ __forceinline__ uint32_t swz(uint32_t row) { return (row & 7u) ^ ((row >> 3) & 1u); }

typedef __attribute__((address_space(3))) bf16x4 lds_bf16x4;

// Workgroup barrier of the K loop: this wave's LDS reads are done, its loads into LDS are not waited for
// (__syncthreads() would wait for every one in flight; the loop waits for those it needs itself).
__device__ __forceinline__ void stage_barrier()
{
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
}

// One operand's stage in LDS.  One of 32 KiB is two arrays of 16 KiB, or one array and its middle; a smaller one
// is `lo`.
struct Part {
    char *lo, *hi;
};

// One operand's side of the tile: R rows of the output's extent, T: column operand.
template <int R, bool T>
struct Side {
    static constexpr int OPS = R / 32;             // 4 KiB loads per K step
    static constexpr int BYTES = R * BK * 2;
    static constexpr int RB = T ? R * 2 : 128;     // LDS bytes per stored row
    static constexpr int RPO = 4096 / RB;          // stored rows per load

    // 64-byte group swizzle of k row k (column operand)
    static __device__ __forceinline__ uint32_t ksw(uint32_t k)
    {
        return R >= 128 ? (k & 3u) : R == 64 ? ((k >> 1) & 1u) : 0u;
    }

    uint32_t voff;         // this thread's byte offset inside a load
    int32_t c16;           // row operand: bytes of this thread's chunk into the K step
    uint32_t op_stride;    // bytes between two loads' first rows
    const char* at;        // where the next step's buffer starts
    int64_t step;          // bytes from one step's buffer to the next
    int32_t left;          // row operand: bytes of the row from `at` on that are still to be read;
                           // column operand: rows still to be read
    int32_t bytes;         // row operand: bytes from `at` to the tile's last; column operand: those of a
                           // whole step
    int32_t col2;          // column operand: bytes of the tile's first column into its row
    int32_t row_bytes;

    __device__ __forceinline__ void init(int tid, int64_t ld)
    {
        row_bytes = (int32_t)(ld * 2);
        if (T) {
            const uint32_t k = (uint32_t)(tid * 16) / RB, p = ((uint32_t)(tid * 16) % RB) / 16;
            const uint32_t c = ((p >> 2) ^ ksw(k)) * 4 + (p & 3);
            voff = k * row_bytes + c * 16;
            c16 = 0;
            step = (int64_t)BK * row_bytes;
        } else {
            const uint32_t r = tid >> 3, c = (tid & 7) ^ swz(r);
            voff = r * row_bytes + c * 16;
            c16 = (int32_t)c * 16;
            step = BK * 2;
        }
        op_stride = RPO * row_bytes;
    }

    // A tile's K steps [kb0, ...) up to reduction index k_end: base = first element of the tile at k = 0
    // (row operand: its first row; column operand: row k = 0 at the tile's first column, col0), rows =
    // the valid tile rows (row operand), K = the reduction length.
    __device__ __forceinline__ void start(const __bf16* base, int64_t rows, int64_t K, int64_t col0, int64_t kb0,
                                          int64_t k_end)
    {
        at = reinterpret_cast<const char*>(base) + kb0 * step;
        const int32_t k_left = (int32_t)(max((int64_t)0, k_end - kb0 * BK));
        if (T) {
            left = k_left;
            col2 = (int32_t)(col0 * 2);
        } else {
            left = k_left * 2;
            bytes = (int32_t)(max((int64_t)0, ((rows - 1) * row_bytes + K * 2) - kb0 * BK * 2));
        }
    }

    // The buffer over what the next step may read, and this thread's offset in it (past the row's end it
    // lies beyond every buffer's size, which stays under 2^31).  Steps past the last read nothing.
    __device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc() const
    {
        if (T)
            return make_rsrc(at, (uint32_t)max(0, min(left, BK) * row_bytes - col2));
        return make_rsrc(at, (uint32_t)max(0, bytes));
    }
    __device__ __forceinline__ uint32_t offset() const { return T || c16 < left ? voff : 0x80000000u; }
    __device__ __forceinline__ void advance()
    {
        at += step;
        left -= T ? BK : BK * 2;
        if (!T)
            bytes -= BK * 2;
    }

    __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t r, const Part& s, uint32_t wave_off, uint32_t off,
                                         uint32_t stride, int q) const
    {
        dma16(r, (OPS == 8 && q >= 4 ? s.hi + (q - 4) * 4096 : s.lo + q * 4096) + wave_off, off + q * stride);
    }
};

// Fragment addressing of one wave: F fragments of 32 rows, those of the waves in turn (INTER: fragment i of wave w
// is the tile's i * R / 32 / F + w, so which half of a 32 KiB stage it is in does not depend on the wave) or
// one wave's next to each other (w * F + i; a row operand's 32 KiB are then one array).
template <int R, bool T, int F, bool INTER>
struct Frag {
    static constexpr int WAVES = R / 32 / F;
    static constexpr bool TWO = R == 256;
    static_assert(!TWO || F == 4, "a stage's half has two of a wave's fragments, or all");
    uint32_t off[4 > F ? 4 : F];

    __device__ __forceinline__ void init(int lane, int w)
    {
        const uint32_t fr = lane & 31, fh = lane >> 5;
        if (T) {
            const uint32_t k = fh * 8 + ((lane & 15) >> 2);
            const uint32_t within = ((lane >> 4) & 1) * 32 + (lane & 3) * 8;
#pragma unroll
            for (int i = 0; i < F; ++i)
                off[i] = k * Side<R, T>::RB +
                         (((uint32_t)(INTER ? i * WAVES + w : w * F + i)) ^ Side<R, T>::ksw(k)) * 64 + within;
        } else {
            const uint32_t fsw = swz(fr & 15);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
                off[kk] = (uint32_t)((INTER ? w : w * F) * 32 + fr) * 128 + (((uint32_t)(2 * kk) + fh) ^ fsw) * 16;
        }
    }

    // Fragment i of substep kk: lane l holds row l % 32, k = 16 kk + 8 (l / 32) .. + 7.
    __device__ __forceinline__ bf16x8 read(const Part& s, int kk, int i) const
    {
        if (T) {
            const char* p = (TWO && kk >= 2 ? s.hi : s.lo) + off[i] + (TWO ? kk & 1 : kk) * 16 * Side<R, T>::RB;
            const bf16x4 lo = __builtin_bit_cast(
                bf16x4, __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_bf16x4*)const_cast<char*>(p)));
            const bf16x4 hi = __builtin_bit_cast(
                bf16x4,
                __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_bf16x4*)const_cast<char*>(p + 4 * Side<R, T>::RB)));
            return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
        }
        if (INTER)
            return *reinterpret_cast<const bf16x8*>((TWO && i >= 2 ? s.hi : s.lo) + off[kk] +
                                                    (TWO ? i & 1 : i) * WAVES * 4096);
        return *reinterpret_cast<const bf16x8*>(s.lo + off[kk] + i * 4096);      // one array
    }
};

// f(0), ..., f(N - 1) with compile-time arguments
template <int N, int I = 0, typename F>
__device__ __forceinline__ void each(F f)
{
    if constexpr (I < N) {
        f(std::integral_constant<int, I>());
        each<N, I + 1>(f);
    }
}

// ------------------------------------------------------------------------------- activations
// Values and slopes in fp32.  exp goes through exp2 (one hardware instruction); its relative error,
// a few 2^-24 times the argument's size, is far below the bf16 rounding of the result.
__device__ __forceinline__ float fast_exp(float x) { return __builtin_amdgcn_exp2f(x * 1.4426950408889634f); }
__device__ __forceinline__ float fast_sigmoid(float x) { return __builtin_amdgcn_rcpf(1.0f + fast_exp(-x)); }

// Phi(x), the normal distribution function, and phi'(x) sqrt(2 pi) = exp(-x^2 / 2), which it takes: erfc by
// Abramowitz & Stegun 7.1.26, off by at most 1.5e-7, as near as 0.5 (1 + erf) gets in fp32.
__device__ __forceinline__ float normal_cdf(float x, float* e)
{
    const float t = __builtin_amdgcn_rcpf(fmaf(0.3275911f * 0.70710678118654752f, fabsf(x), 1.0f));
    *e = fast_exp(-0.5f * x * x);
    float p = fmaf(t, 1.061405429f, -1.453152027f);
    p = fmaf(t, p, 1.421413741f);
    p = fmaf(t, p, -0.284496736f);
    p = fmaf(t, p, 0.254829592f);
    const float q = 0.5f * t * p * *e;                 // Phi(-|x|)
    return x >= 0.0f ? 1.0f - q : q;
}

constexpr float kTanh0 = 1.5957691216057308f;          // 2 sqrt(2 / pi): 0.5 (1 + tanh u) = sigmoid(2u)

// The activation is chosen once for eight values, not for each.
__device__ __forceinline__ void act_value8(float* x, int act)
{
    switch (act) {
    case kActRelu:
#pragma unroll
        for (int e = 0; e < 8; ++e)
            x[e] = x[e] > 0.0f || x[e] != x[e] ? x[e] : 0.0f;
        break;
    case kActSilu:
#pragma unroll
        for (int e = 0; e < 8; ++e)
            x[e] *= fast_sigmoid(x[e]);
        break;
    case kActGelu:
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            float ignored;
            x[e] *= normal_cdf(x[e], &ignored);
        }
        break;
    case kActGeluTanh:
#pragma unroll
        for (int e = 0; e < 8; ++e)
            x[e] *= fast_sigmoid(kTanh0 * (x[e] + 0.044715f * x[e] * x[e] * x[e]));
        break;
    default: break;
    }
}

__device__ __forceinline__ float silu_slope(float x)
{
    const float s = fast_sigmoid(x);
    return s * (1.0f + x * (1.0f - s));
}

__device__ __forceinline__ float gelu_slope(float x)
{
    float e;
    const float c = normal_cdf(x, &e);
    return fmaf(0.3989422804014327f * x, e, c);
}

__device__ __forceinline__ float gelu_tanh_slope(float x)
{
    if (fabsf(x) > 30.0f)              // s is 0 or 1 there; x^2 could overflow and meet its zero
        return x > 0.0f ? 1.0f : 0.0f;
    const float s = fast_sigmoid(kTanh0 * (x + 0.044715f * x * x * x));
    return s + x * s * (1.0f - s) * kTanh0 * (1.0f + 0.134145f * x * x);
}

// x[e] *= act'(z[e])
__device__ __forceinline__ void act_slope8(float* x, const float* z, int act)
{
    switch (act) {
    case kActRelu:
#pragma unroll
        for (int e = 0; e < 8; ++e)
            x[e] = z[e] > 0.0f ? x[e] : 0.0f;
        break;
    case kActSilu:
#pragma unroll
        for (int e = 0; e < 8; ++e)
            x[e] *= silu_slope(z[e]);
        break;
    case kActGelu:
#pragma unroll
        for (int e = 0; e < 8; ++e)
            x[e] *= gelu_slope(z[e]);
        break;
    case kActGeluTanh:
#pragma unroll
        for (int e = 0; e < 8; ++e)
            x[e] *= gelu_tanh_slope(z[e]);
        break;
    default: break;
    }
}

// Sixteen bytes at any element: rows of an odd length start anywhere, and the memory takes them so.
typedef bf16x8 bf16x8_any __attribute__((aligned(2)));
typedef i32x4 i32x4_any __attribute__((aligned(2)));

// Eight consecutive bf16, `n` of them valid.  Less than eight come one by one, all at a time: the loads are not
// left out past the last but repeat it.
__device__ __forceinline__ bf16x8 load8_few(const __bf16* p, int n)
{
    bf16x8 v = {};
    if (n > 0) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            v[e] = p[min(e, n - 1)];
    }
    return v;
}

__device__ __forceinline__ void load8(const __bf16* p, int n, float* x)
{
    const bf16x8 v = n >= 8 ? *reinterpret_cast<const bf16x8_any*>(p) : load8_few(p, n);
#pragma unroll
    for (int e = 0; e < 8; ++e)
        x[e] = e < n ? (float)v[e] : 0.0f;
}

__device__ __forceinline__ void store8(__bf16* p, const float* x)
{
    bf16x8 o;
#pragma unroll
    for (int e = 0; e < 8; ++e)
        o[e] = (__bf16)x[e];
    __builtin_nontemporal_store(o, reinterpret_cast<bf16x8_any*>(p));
}

__device__ __forceinline__ void store8(__bf16* p, int n, const float* x)
{
    if (n >= 8)
        return store8(p, x);
#pragma unroll
    for (int e = 0; e < 7; ++e)
        if (e < n)
            p[e] = (__bf16)x[e];
}

// act(x + bias) + residual of eight columns into C; `pre` gets x + bias.  b and r: the eight columns of bias and
// residual (zeros without), at: the place of the first in pre.
__device__ __forceinline__ void finish_linear8(const LinearOut& o, __bf16* C, int64_t at, int n, float* x, const float* b,
                                               const float* r)
{
#pragma unroll
    for (int e = 0; e < 8; ++e)
        x[e] += b[e];
    if (o.pre)
        store8(o.pre + at, n, x);
    act_value8(x, o.act);
#pragma unroll
    for (int e = 0; e < 8; ++e)
        x[e] += r[e];
    store8(C, n, x);
}

__device__ __forceinline__ void linear8(const LinearOut& o, int64_t row, int64_t col, int n, float* x)
{
    const int64_t at = row * o.ldc + col;
    float b[8] = {}, r[8] = {};
    if (o.bias)
        load8(o.bias + col, n, b);
    if (o.residual)
        load8(o.residual + at, n, r);
    finish_linear8(o, o.C + at, at, n, x, b, r);
}

// ------------------------------------------------------------------------------------- groups
// The groups as the kernel uses them.  end[e] is the running maximum of ends[0..e] within [0, limit], so
// groups from any table stay inside the tensors, and end[E] = limit closes a last group of rows that belong to
// none.  Rows of group e are cut into tile rows of BM and, where at most BM / 2 remain, one of BM / 2: big[e]
// and half[e] are the first of each kind, big[E + 1] and half[E + 1] their numbers.
struct Groups {
    int32_t end[kMaxGroups + 1], big[kMaxGroups + 2], half[kMaxGroups + 2];
};
// Groups of the reduction have no tile rows of their own, but an order: by their size, largest first.
struct KGroups {
    int32_t end[kMaxGroups + 1], order[kMaxGroups];
};

// Tile rows of n rows: of BM rows, and (HALF) of BM / 2.
template <int BM, bool HALF>
__host__ __device__ __forceinline__ int big_rows(int n)
{
    return HALF ? n / BM + (n % BM > BM / 2) : (n + BM - 1) / BM;
}
template <int BM, bool HALF>
__host__ __device__ __forceinline__ int half_rows(int n)
{
    return HALF && n % BM > 0 && n % BM <= BM / 2;
}

// Wave 0 scans, 64 lanes over E + 1 entries; ends with a barrier.
template <int BM, bool HALF, typename G>
__device__ void group_scan(const int32_t* ends, int E, int64_t limit, G& s)
{
    if (__builtin_amdgcn_readfirstlane(threadIdx.x >> 6) == 0) {
        const int lane = threadIdx.x & 63;
        const int per = (E + 1 + 63) / 64, e0 = min(lane * per, E + 1), e1 = min(e0 + per, E + 1);
        const int lim = (int)limit;
        int top = 0;
        for (int e = e0; e < e1; ++e)
            top = max(top, e < E ? min(ends[e], lim) : lim);
        int before = top;                                    // inclusive, then exclusive running maximum
        for (int s = 1; s < 64; s <<= 1) {
            const int o = __shfl_up(before, s);
            if (lane >= s)
                before = max(before, o);
        }
        before = __shfl_up(before, 1);
        if (lane == 0)
            before = 0;
        int prev = before, big = 0, half = 0;
        for (int e = e0; e < e1; ++e) {
            const int end = max(prev, e < E ? min(ends[e], lim) : lim);
            s.end[e] = end;
            big += big_rows<BM, HALF>(end - prev);
            half += half_rows<BM, HALF>(end - prev);
            prev = end;
        }
        if constexpr (std::is_same<G, Groups>::value) {
            int big0 = big, half0 = half;
            for (int s = 1; s < 64; s <<= 1) {
                const int o = __shfl_up(big0, s), q = __shfl_up(half0, s);
                if (lane >= s) {
                    big0 += o;
                    half0 += q;
                }
            }
            big0 -= big;
            half0 -= half;
            prev = before;
            for (int e = e0; e < e1; ++e) {
                s.big[e] = big0;
                s.half[e] = half0;
                const int n = s.end[e] - prev;
                big0 += big_rows<BM, HALF>(n);
                half0 += half_rows<BM, HALF>(n);
                prev = s.end[e];
            }
            if (e1 == E + 1 && e0 < e1) {
                s.big[E + 1] = big0;
                s.half[E + 1] = half0;
            }
        }
    }
    barrier_after_lds_write();
}

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// The last group whose first, as first(group) says, is <= x.
template <typename First>
__device__ __forceinline__ int group_of(int E, int x, First first)
{
    int lo = 0, hi = E + 1;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (uniform(first(mid)) <= x)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

// Ends with a barrier.
__device__ __forceinline__ void order_groups(KGroups& s, int E)
{
    for (int e = threadIdx.x; e < E; e += NT) {
        const int n = s.end[e] - (e ? s.end[e - 1] : 0);
        int rank = 0, prev = 0;
        for (int f = 0; f < E; ++f) {
            const int end = s.end[f], m = end - prev;
            rank += m > n || (m == n && f < e);
            prev = end;
        }
        s.order[rank] = e;
    }
    barrier_after_lds_write();
}

// Tile t of a rows x cols grid, GROUP_M tile rows at a time column by column, so that the tiles in flight
// share rows of A and of B in the caches.
__device__ __forceinline__ void tile_of(int t, int rows, int cols, int& m, int& n)
{
    const int per = GROUP_M * cols, group = t / per, first = group * GROUP_M;
    const int here = min(rows - first, GROUP_M), in = t - group * per;
    n = in / here;
    m = first + in - n * here;
}

// How the last tiles are cut: `cut` units (tile rows, or two halves) go in halves or, four for a tile, in quarters.
struct Tail {
    int cut;
    bool quarters;
};

// A last round of tiles that fills few of G workgroups becomes a shorter one: n units and `lone` halves of c tiles, cq
// columns of quarters each.  In twentieths of a tile's time a half takes about 12 and a quarter 6, 7 where there is
// more than a round of them.
__host__ __device__ __forceinline__ Tail tail_of(int n, int lone, int c, int cq, int G)
{
    const int last = (int)((int64_t)n * c % G), d = (last + c - 1) / c;
    const int free0 = last ? G - last : 0, free1 = d * c - last;       // workgroups left idle without and with cutting
    auto halves = [&](int rows, int idle) { return 12 * ((max((int64_t)0, (int64_t)rows * c - 2 * idle) + G - 1) / G); };
    auto quarters = [&](int rows, int idle) {
        const int64_t q = max((int64_t)0, (int64_t)rows * cq - 3 * idle);
        return q > G ? 7 * ((q + G - 1) / G) : q > 0 ? (int64_t)6 : 0;
    };
    int64_t best = (last ? 20 : 0) + halves(lone, free0);
    Tail t = {0, false};
    if ((last ? 20 : 0) + quarters(lone, free0) < best) {
        best = (last ? 20 : 0) + quarters(lone, free0);
        t = {0, true};
    }
    if (last && halves(lone + 2 * d, free1) < best) {
        best = halves(lone + 2 * d, free1);
        t = {d, false};
    }
    if (last && quarters(lone + 2 * d, free1) < best)
        t = {d, true};
    return t;
}

// ------------------------------------------------------------------------------ cross entropy
// Softmax statistics of the columns [col, col + 8) of a row, n of them valid: LPR neighbouring lanes hold
// the row's part that pair `slot` covers, so the steps below stay inside the row.
template <int LPR>
__device__ __forceinline__ void stat8(const TileArgs& a, int64_t mrow, int64_t M, int64_t col, int n, int64_t slot,
                                      int lane, const float* x)
{
    float mx = -INFINITY;
    bool nan = false;
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (e < n) {
            mx = fmaxf(mx, x[e]);
            nan |= x[e] != x[e];
        }
#pragma unroll
    for (int s = 1; s < LPR; s <<= 1)
        mx = fmaxf(mx, __shfl_xor(mx, s));
    const float base = mx == -INFINITY ? 0.0f : mx;
    float sum = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (e < n)
            sum += fast_exp(x[e] - base);
    if (nan)
        sum = NAN;
#pragma unroll
    for (int s = 1; s < LPR; s <<= 1)
        sum += __shfl_xor(sum, s);
    if (mrow < M) {
        if ((lane % LPR) == 0) {
            float* p = a.stat + (mrow * a.stat_n + slot) * 2;
            p[0] = mx;
            p[1] = sum;
        }
        const int64_t y = a.targets[mrow] - col;
        if (y >= 0 && y < n) {
            float hit = 0.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e)
                hit = e == (int)y ? x[e] : hit;
            a.hit[mrow] = hit;
        }
    }
}

// d logits are rounded to bf16 for the products that follow, whose matrix instructions take both factors so.  They are
// counted in units of one of dloss's values, which multiplies the sums: where all rows have the same (a mean's 1 / n),
// what is rounded is softmax - 1 at the targets, next to -1 and exact there, and not -1 / n, whose error every row would
// have alike (the gradients' norm was up to 2^-8 too large or too small).  The unit is the first of 64 evenly spread
// rows' values between 2^-40 and 2^40, or 1.  What a lane has read of them, loaded ahead of its use:
__device__ __forceinline__ float loss_sample(const float* dloss, int64_t rows)
{
    return rows > 0 ? fabsf(dloss[(int64_t)(threadIdx.x & 63) * rows >> 6]) : 1.0f;
}
// All lanes of the wave.
__device__ __forceinline__ float loss_unit(float sample)
{
    const uint64_t fit = __ballot(sample >= 0x1p-40f && sample <= 0x1p40f);
    return fit ? __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, sample), __builtin_ctzll(fit)))
               : 1.0f;
}

// d logits = dloss / unit (softmax - one at the target); padding columns of the buffer are zero.
__device__ __forceinline__ void grad8(const TileArgs& a, int64_t mrow, int64_t M, int64_t col, int n, const float* x,
                                      float unit)
{
    if (mrow >= M || col >= a.out.ldc)
        return;
    const int64_t y = a.targets[mrow];
    const bool has = y >= 0 && y < a.vocab;
    const float lse = a.lse[mrow], w = has ? a.dloss[mrow] / unit : 0.0f;
    const int64_t hit = y - a.col0 - col;
    bf16x8 o;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        float p = fast_exp(x[e] - lse);
        if (hit == e)
            p -= 1.0f;
        o[e] = (__bf16)(e < n && has ? p * w : 0.0f);
    }
    *reinterpret_cast<bf16x8*>(a.out.C + mrow * a.out.ldc + col) = o;
}

// A tile's 32 rows x 32 FN columns in the accumulators of a wave, transposed: lane l has row l % 32 and, of each
// 8 columns, the four from 4 (l / 32); acc[j][4 q + e] is column 32 j + 8 q + 4 (l / 32) + e.  Two lanes have a
// row, so a row's maximum and sum need one step between lanes and no LDS.  `n`: valid columns of the block, yo:
// the target's column in it, or -1.
template <int FN>
__device__ __forceinline__ void stat_block(const TileArgs& a, const f32x16* acc, int64_t row0, int64_t rows, int n, int yo,
                                           int64_t slot, int lane)
{
    const uint32_t fh = lane >> 5;
    const int64_t mrow = row0 + (lane & 31);
    const bool valid = mrow < rows;
    const int nr = n - (int)fh * 4;            // valid columns counted from the lane's first
    constexpr float kLog2e = 1.4426950408889634f;
    float v[FN * 16];
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
        for (int e = 0; e < 16; ++e)
            v[j * 16 + e] = acc[j][e];
    if (n < FN * 32) {                         // the vocabulary's last columns
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
            for (int e = 0; e < 16; ++e)
                if (j * 32 + (e >> 2) * 8 + (e & 3) >= nr)
                    v[j * 16 + e] = -INFINITY;
    }
    float mx = v[0];                           // fmaxf passes over NaN: it comes back in the sum
#pragma unroll
    for (int e = 1; e < FN * 16; ++e)
        mx = fmaxf(mx, v[e]);
    mx = fmaxf(mx, __shfl_xor(mx, 32));
    const float base = mx == -INFINITY || mx != mx ? 0.0f : mx * kLog2e;
    float sum[4] = {};
#pragma unroll
    for (int e = 0; e < FN * 16; ++e)
        sum[e & 3] += __builtin_amdgcn_exp2f(fmaf(v[e], kLog2e, -base));
    float all = (sum[0] + sum[1]) + (sum[2] + sum[3]);
    all += __shfl_xor(all, 32);
    if (valid && fh == 0) {
        float2* p = reinterpret_cast<float2*>(a.stat) + mrow * a.stat_n + slot;
        *p = make_float2(mx, all);
    }
    const bool here = valid && yo >= 0 && yo < n && ((uint32_t)yo >> 2 & 1) == fh;
    if (__ballot(here)) {
        const int at = (yo >> 5) * 16 + (yo >> 3 & 3) * 4 + (yo & 3);
        float hit = 0.0f;
#pragma unroll
        for (int e = 0; e < FN * 16; ++e)
            hit = e == at ? v[e] : hit;
        if (here)
            a.hit[mrow] = hit;
    }
}

// A wave's block in bf16 through its LDS slab: 32 rows of 64 FN bytes, 16-byte units swizzled by the row, the
// units' halves by the row's bit 4, so that 32 rows of one column fall into distinct banks.
template <int FN>
__device__ __forceinline__ bf16x4* half_slab_at(char* slab, int j, int q, uint32_t fr, uint32_t fh)
{
    constexpr uint32_t RB = FN * 64, UN = RB / 16;
    return reinterpret_cast<bf16x4*>(slab + fr * RB + (fh ^ (fr >> 4)) * 8 + (((uint32_t)(j * 4 + q) ^ (fr & (UN - 1))) * 16));
}

// The slab to memory in 16-byte pieces; p: the block's first element, rows, cols: what is valid of it.  PAST: the
// stores pass the tiles' lines in L2 by (16384 x 14336 x 4096 takes 5 % more without).
template <int FN, bool PAST>
__device__ __forceinline__ void half_slab_out(const char* slab, __bf16* p, int64_t ld, int64_t rows, int64_t cols, int lane)
{
    constexpr uint32_t RB = FN * 64, UN = RB / 16;         // bytes and 16-byte units of a slab row
    constexpr int RPI = 64 / UN;                           // rows of one read-back
    __builtin_amdgcn_s_waitcnt(0xC07F);   // lgkmcnt(0): this wave's slab is written
    __builtin_amdgcn_wave_barrier();
    const uint32_t u = lane % UN, r0 = lane / UN;
    p += r0 * ld + u * 8;
    auto row_of = [&](int it) {
        const uint32_t r = it * RPI + r0;
        const i32x4 x = *reinterpret_cast<const i32x4*>(slab + r * RB + ((u ^ (r & (UN - 1))) * 16));
        return it * RPI >= 16 ? i32x4{x[2], x[3], x[0], x[1]} : x;   // RPI divides 16
    };
    if (cols >= FN * 32) {
#pragma unroll
        for (int it = 0; it < 32 / RPI; ++it) {
            const i32x4 y = row_of(it);
            i32x4_any* const out = reinterpret_cast<i32x4_any*>(p + it * RPI * ld);
            if (it * RPI + r0 < rows) {
                if (PAST)
                    __builtin_nontemporal_store(y, out);
                else
                    *out = y;
            }
        }
    } else {                                               // the last columns
#pragma unroll 2
        for (int it = 0; it < 32 / RPI; ++it) {
            const bf16x8 y = __builtin_bit_cast(bf16x8, row_of(it));
            const int n = (int)cols - (int)u * 8;
            if (it * RPI + r0 < rows) {
                if (n >= 8)
                    *reinterpret_cast<bf16x8_any*>(p + it * RPI * ld) = y;
                else
#pragma unroll
                    for (int e = 0; e < 7; ++e)
                        if (e < n)
                            p[it * RPI * ld + e] = y[e];
            }
        }
    }
    __builtin_amdgcn_s_waitcnt(0xC07F);   // reads done before the slab is rewritten
    __builtin_amdgcn_wave_barrier();
}

// d logits of the same block, w (softmax - one at the target) with w = dloss / unit, rounded to bf16; zero in rows
// without a target.  neg_lse2: -lse log2(e).
template <int FN>
__device__ __forceinline__ void grad_block(const TileArgs& a, const f32x16* acc, char* slab, int64_t ldc, int64_t row0, int64_t rows,
                                           int64_t col0, int n, int yo, bool has, float neg_lse2, float w, int lane)
{
    constexpr float kLog2e = 1.4426950408889634f;
    const uint32_t fr = lane & 31, fh = lane >> 5;
    const int nr = has ? n - (int)fh * 4 : 0;  // valid columns counted from the lane's first
    float p[FN * 16];
#pragma unroll
    for (int e = 0; e < FN * 16; ++e)
        p[e] = __builtin_amdgcn_exp2f(fmaf(acc[e >> 4][e & 15], kLog2e, neg_lse2));
    if (__ballot(yo >= 0)) {
        const int at = ((uint32_t)yo >> 2 & 1) == fh ? (yo >> 5) * 16 + (yo >> 3 & 3) * 4 + (yo & 3) : -1;
#pragma unroll
        for (int e = 0; e < FN * 16; ++e)
            p[e] -= yo >= 0 && e == at ? 1.0f : 0.0f;
    }
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            bf16x4 o;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                o[e] = (__bf16)(j * 32 + q * 8 + e < nr ? p[j * 16 + q * 4 + e] * w : 0.0f);
            }
            *half_slab_at<FN>(slab, j, q, fr, fh) = o;
        }
    half_slab_out<FN, false>(slab, a.out.C + row0 * ldc + col0, ldc, rows - row0, ldc - col0, lane);
}

// act(x + bias) + residual of the same block, x in the accumulators, through the wave's LDS slab (32 rows of
// 128 FN bytes of fp32, 16-byte units swizzled by the row); or x itself into `part` where the reduction is
// split (all that there is without ACT).  A row's eight columns come back to one lane.  part and C: the block's first row and column; at: the
// same place in residual and pre; rows, cols: what is valid of the block.
template <int FN, bool ACT, typename Fill>
__device__ __forceinline__ void linear_block(const TileArgs& a, Fill fill, char* slab, __bf16* C, float* part,
                                             int64_t at, int64_t ldc, int64_t ldp, int rows, int cols, const float* bias,
                                             bool between, int lane)
{
    constexpr int WNC = FN * 32;
    constexpr uint32_t SW = WNC / 4 - 1;           // 16-byte units of a slab row, minus one
    constexpr int LPR = WNC / 8;                   // lanes per slab row on the way back
    constexpr int ITS = WNC / 16, RSTEP = 64 / LPR;  // read-backs of a slab, rows of one
    const uint32_t fr = lane & 31, fh = lane >> 5;
    const uint32_t c8 = (lane % LPR) * 8;
    const int r0 = lane / LPR, n = min(8, cols - (int)c8);
    const bool edge = cols < WNC, residual = ACT && a.out.residual && !part;      // edge: some lanes have less than eight
    at += r0 * ldc + c8;
    C += r0 * ldc + c8;
    // the slab's residual is on its way while the slab is written
    bf16x8 res[ITS] = {};
    if (residual && (!edge || n >= 8)) {
#pragma unroll
        for (int it = 0; it < ITS; ++it)
            if (r0 + it * RSTEP < rows)
                res[it] = *reinterpret_cast<const bf16x8_any*>(a.out.residual + at + it * RSTEP * ldc);
    }
    if (residual && edge && n < 8) {
#pragma unroll
        for (int it = 0; it < ITS; ++it)
            if (r0 + it * RSTEP < rows)
                res[it] = load8_few(a.out.residual + at + it * RSTEP * ldc, n);
    }
    fill([&](const f32x16* acc) {
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const uint32_t colb = (j * 32 + q * 8 + fh * 4) * 4;
                const f32x4 v4 = {acc[j][q * 4 + 0], acc[j][q * 4 + 1], acc[j][q * 4 + 2], acc[j][q * 4 + 3]};
                *reinterpret_cast<f32x4*>(slab + fr * (WNC * 4) + (colb ^ ((fr & SW) << 4))) = v4;
            }
    });
    __builtin_amdgcn_s_waitcnt(0xC07F);   // lgkmcnt(0): this wave's slab is written
    __builtin_amdgcn_wave_barrier();
    auto unit = [&](int it, int half) {   // four of this lane's eight columns in its row it
        const uint32_t r = it * RSTEP + r0;
        return reinterpret_cast<f32x4*>(slab + r * (WNC * 4) + (((c8 + 4 * half) * 4) ^ ((r & SW) << 4)));
    };
    if (part) {
        part += r0 * ldp + c8;
#pragma unroll
        for (int it = 0; it < ITS; ++it) {
            f32x4 x0 = *unit(it, 0), x1 = *unit(it, 1);
            if (r0 + it * RSTEP < rows && n > 0) {       // ldp % 8 == 0: whole vectors
                f32x4* pv = reinterpret_cast<f32x4*>(part + it * RSTEP * ldp);
                if (a.accumulate) {
                    x0 += pv[0];
                    x1 += pv[1];
                }
                pv[0] = x0;
                pv[1] = x1;
            }
        }
    } else if constexpr (ACT) {
        // bias, pre and the activation in a loop of their own: unrolled into the stores below, the activations
        // would be there once for each row of the block
        auto activate = [&](int it, auto store_pre) {
            const f32x4 x0 = *unit(it, 0), x1 = *unit(it, 1);
            float x[8] = {x0[0] + bias[0], x0[1] + bias[1], x0[2] + bias[2], x0[3] + bias[3],
                          x1[0] + bias[4], x1[1] + bias[5], x1[2] + bias[6], x1[3] + bias[7]};
            if (a.out.pre && r0 + it * RSTEP < rows)
                store_pre(a.out.pre + at + it * RSTEP * ldc, x);
            act_value8(x, a.out.act);
            if (residual || edge) {
                *unit(it, 0) = f32x4{x[0], x[1], x[2], x[3]};
                *unit(it, 1) = f32x4{x[4], x[5], x[6], x[7]};
            } else if (r0 + it * RSTEP < rows) {
                store8(C + it * RSTEP * ldc, x);
            }
        };
        if (between && edge) {
#pragma unroll 1
            for (int it = 0; it < ITS; ++it)
                activate(it, [&](__bf16* p, const float* x) { store8(p, n, x); });
        } else if (between) {
#pragma unroll 2
            for (int it = 0; it < ITS; ++it)
                activate(it, [&](__bf16* p, const float* x) { store8(p, x); });
        }
        if (residual) {
#pragma unroll
            for (int it = 0; it < ITS; ++it) {
                f32x4 x0 = *unit(it, 0), x1 = *unit(it, 1);
                x0 += f32x4{(float)res[it][0], (float)res[it][1], (float)res[it][2], (float)res[it][3]};
                x1 += f32x4{(float)res[it][4], (float)res[it][5], (float)res[it][6], (float)res[it][7]};
                if (edge) {
                    *unit(it, 0) = x0;
                    *unit(it, 1) = x1;
                } else if (r0 + it * RSTEP < rows) {
                    const float x[8] = {x0[0], x0[1], x0[2], x0[3], x1[0], x1[1], x1[2], x1[3]};
                    store8(C + it * RSTEP * ldc, x);
                }
            }
        }
        if (edge) {
#pragma unroll 1
            for (int it = 0; it < ITS; ++it) {
                const f32x4 x0 = *unit(it, 0), x1 = *unit(it, 1);
                const float x[8] = {x0[0], x0[1], x0[2], x0[3], x1[0], x1[1], x1[2], x1[3]};
                if (r0 + it * RSTEP < rows)
                    store8(C + it * RSTEP * ldc, n, x);
            }
        }
    }
    __builtin_amdgcn_s_waitcnt(0xC07F);   // reads done before the slab is rewritten
    __builtin_amdgcn_wave_barrier();
}

// ---------------------------------------------------------------------------------- the kernel
// The stages, in arrays of their own: the compiler then sees that the loads in flight fill another stage than the
// one being read, and does not wait for them.  slab: this wave's part of them in the epilogue.
template <int S>
struct Stages {
    Part a[S], b[S];
    char* slab;
};

// Where a tile lies: its first row within its group (or among all rows) and first column.
struct Where {
    int64_t m0, n0, M, K, k_first, grow0;
    int tn, g, split;
    bool zero;                                         // rows past the last group
    float scale = 1.0f;                                // newton_schulz: OrthoArgs::scale of the tile's matrix
};

struct OrthoArgs;
template <int EPI, int FM, int FN, int WM, typename Acc>
__device__ void after_sums(const OrthoArgs& a, const Where& w, Acc acc, char* slab, int64_t row0, int64_t col0, int lane);

// One tile.  EPI: kEpiLinear, kEpiSum (the sums alone: a kernel without the activations' code
// takes 37 us instead of 41 for 16384 x 4096 x 8), kEpiScaled (the sums times the unit of the d logits), kEpiStat (softmax
// statistics of a row's columns), kEpiGrad (d logits).  From kEpiGram on the factors are fp16 and what follows is
// after_sums(), which lm_ortho.hip has.
template <int BM, int BN, int WM, int WN, int S, bool TA, bool TB, int EPI, typename Args = TileArgs>
__device__ __forceinline__ void product_tile(const Args& a, const Stages<S>& l, const Where& w)
{
    static_assert(WM * WN == 4, "four waves");
    constexpr int FM = BM / WM / 32, FN = BN / WN / 32, NM = FM * FN;
    typedef Side<BM, TA> SA;
    typedef Side<BN, TB> SB;
    constexpr int ND = SA::OPS + SB::OPS;
    constexpr int WNC = FN * 32;                       // columns of a wave's block
    constexpr bool LIN = EPI == kEpiLinear || EPI == kEpiSum || EPI == kEpiScaled, FP16 = EPI >= kEpiGram;

    const int tid = threadIdx.x;
    const int lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / WN, wn = wave % WN;
    const int64_t m0 = w.m0, n0 = w.n0, M = w.M, K = w.K, grow0 = w.grow0, g = w.g, split = w.split;

    SA sa;
    SB sb;
    Frag<BM, TA, FM, true> fa;
    Frag<BN, TB, FN, false> fb;
    fa.init(lane, wm);
    fb.init(lane, wn);
    sa.init(tid, a.lda);
    sb.init(tid, a.ldb);
    const uint32_t wave_off = wave * 1024;
    {
        const int64_t a_rows = min((int64_t)BM, M - m0), b_rows = min((int64_t)BN, a.N - n0);
        const int64_t gb = w.zero ? 0 : g;
        const __bf16* const Ab = TA ? a.A + w.k_first * a.lda + m0 : a.A + (grow0 + m0) * a.lda;
        const __bf16* const Bb = TB ? a.B + (a.group == kGroupK ? w.k_first * a.ldb : gb * a.strideB) + n0
                                    : a.B + gb * a.strideB + n0 * a.ldb;
        const int64_t nk_all = (K + BK - 1) / BK;
        const int64_t kb0 = min(split * a.split_steps, nk_all);
        const int64_t kb1 = a.splits > 1 ? min(kb0 + a.split_steps, nk_all) : nk_all;
        const int64_t k_end = min(K, kb1 * BK);
        sa.start(Ab, a_rows, K, m0, kb0, k_end);
        sb.start(Bb, b_rows, K, n0, kb0, !TA && TB ? min(k_end, a.k_valid) : k_end);

        f32x16 acc[FM][FN];
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int j = 0; j < FN; ++j)
#pragma unroll
                for (int v = 0; v < 16; ++v)
                    acc[i][j][v] = 0.0f;

        // cross entropy: what a lane's rows need in the epilogue is on its way during the K loop
        const uint32_t fr = lane & 31;
        int64_t target[FM];
        float row_lse[FM], row_w[FM], sample = 1.0f;
        if constexpr (EPI == kEpiGrad || EPI == kEpiScaled)
            sample = loss_sample(a.dloss, a.dloss_rows);
        if constexpr (!LIN && !FP16) {
#pragma unroll
            for (int i = 0; i < FM; ++i) {
                const int64_t mrow = min(m0 + (i * WM + wm) * 32 + fr, M - 1);
                target[i] = a.targets[mrow];
                if (EPI == kEpiGrad) {
                    row_lse[i] = a.lse[mrow];
                    row_w[i] = a.dloss[mrow];
                }
            }
        }

        struct Dma {
            __amdgpu_buffer_rsrc_t ra, rb;
            uint32_t va, vb, lw, sa_, sb_;
            Part la, lb;
        };
        // the next step's loads, into a stage; past the last step they read nothing but still count
        auto dma_setup = [&](int c) {
            Dma d;
            d.lw = wave_off;
            d.sa_ = sa.op_stride;
            d.sb_ = sb.op_stride;
            asm volatile("" : "+s"(d.lw), "+s"(d.sa_), "+s"(d.sb_));
            d.ra = sa.rsrc();
            d.rb = sb.rsrc();
            d.va = sa.offset();
            d.vb = sb.offset();
            d.la = l.a[c];
            d.lb = l.b[c];
            sa.advance();
            sb.advance();
            return d;
        };
        auto dma_op = [&](const Dma& d, int q) {
            if (q < SA::OPS)
                sa.load(d.ra, d.la, d.lw, d.va, d.sa_, q);
            else
                sb.load(d.rb, d.lb, d.lw, d.vb, d.sb_, q - SA::OPS);
        };
        auto issue_all = [&](int c) {
            const Dma d = dma_setup(c);
#pragma unroll
            for (int q = 0; q < ND; ++q)
                dma_op(d, q);
        };
        // MFMAs of one substep out of (bf, af), with what is to be issued between them: the next
        // substep's fragment reads (out of stage c), one after each of the first MFMAs, and loads
        // [q0, q1) spread over all of them, so neither queue backs up into the matrix instructions.
        bf16x8 af[2][FM], bf[2][FN];
        auto block = [&](int set, int c, int next, const Dma& d, int q0, int q1) {
            const int other = set ^ 1;
#pragma unroll
            for (int gi = 0; gi < NM; ++gi) {
                const int i = gi / FN, j = gi % FN;
                if constexpr (FP16)
                    acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, bf[set][j]),
                                                                       __builtin_bit_cast(f16x8, af[set][i]), acc[i][j], 0, 0, 0);
                else
                    acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(bf[set][j], af[set][i], acc[i][j], 0, 0, 0);
                __builtin_amdgcn_sched_barrier(0);
                constexpr int NR = FM + FN;
                constexpr int RS = NM >= NR ? NR : NM;            // MFMAs that a read follows
                if (next >= 0 && gi < RS) {
#pragma unroll
                    for (int r = gi * NR / RS; r < (gi + 1) * NR / RS; ++r) {
                        if (r < FN)
                            bf[other][r] = fb.read(l.b[c], next, r);
                        else
                            af[other][r - FN] = fa.read(l.a[c], next, r - FN);
                    }
                }
#pragma unroll
                for (int q = q0 + (q1 - q0) * gi / NM; q < q0 + (q1 - q0) * (gi + 1) / NM; ++q)
                    dma_op(d, q);
                __builtin_amdgcn_sched_barrier(0);
            }
        };
        auto first_frags = [&](int c) {
#pragma unroll
            for (int j = 0; j < FN; ++j)
                bf[0][j] = fb.read(l.b[c], 0, j);
#pragma unroll
            for (int i = 0; i < FM; ++i)
                af[0][i] = fa.read(l.a[c], 0, i);
            __builtin_amdgcn_sched_barrier(0);
        };

        if constexpr (S == 1) {
            // one stage: what is loaded is waited for, while other workgroups of the CU compute and store
            for (int64_t kb = kb0; kb < kb1; ++kb) {
                issue_all(0);
                wait_vmcnt0();
                stage_barrier();
                const Dma none = {};
                first_frags(0);
                block(0, 0, 1, none, 0, 0);
                block(1, 0, 2, none, 0, 0);
                block(0, 0, 3, none, 0, 0);
                block(1, 0, -1, none, 0, 0);
                stage_barrier();
            }
        } else {
            // A step out of stage c is four substeps; its barrier stands before the last one: there every wave
            // has read all of stage c's fragments, and the next stage's loads have landed.  The last substep's
            // MFMAs then cover the first fragment reads of the next step and the first half of the loads that
            // refill stage c; the other half follows in the next step's first substep.
            Dma d;
            auto step = [&](int c) {
                const int n = (c + 1) % S;
                block(0, c, 1, d, ND / 2, ND);
                block(1, c, 2, d, 0, 0);
                block(0, c, 3, d, 0, 0);
                wait_vmcnt<(S - 2) * ND>();
                stage_barrier();
                d = dma_setup(c);
                block(1, n, 0, d, 0, ND / 2);
            };
            // the start of a tile: its first S - 1 steps into the stages from c on, half of the next one
            auto start = [&](int c) {
#pragma unroll
                for (int i = 0; i < S - 1; ++i)
                    issue_all((c + i) % S);
                wait_vmcnt<(S - 2) * ND>();
                stage_barrier();
                d = dma_setup((c + S - 1) % S);
#pragma unroll
                for (int q = 0; q < ND / 2; ++q)
                    dma_op(d, q);
                first_frags(c);
            };
            int64_t kb = kb0;
            if constexpr (S == 2) {
                // with an odd number of steps the first runs alone out of stage 1, so the pair loop always
                // computes twice per iteration
                if ((kb1 - kb0) & 1) {
                    start(1);
                    step(1);
                    ++kb;
                } else if (kb1 > kb0) {
                    start(0);
                }
            } else if (kb1 > kb0) {
                start(0);
            }
            for (; kb + S <= kb1; kb += S) {
#pragma unroll
                for (int c = 0; c < S; ++c)
                    step(c);
            }
            if constexpr (S > 2) {               // what is left, out of the first stages
                if (kb < kb1) {
                    step(0);
                    if (kb + 1 < kb1) {
                        step(1);
                        if (S > 3 && kb + 2 < kb1)
                            step(2);
                    }
                }
            }
        }
        wait_vmcnt0();     // loads past the last step have landed too
        __syncthreads();   // all waves are done with the stages

        // ---- epilogue, 32 rows of the wave's block at a time
        char* const slab = l.slab;
        // one block at a time in registers: its accumulators leave the matrix unit's registers here and not
        // before, and nothing it computes is shared with the next block's or moved across
        auto one_block = [&](f32x16* blk, int& lane_, int& flag) {
            __builtin_amdgcn_sched_barrier(0);
            if constexpr (NM >= 16) {
#pragma unroll
                for (int j = 0; j < FN; ++j)
                    asm volatile("" : "+a"(blk[j]));
            }
            asm volatile("" : "+v"(lane_), "+s"(flag));
        };
        // what only the epilogue uses is computed here, not ahead of the tile loop where it would hold registers
        // through the K loop
        int el = lane;
        int64_t ldc = a.out.ldc, ldp = a.ldp;
        asm volatile("" : "+v"(el), "+s"(ldc), "+s"(ldp));
        const int64_t wcol = n0 + wn * WNC;                            // the wave's first column
        const int wcols = (int)max((int64_t)0, min((int64_t)WNC, a.N - wcol));
        if constexpr (FP16) {
            after_sums<EPI, FM, FN, WM>(a, w, [&](int i) {
                int flag = 0;
                one_block(acc[i], el, flag);
                return acc[i];
            }, slab, m0 + wm * 32, wcol, el);
        } else if constexpr (LIN) {
            const int64_t mrow0 = m0 + wm * 32;                        // blocks WM x 32 rows apart
            const int64_t at = (grow0 + mrow0) * ldc + wcol;
            __bf16* const C = a.out.C + (a.group == kGroupK ? g * a.M * ldc : 0) + at;
            float* const part = a.part ? a.part + (split * a.M + mrow0) * ldp + wcol : nullptr;
            const bool between = a.out.bias || a.out.pre || a.out.act != kActNone;
            float bias[8] = {};
            const int c8 = (el % (WNC / 8)) * 8, n = min(8, wcols - c8);
            if (EPI == kEpiLinear && a.out.bias && n > 0)
                load8(a.out.bias + wcol + c8, n, bias);
            if (EPI == kEpiScaled || a.plain) {
                const float unit = EPI == kEpiScaled ? loss_unit(sample) : 1.0f;
#pragma unroll
                for (int i = 0; i < FM; ++i) {
                    int cols = wcols;
                    one_block(acc[i], el, cols);
                    auto value = [&](int j, int e) {
                        return (__bf16)(EPI == kEpiScaled ? acc[i][j][e] * unit : acc[i][j][e]);
                    };
#pragma unroll
                    for (int j = 0; j < FN; ++j)
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            *half_slab_at<FN>(slab, j, q, el & 31, (uint32_t)el >> 5) =
                                bf16x4{value(j, q * 4 + 0), value(j, q * 4 + 1), value(j, q * 4 + 2), value(j, q * 4 + 3)};
                    half_slab_out<FN, true>(slab, C + i * WM * 32 * ldc, ldc, M - mrow0 - i * WM * 32, cols, el);
                }
            } else {
                // a loop at run time, in which only the accumulators' way into the slab is there for each block:
                // the waves of a CU go through this code one tile at a time, and what the instruction cache does
                // not hold they wait for (four copies: silu 5 % more time at 8192 x 8192 x 2048)
#pragma unroll 1
                for (int i = 0; i < FM; ++i) {
                    __builtin_amdgcn_sched_barrier(0);
                    auto fill = [&](auto write) {
                        each<FM>([&](auto index) {
                            constexpr int I = decltype(index)::value;
                            if (i == I) {
                                int flag = 0;
                                one_block(acc[I], el, flag);
                                write(acc[I]);
                            }
                        });
                    };
                    linear_block<FN, EPI == kEpiLinear>(
                        a, fill, slab, C + i * WM * 32 * ldc, part ? part + i * WM * 32 * ldp : nullptr,
                        at + i * WM * 32 * ldc, ldc, ldp, (int)max((int64_t)0, min((int64_t)32, M - mrow0 - i * WM * 32)),
                        wcols, bias, between, el);
                }
            }
        } else {
            const float unit = EPI == kEpiGrad ? loss_unit(sample) : 1.0f;
#pragma unroll
            for (int i = 0; i < FM; ++i) {
                int cols = wcols;
                one_block(acc[i], el, cols);
                const int64_t brow = m0 + (i * WM + wm) * 32;
                const int64_t y = target[i] - a.col0 - wcol;
                const int yo = y >= 0 && y < WNC ? (int)y : -1;
                if constexpr (EPI == kEpiStat) {
                    // a pair for each 64 columns, whatever the tile
#pragma unroll
                    for (int h = 0; h < FN / 2; ++h)
                        if (cols > h * 64)
                            stat_block<2>(a, acc[i] + h * 2, brow, M, min(64, cols - h * 64),
                                          yo >= h * 64 && yo < h * 64 + 64 ? yo - h * 64 : -1, wcol / 64 + h, el);
                } else {
                    const bool has = target[i] >= 0 && target[i] < a.vocab;
                    grad_block<FN>(a, acc[i], slab, ldc, brow, M, wcol, cols, yo, has, -row_lse[i] * 1.4426950408889634f,
                                   row_w[i] / unit, el);
                }
            }
        }
        __syncthreads();   // LDS is free for the next tile's loads
    }
}

// The tiles of one workgroup.  HALF: tiles of half the height exist too, for what is left of a group's rows, and with
// quarters for the last round of tiles.
template <int BM, int BN, int WM, int WN, int S, bool TA, bool TB, int EPI, bool HALF>
__device__ __forceinline__ void tile_body(const TileArgs& a)
{
    // The half tile has three stages, for it computes on one for half as long: A of two in the halves of A's first
    // stage, in arrays of their own, B of the third where A's second is.
    constexpr int AB = Side<BM, TA>::BYTES, BB = Side<BN, TB>::BYTES, HALF_A = 16384;
    static_assert(!HALF || (AB == 32768 && BB == 32768), "256 x 256");
    __shared__ __attribute__((aligned(1024))) char sA0[HALF ? HALF_A : AB], sU0[HALF ? HALF_A : 16];
    __shared__ __attribute__((aligned(1024))) char sB0[BB];
    __shared__ __attribute__((aligned(1024))) char sA1[S > 1 ? AB : 16];
    __shared__ __attribute__((aligned(1024))) char sB1[S > 1 ? BB : 16];
    __shared__ __attribute__((aligned(1024))) char sA2[S > 2 ? AB : HALF ? HALF_A : 16];
    __shared__ __attribute__((aligned(1024))) char sB2[S > 2 ? BB : 16];
    __shared__ __attribute__((aligned(1024))) char sA3[S > 2 ? AB : 16];
    __shared__ __attribute__((aligned(1024))) char sB3[S > 2 ? BB : 16];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    constexpr int SLAB = 32 * (BN / WN) * 4;           // 32 rows of a wave's block in fp32
    Stages<S> l;
    l.a[0] = {sA0, sU0};
    l.b[0] = {sB0, sB0 + 16384};
    if constexpr (S > 1) {
        l.a[1] = {sA1, sA1 + AB / 2};
        l.b[1] = {sB1, sB1 + 16384};
    }
    if constexpr (S == 4) {

        l.a[2].lo = sA2;
        l.b[2] = {sB2, sB2 + 16384};
        l.a[3].lo = sA3;
        l.b[3] = {sB3, sB3 + 16384};
        static_assert(2 * SLAB <= BB, "slabs fit two stages of B");
        l.slab = (wave < 2 ? sB0 : sB1) + (wave & 1) * SLAB;
    } else {
        static_assert(HALF ? SLAB == HALF_A : 2 * SLAB <= AB && 2 * SLAB <= BB, "slabs fit a stage");
        l.slab = wave >= 2 ? sB0 + (wave - 2) * SLAB : !HALF ? sA0 + wave * SLAB : wave ? sU0 : sA0;
    }
    Stages<3> lh;
    if constexpr (HALF) {
        lh.a[0].lo = sA0;
        lh.a[1].lo = sU0;
        lh.a[2].lo = sA2;
        lh.b[0] = l.b[0];
        lh.b[1] = l.b[1];
        lh.b[2] = l.a[1];
        lh.slab = l.slab;
    }
    constexpr bool LIN = EPI == kEpiLinear || EPI == kEpiSum, ROWS = LIN && !TA && S > 1, KS = LIN && TA && S > 1;   // groups there can be
    __shared__ typename std::conditional<ROWS, Groups, typename std::conditional<KS, KGroups, int>::type>::type s_groups;

    // a quarter's four stages, each of one array (or two)
    Stages<4> lq;
    if constexpr (HALF) {
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

    const int G = gridDim.x;
    // workgroups are dispatched round-robin over the 8 XCDs: each XCD takes a contiguous run of tiles
    const int vid = (G % 8 == 0) ? (int)(blockIdx.x % 8) * (G / 8) + (int)(blockIdx.x / 8) : (int)blockIdx.x;
    const int cols = (int)a.tiles_n;
    const bool by_rows = ROWS && a.group == kGroupRows, by_k = KS && a.group == kGroupK;

    // Units of one tile's time: a tile row, or two groups' halves, which stand where the second group's rows end,
    // so that a group's weights are read for its tiles and its half at about the same time.  `lone`: a half left
    // over.  (Of groups that split the reduction each has all the rows.)
    int nb = big_rows<BM, HALF>((int)a.M), nh = half_rows<BM, HALF>((int)a.M);
    if constexpr (ROWS) {
        if (by_rows) {
            group_scan<BM, HALF>(a.ends, a.E, a.M, s_groups);
            nb = uniform(s_groups.big[a.E + 1]);
            nh = uniform(s_groups.half[a.E + 1]);
        }
    }
    if constexpr (KS) {
        if (by_k) {
            group_scan<BM, HALF>(a.ends, a.E, a.K, s_groups);
            order_groups(s_groups, a.E);
        }
    }
    const int parts = by_k ? a.E : a.splits, lone = nh & 1;
    const int all_units = nb + nh / 2, quarter_cols = (int)((a.N + BN / 2 - 1) / (BN / 2));
    const Tail tail = HALF && !by_k ? tail_of(all_units, lone, cols * parts, quarter_cols * parts, G) : Tail{0, false};
    const int cut = tail.cut, units = all_units - cut, halves = 2 * cut + lone;        // rows of tiles
    const int tail_cols = tail.quarters ? quarter_cols : cols;

    auto in_part = [&](int t, int rows, int columns, int& tm, Where& w) {   // tile t of rows x columns for each part
        const int per = rows * columns, part = t / per;
        tile_of(t - part * per, rows, columns, tm, w.tn);
        if constexpr (KS) {
            if (by_k) {
                const int g = uniform(s_groups.order[part]);
                w.g = g;
                w.k_first = g ? uniform(s_groups.end[g - 1]) : 0;
                w.K = uniform(s_groups.end[g]) - w.k_first;
                return;
            }
        }
        w.split = part;
    };
    auto in_group = [&](int g, Where& w) {
        if constexpr (ROWS) {
            w.g = g;
            w.grow0 = g ? uniform(s_groups.end[g - 1]) : 0;
            w.M = uniform(s_groups.end[g]) - w.grow0;
            w.zero = g == a.E;
            if (w.zero)
                w.K = 0;
        }
    };
    auto unit_of = [&](int g) { return ROWS ? ((const Groups&)s_groups).big[g] + ((const Groups&)s_groups).half[g] / 2 : 0; };
    auto group_half = [&](int q, Where& w) {                           // the groups' half number q
        if constexpr (ROWS) {
            const int g = group_of(a.E, q, [&](int e) { return s_groups.half[e]; });
            in_group(g, w);
            w.m0 = (int64_t)(uniform(s_groups.big[g + 1]) - uniform(s_groups.big[g])) * BM;
        }
    };

    const int tiles = units * cols * parts, last = tiles % G, idle = last ? G - last : 0;
    int p = vid >= last ? vid - last : vid - last + G;
    const int tail_tiles = halves * tail_cols * parts;
    if (last == 0 && tail_tiles < G && G % 8 == 0) {
        // few tiles and no more: an eighth for each XCD, not all for the first ones
        const int each_xcd = (tail_tiles + 7) / 8, y = blockIdx.x / 8;
        p = y < each_xcd ? (int)(blockIdx.x % 8) * each_xcd + y : tail_tiles;
    }
    bool whole = true;                                                 // units, then halves
    for (int i = 0;; ++i) {
        Where w = {0, 0, a.M, a.K, 0, 0, 0, 0, 0, false};
        int two = -1;                                                  // first of a unit's two halves
        bool full = false;
        if (whole) {
            // groups that split the reduction come by size: a workgroup that had the first of a round has the
            // last of the next
            const int t = i * G + (by_k && (i & 1) ? G - 1 - vid : vid);
            if (i * G >= tiles) {
                if (!HALF)
                    break;
                whole = false;
                i = -1;
                continue;
            }
            if (t >= tiles)
                continue;
            int tm = 0;
            full = true;
            if (by_rows) {
                if constexpr (ROWS) {
                    const int g = group_of(a.E, t / cols, unit_of), u0 = uniform(unit_of(g));
                    const int big = min(uniform(s_groups.big[g + 1]) - uniform(s_groups.big[g]), units - u0);
                    const int in = t - u0 * cols;
                    full = !HALF || in < big * cols;
                    if (full) {
                        tile_of(in, big, cols, tm, w.tn);
                        in_group(g, w);
                    } else {
                        w.tn = in - big * cols;
                        two = uniform(s_groups.half[g]) - 1;
                    }
                }
            } else {
                in_part(t, units, cols, tm, w);
            }
            w.m0 = (int64_t)tm * BM;
        } else {
            // the workgroups that the last round left without a unit take two of the halves, or three quarters, first
            const int ahead = tail.quarters ? 3 : 2;
            int h = ahead * idle + p + (i - ahead) * G;
            if (i < ahead) {
                if (p >= idle)
                    continue;
                h = p + i * idle;
            }
            if (h >= tail_tiles)
                break;
            int hr = 0;
            if (by_rows) {
                if constexpr (ROWS) {
                    hr = h / tail_cols;
                    w.tn = h - hr * tail_cols;
                    if (hr == 2 * cut) {
                        group_half(nh - 1, w);
                    } else {
                        const int u = units + hr / 2, g = group_of(a.E, u, unit_of), in = u - uniform(unit_of(g));
                        if (in < uniform(s_groups.big[g + 1]) - uniform(s_groups.big[g])) {
                            in_group(g, w);
                            w.m0 = (int64_t)in * BM + (hr & 1) * (BM / 2);
                        } else {
                            group_half(uniform(s_groups.half[g]) - 1 + (hr & 1), w);
                        }
                    }
                }
            } else {
                in_part(h, halves, tail_cols, hr, w);
                w.m0 = (int64_t)units * BM + (int64_t)hr * (BM / 2);
            }
        }
        const bool quarter = !whole && tail.quarters;
        w.n0 = (int64_t)w.tn * (quarter ? BN / 2 : BN);
        if (full) {
            product_tile<BM, BN, WM, WN, S, TA, TB, EPI>(a, l, w);
        } else if constexpr (HALF) {
            if (quarter) {
                product_tile<BM / 2, BN / 2, WM, WN, 4, TA, TB, EPI>(a, lq, w);
                continue;
            }
            for (int q = 0; q < 2; ++q) {
                if (two >= 0)
                    group_half(two + q, w);
                product_tile<BM / 2, BN, WM, WN, 3, TA, TB, EPI>(a, lh, w);
                if (two < 0)
                    break;
            }
        }
    }
}

}  // namespace lm
}  // namespace ag
