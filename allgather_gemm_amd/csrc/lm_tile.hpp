// lm_tile.hpp -- the tiled matrix product behind the language-model operators (gemm_bias_act,
// gemm_grouped, gemm_xent and their gradients), with what follows the product in its epilogue.
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
#include "ag_protocol.hpp"
#include "lm_internal.hpp"

namespace ag {
namespace lm {

constexpr int NT = 256;        // threads per workgroup
constexpr int BK = 64;         // reduction elements per step
constexpr int GROUP_M = 8;     // tile rows per group of the grouped tile order

__device__ __forceinline__ uint32_t swz(uint32_t row) { return (row & 7u) ^ ((row >> 3) & 1u); }

typedef __attribute__((address_space(3))) bf16x4 lds_bf16x4;

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
    uint32_t op_stride;    // bytes between two loads' first rows
    int32_t klim;          // row operand: this thread's chunk lies inside the row while 128 kb < klim

    __device__ __forceinline__ void init(int tid, int64_t ld, int64_t K)
    {
        const uint32_t ldb = (uint32_t)(ld * 2);
        if (T) {
            const uint32_t k = (uint32_t)(tid * 16) / RB, p = ((uint32_t)(tid * 16) % RB) / 16;
            const uint32_t c = ((p >> 2) ^ ksw(k)) * 4 + (p & 3);
            voff = k * ldb + c * 16;
            klim = 0;
        } else {
            const uint32_t r = tid >> 3, c = (tid & 7) ^ swz(r);
            voff = r * ldb + c * 16;
            klim = (int32_t)(K * 2) - (int32_t)c * 16;
        }
        op_stride = RPO * ldb;
    }

    // Buffer over what step kb of this tile may read: base = first element of the tile at k = 0
    // (row operand: its first row; column operand: row k = 0 at the tile's first column), `rows` the
    // valid tile rows (row operand), K the reduction length, col0 the tile's first column.
    static __device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(const __bf16* base, int64_t ld, int64_t rows,
                                                                  int64_t K, int64_t col0, int64_t kb)
    {
        if (T) {
            const int64_t left = K - kb * BK;
            const int64_t n = left <= 0 ? 0 : (left < BK ? left : (int64_t)BK) * ld * 2 - col0 * 2;
            return make_rsrc(reinterpret_cast<const char*>(base) + (left <= 0 ? 0 : kb * BK * ld * 2), (uint32_t)n);
        }
        const int64_t kbyte = kb * 128;
        const int64_t n = K * 2 <= kbyte ? 0 : ((rows - 1) * ld + K) * 2 - kbyte;
        return make_rsrc(reinterpret_cast<const char*>(base) + (n <= 0 ? 0 : kbyte), (uint32_t)(n <= 0 ? 0 : n));
    }

    // This thread's offset in step kb; past the row's end it starts beyond every buffer size.
    __device__ __forceinline__ uint32_t offset(int64_t kb) const
    {
        if (T)
            return voff;
        return (int32_t)(kb * 128) < klim ? voff : 0x80000000u;
    }

    __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t r, char* stage, uint32_t wave_off, uint32_t off,
                                         uint32_t stride, int q) const
    {
        dma16(r, stage + q * 4096 + wave_off, off + q * stride);
    }
};

// Fragment addressing of one wave: F fragments of 32 rows, the wave's first row w * F * 32.
template <int R, bool T, int F>
struct Frag {
    uint32_t off[4 > F ? 4 : F];

    __device__ __forceinline__ void init(int lane, int w)
    {
        const uint32_t fr = lane & 31, fh = lane >> 5;
        if (T) {
            const uint32_t k = fh * 8 + ((lane & 15) >> 2);
            const uint32_t within = ((lane >> 4) & 1) * 32 + (lane & 3) * 8;
#pragma unroll
            for (int i = 0; i < F; ++i)
                off[i] = k * Side<R, T>::RB + (((uint32_t)(w * F + i)) ^ Side<R, T>::ksw(k)) * 64 + within;
        } else {
            const uint32_t fsw = swz(fr & 15);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
                off[kk] = (uint32_t)(w * F * 32 + fr) * 128 + (((uint32_t)(2 * kk) + fh) ^ fsw) * 16;
        }
    }

    // Fragment i of substep kk: lane l holds row l % 32, k = 16 kk + 8 (l / 32) .. + 7.
    __device__ __forceinline__ bf16x8 read(const char* stage, int kk, int i) const
    {
        if (T) {
            const char* p = stage + off[i] + kk * 16 * Side<R, T>::RB;
            const bf16x4 lo = __builtin_bit_cast(
                bf16x4, __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_bf16x4*)const_cast<char*>(p)));
            const bf16x4 hi = __builtin_bit_cast(
                bf16x4,
                __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_bf16x4*)const_cast<char*>(p + 4 * Side<R, T>::RB)));
            return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
        }
        return *reinterpret_cast<const bf16x8*>(stage + off[kk] + i * 4096);
    }
};

// ------------------------------------------------------------------------------- activations
// Values and slopes in fp32.  exp goes through exp2 (one hardware instruction); its relative error,
// a few 2^-24 times the argument's size, is far below the bf16 rounding of the result.
__device__ __forceinline__ float fast_exp(float x) { return __builtin_amdgcn_exp2f(x * 1.4426950408889634f); }
__device__ __forceinline__ float fast_sigmoid(float x) { return __builtin_amdgcn_rcpf(1.0f + fast_exp(-x)); }

__device__ __forceinline__ float act_value(float x, int act)
{
    switch (act) {
    case kActRelu: return x > 0.0f ? x : (x != x ? x : 0.0f);
    case kActSilu: return x * fast_sigmoid(x);
    case kActGelu: return 0.5f * x * (1.0f + erff(x * 0.70710678118654752f));
    // 0.5 (1 + tanh u) = sigmoid(2u)
    case kActGeluTanh: return x * fast_sigmoid(1.5957691216057308f * (x + 0.044715f * x * x * x));
    default: return x;
    }
}

__device__ __forceinline__ float act_slope(float x, int act)
{
    switch (act) {
    case kActRelu: return x > 0.0f ? 1.0f : 0.0f;
    case kActSilu: {
        const float s = fast_sigmoid(x);
        return s * (1.0f + x * (1.0f - s));
    }
    case kActGelu:
        return 0.5f * (1.0f + erff(x * 0.70710678118654752f)) + x * 0.3989422804014327f * fast_exp(-0.5f * x * x);
    case kActGeluTanh: {
        if (fabsf(x) > 30.0f)              // s is 0 or 1 there; x^2 could overflow and meet its zero
            return x > 0.0f ? 1.0f : 0.0f;
        const float s = fast_sigmoid(1.5957691216057308f * (x + 0.044715f * x * x * x));
        return s + x * s * (1.0f - s) * 1.5957691216057308f * (1.0f + 0.134145f * x * x);
    }
    default: return 1.0f;
    }
}

// Eight consecutive bf16 of row `row`, columns [col, col + 8) with `n` of them valid.
__device__ __forceinline__ void load8(const __bf16* p, int n, bool vec, float* x)
{
    if (vec && n >= 8) {
        const bf16x8 v = *reinterpret_cast<const bf16x8*>(p);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            x[e] = (float)v[e];
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            x[e] = e < n ? (float)p[e] : 0.0f;
    }
}

__device__ __forceinline__ void store8(__bf16* p, int n, bool vec, const float* x)
{
    bf16x8 o;
#pragma unroll
    for (int e = 0; e < 8; ++e)
        o[e] = (__bf16)x[e];
    if (vec && n >= 8) {
        __builtin_nontemporal_store(o, reinterpret_cast<bf16x8*>(p));
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e < n)
                p[e] = o[e];
    }
}

// act(x + bias) + residual of eight columns, stored; `pre` gets x + bias.
__device__ __forceinline__ void linear8(const LinearOut& o, int64_t row, int64_t col, int n, bool vec, float* x)
{
    if (o.bias) {
        float b[8];
        load8(o.bias + col, n, vec, b);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            x[e] += b[e];
    }
    const int64_t at = row * o.ldc + col;
    if (o.pre)
        store8(o.pre + at, n, vec, x);
    if (o.act != kActNone) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            x[e] = act_value(x[e], o.act);
    }
    if (o.residual) {
        float r[8];
        load8(o.residual + at, n, vec, r);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            x[e] += r[e];
    }
    store8(o.C + at, n, vec, x);
}

// ------------------------------------------------------------------------------------- groups
// Ends of the groups as the kernel uses them: s_end[e] is the running maximum of ends[0..e] within
// [0, limit], so groups from any table stay inside the tensors, and s_end[E] = limit closes a last
// group of rows that belong to none.  s_tile[e] is the first of group e's tile rows of bm rows,
// s_tile[E + 1] their number.  Wave 0 scans, 64 lanes over E + 1 entries; ends with a barrier.
__device__ void group_scan(const int32_t* ends, int E, int64_t limit, int bm, int32_t* s_end, int32_t* s_tile)
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
        int prev = before, tiles = 0;
        for (int e = e0; e < e1; ++e) {
            const int end = max(prev, e < E ? min(ends[e], lim) : lim);
            s_end[e] = end;
            tiles += (end - prev + bm - 1) / bm;
            prev = end;
        }
        int first = tiles;
        for (int s = 1; s < 64; s <<= 1) {
            const int o = __shfl_up(first, s);
            if (lane >= s)
                first += o;
        }
        first -= tiles;
        prev = before;
        for (int e = e0; e < e1; ++e) {
            s_tile[e] = first;
            const int end = s_end[e];
            first += (end - prev + bm - 1) / bm;
            prev = end;
        }
        if (e1 == E + 1 && e0 < e1)
            s_tile[E + 1] = first;
    }
    barrier_after_lds_write();
}

// ---------------------------------------------------------------------------------- the kernel
// EPI: kEpiLinear, kEpiStat (softmax statistics of a row's columns), kEpiGrad (d logits).
template <int BM, int BN, int WM, int WN, int S, bool TA, bool TB, int EPI>
__device__ __forceinline__ void tile_body(const TileArgs& a)
{
    static_assert(WM * WN == 4 && (S == 2 || S == 4), "four waves; two or four stages");
    constexpr int FM = BM / WM / 32, FN = BN / WN / 32, NM = FM * FN;
    typedef Side<BM, TA> SA;
    typedef Side<BN, TB> SB;
    constexpr int ND = SA::OPS + SB::OPS;
    constexpr int WNC = FN * 32;                       // columns of a wave's block

    // one array per stage and operand: the compiler then sees that the loads in flight fill another
    // stage than the one being read, and does not wait for them
    __shared__ __attribute__((aligned(1024))) char sA0[SA::BYTES];
    __shared__ __attribute__((aligned(1024))) char sB0[SB::BYTES];
    __shared__ __attribute__((aligned(1024))) char sA1[SA::BYTES];
    __shared__ __attribute__((aligned(1024))) char sB1[SB::BYTES];
    __shared__ __attribute__((aligned(1024))) char sA2[S > 2 ? SA::BYTES : 16];
    __shared__ __attribute__((aligned(1024))) char sB2[S > 2 ? SB::BYTES : 16];
    __shared__ __attribute__((aligned(1024))) char sA3[S > 2 ? SA::BYTES : 16];
    __shared__ __attribute__((aligned(1024))) char sB3[S > 2 ? SB::BYTES : 16];
    __shared__ int32_t s_end[EPI == kEpiLinear ? kMaxGroups + 2 : 1];    // clamped ends of the groups, and M
    __shared__ int32_t s_tile[EPI == kEpiLinear ? kMaxGroups + 2 : 1];   // first tile row of each group

    const int tid = threadIdx.x;
    const int lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / WN, wn = wave % WN;
    const int G = gridDim.x;
    // workgroups are dispatched round-robin over the 8 XCDs: each XCD takes a contiguous run of tiles
    const int vid = (G % 8 == 0) ? (int)(blockIdx.x % 8) * (G / 8) + (int)(blockIdx.x / 8) : (int)blockIdx.x;

    int64_t tile_rows = a.tiles_m;
    if (EPI == kEpiLinear && a.group != kGroupNone) {
        group_scan(a.ends, a.E, a.group == kGroupRows ? a.M : a.K, BM, s_end, s_tile);
        if (a.group == kGroupRows)
            tile_rows = __builtin_amdgcn_readfirstlane(s_tile[a.E + 1]);
    }
    const int64_t num_tiles = tile_rows * a.tiles_n * (a.group == kGroupK ? a.E : 1) * a.splits;

    SA sa;
    SB sb;
    Frag<BM, TA, FM> fa;
    Frag<BN, TB, FN> fb;
    fa.init(lane, wm);
    fb.init(lane, wn);
    const uint32_t wave_off = wave * 1024;

    for (int64_t t = vid; t < num_tiles; t += G) {
        // ---- which tile
        int64_t tm, tn, split = 0, g = 0, grow0 = 0, M = a.M, K = a.K, k_first = 0;
        bool zero = false;
        if (EPI == kEpiLinear && a.group == kGroupRows) {
            const int64_t tr = t / a.tiles_n;            // tile rows of one group lie together
            int lo = 0, hi = a.E + 1;
            while (hi - lo > 1) {                        // last group whose first tile row is <= tr
                const int mid = (lo + hi) >> 1;
                if (__builtin_amdgcn_readfirstlane(s_tile[mid]) <= tr)
                    lo = mid;
                else
                    hi = mid;
            }
            g = lo;
            const int64_t first = __builtin_amdgcn_readfirstlane(s_tile[lo]);
            const int64_t rows_here = __builtin_amdgcn_readfirstlane(s_tile[lo + 1]) - first;
            pm_tile_of(t - first * a.tiles_n, rows_here, a.tiles_n, 0, GROUP_M, tm, tn);
            grow0 = lo == 0 ? 0 : __builtin_amdgcn_readfirstlane(s_end[lo - 1]);
            M = __builtin_amdgcn_readfirstlane(s_end[lo]) - grow0;
            zero = lo == a.E;                            // rows past the last group
            if (zero)
                K = 0;
        } else {
            int64_t u = t;
            if (EPI == kEpiLinear) {
                const int64_t per = a.tiles_m * a.tiles_n;
                if (a.group == kGroupK) {
                    g = u / per;
                    u -= g * per;
                    k_first = g == 0 ? 0 : __builtin_amdgcn_readfirstlane(s_end[g - 1]);
                    K = __builtin_amdgcn_readfirstlane(s_end[g]) - k_first;
                } else {
                    split = u / per;
                    u -= split * per;
                }
            }
            pm_tile_of(u, a.tiles_m, a.tiles_n, 0, GROUP_M, tm, tn);
        }
        const int64_t m0 = tm * BM, n0 = tn * BN;
        const int64_t a_rows = min((int64_t)BM, M - m0), b_rows = min((int64_t)BN, a.N - n0);
        const __bf16* Ab;
        const __bf16* Bb;
        if (TA)
            Ab = a.A + k_first * a.lda + m0;
        else
            Ab = a.A + (grow0 + m0) * a.lda;
        if (TB)
            Bb = a.B + (a.group == kGroupK ? k_first * a.ldb : (zero ? 0 : g) * a.strideB) + n0;
        else
            Bb = a.B + (zero ? 0 : g) * a.strideB + n0 * a.ldb;
        sa.init(tid, a.lda, K);
        sb.init(tid, a.ldb, K);
        const int64_t nk_all = (K + BK - 1) / BK;
        const int64_t kb0 = min(split * a.split_steps, nk_all);
        const int64_t kb1 = a.splits > 1 ? min(kb0 + a.split_steps, nk_all) : nk_all;

        f32x16 acc[FM][FN];
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int j = 0; j < FN; ++j)
#pragma unroll
                for (int v = 0; v < 16; ++v)
                    acc[i][j][v] = 0.0f;

        struct Dma {
            __amdgpu_buffer_rsrc_t ra, rb;
            uint32_t va, vb, lw, sa_, sb_;
            char *la, *lb;
        };
        // loads of step kb into a stage; past the last step they read nothing but still count
        auto dma_setup = [&](int64_t kb, char* la, char* lb) {
            Dma d;
            d.lw = wave_off;
            d.sa_ = sa.op_stride;
            d.sb_ = sb.op_stride;
            asm volatile("" : "+s"(d.lw), "+s"(d.sa_), "+s"(d.sb_));
            const int64_t Kd = kb < kb1 ? K : 0;
            d.ra = SA::rsrc(Ab, a.lda, a_rows, Kd, m0, kb);
            d.rb = SB::rsrc(Bb, a.ldb, b_rows, !TA && TB ? min(Kd, a.k_valid) : Kd, n0, kb);
            d.va = sa.offset(kb);
            d.vb = sb.offset(kb);
            d.la = la;
            d.lb = lb;
            return d;
        };
        auto dma_op = [&](const Dma& d, int q) {
            if (q < SA::OPS)
                sa.load(d.ra, d.la, d.lw, d.va, d.sa_, q);
            else
                sb.load(d.rb, d.lb, d.lw, d.vb, d.sb_, q - SA::OPS);
        };
        auto issue_all = [&](int64_t kb, char* la, char* lb) {
            const Dma d = dma_setup(kb, la, lb);
#pragma unroll
            for (int q = 0; q < ND; ++q)
                dma_op(d, q);
        };
        // One K step: four substeps of NM MFMAs.  The next stage's loads go out spread over the first
        // two substeps, the next substep's fragments are read in between, so neither queue backs up
        // into the matrix instructions.
        auto compute = [&](const char* la, const char* lb, const Dma& d) {
            bf16x8 af[2][FM], bf[2][FN];
#pragma unroll
            for (int j = 0; j < FN; ++j)
                bf[0][j] = fb.read(lb, 0, j);
#pragma unroll
            for (int i = 0; i < FM; ++i)
                af[0][i] = fa.read(la, 0, i);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
                const int cur = kk & 1, nxt = cur ^ 1;
#pragma unroll
                for (int gidx = 0; gidx < NM; ++gidx) {
                    const int i = gidx / FN, j = gidx % FN;
                    acc[i][j] =
                        __builtin_amdgcn_mfma_f32_32x32x16_bf16(bf[cur][j], af[cur][i], acc[i][j], 0, 0, 0);
                    __builtin_amdgcn_sched_barrier(0);
                    if (kk < 2) {
                        const int s0 = kk * NM + gidx;
#pragma unroll
                        for (int q = s0 * ND / (2 * NM); q < (s0 + 1) * ND / (2 * NM); ++q)
                            dma_op(d, q);
                    }
                    if (kk < 3) {
                        constexpr int NR = FM + FN;
#pragma unroll
                        for (int r = (gidx * NR + NM - 1) / NM; r < ((gidx + 1) * NR + NM - 1) / NM; ++r) {
                            if (r < FN)
                                bf[nxt][r] = fb.read(lb, kk + 1, r);
                            else
                                af[nxt][r - FN] = fa.read(la, kk + 1, r - FN);
                        }
                    }
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
        };

        if constexpr (S == 2) {
            // double buffer; with an odd number of steps the first runs alone out of stage 1, so the
            // pair loop always computes twice per iteration
            int64_t kb = kb0;
            if ((kb1 - kb0) & 1) {
                issue_all(kb, sA1, sB1);
                wait_vmcnt0();
                __syncthreads();
                compute(sA1, sB1, dma_setup(kb + 1, sA0, sB0));
                ++kb;
            } else if (kb1 > kb0) {
                issue_all(kb, sA0, sB0);
            }
            for (; kb < kb1; kb += 2) {
                wait_vmcnt0();
                __syncthreads();
                compute(sA0, sB0, dma_setup(kb + 1, sA1, sB1));
                wait_vmcnt0();
                __syncthreads();
                compute(sA1, sB1, dma_setup(kb + 2, sA0, sB0));
            }
        } else {
            // four stages: the loads of three steps are in flight while one is computed
            issue_all(kb0, sA0, sB0);
            issue_all(kb0 + 1, sA1, sB1);
            issue_all(kb0 + 2, sA2, sB2);
            for (int64_t kb = kb0; kb < kb1; kb += 4) {
                wait_vmcnt<2 * ND>();
                __syncthreads();
                compute(sA0, sB0, dma_setup(kb + 3, sA3, sB3));
                if (kb + 1 < kb1) {
                    wait_vmcnt<2 * ND>();
                    __syncthreads();
                    compute(sA1, sB1, dma_setup(kb + 4, sA0, sB0));
                }
                if (kb + 2 < kb1) {
                    wait_vmcnt<2 * ND>();
                    __syncthreads();
                    compute(sA2, sB2, dma_setup(kb + 5, sA1, sB1));
                }
                if (kb + 3 < kb1) {
                    wait_vmcnt<2 * ND>();
                    __syncthreads();
                    compute(sA3, sB3, dma_setup(kb + 6, sA2, sB2));
                }
            }
        }
        wait_vmcnt0();     // loads past the last step have landed too
        __syncthreads();   // all waves are done with the stages

        // ---- epilogue, one 32-row slab of the wave's block at a time through LDS: the read-back gives
        // each lane eight consecutive columns of a row
        constexpr int SLAB = 32 * WNC * 4;
        static_assert(4 * SLAB <= SB::BYTES || (2 * SLAB <= SA::BYTES && 2 * SLAB <= SB::BYTES), "slabs fit a stage");
        char* slab = 4 * SLAB <= SB::BYTES ? sB0 + wave * SLAB : (wave < 2 ? sA0 : sB0) + (wave & 1) * SLAB;
        constexpr uint32_t SW = WNC / 4 - 1;           // 16-byte units of a slab row, minus one
        constexpr int LPR = WNC / 8;                   // lanes per slab row on the way back
        const uint32_t fr = lane & 31, fh = lane >> 5;
#pragma unroll
        for (int i = 0; i < FM; ++i) {
#pragma unroll
            for (int j = 0; j < FN; ++j)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const uint32_t colb = (j * 32 + q * 8 + fh * 4) * 4;
                    const f32x4 v4 = {acc[i][j][q * 4 + 0], acc[i][j][q * 4 + 1], acc[i][j][q * 4 + 2],
                                      acc[i][j][q * 4 + 3]};
                    *reinterpret_cast<f32x4*>(slab + fr * (WNC * 4) + (colb ^ ((fr & SW) << 4))) = v4;
                }
            __builtin_amdgcn_s_waitcnt(0xC07F);   // lgkmcnt(0): this wave's slab is written
            __builtin_amdgcn_wave_barrier();
#pragma unroll
            for (int it = 0; it < WNC / 16; ++it) {
                const uint32_t pidx = it * 64 + lane;
                const uint32_t r = pidx / LPR, c8 = (pidx % LPR) * 8;
                const f32x4 x0 = *reinterpret_cast<const f32x4*>(slab + r * (WNC * 4) + ((c8 * 4) ^ ((r & SW) << 4)));
                const f32x4 x1 =
                    *reinterpret_cast<const f32x4*>(slab + r * (WNC * 4) + (((c8 + 4) * 4) ^ ((r & SW) << 4)));
                float x[8] = {x0[0], x0[1], x0[2], x0[3], x1[0], x1[1], x1[2], x1[3]};
                const int64_t mrow = m0 + (wm * FM + i) * 32 + r, col = n0 + wn * WNC + c8;
                const int n = (int)max((int64_t)0, min((int64_t)8, a.N - col));
                const bool in = mrow < M && n > 0;
                if constexpr (EPI == kEpiLinear) {
                    if (in) {
                        const int64_t row = grow0 + mrow;
                        if (a.part) {
                            float* p = a.part + (split * a.M + row) * a.ldp + col;   // ldp % 8 == 0: whole vectors
                            f32x4* pv = reinterpret_cast<f32x4*>(p);
                            if (a.accumulate) {
                                const f32x4 o0 = pv[0], o1 = pv[1];
                                pv[0] = f32x4{x[0], x[1], x[2], x[3]} + o0;
                                pv[1] = f32x4{x[4], x[5], x[6], x[7]} + o1;
                            } else {
                                pv[0] = f32x4{x[0], x[1], x[2], x[3]};
                                pv[1] = f32x4{x[4], x[5], x[6], x[7]};
                            }
                        } else {
                            LinearOut o = a.out;
                            if (a.group == kGroupK)
                                o.C += g * a.M * a.out.ldc;
                            linear8(o, row, col, n, a.vec, x);
                        }
                    }
                } else if constexpr (EPI == kEpiStat) {
                    // maximum and sum of exponentials of this row's WNC columns: LPR neighbouring lanes
                    // hold them, so the steps below stay inside the row
                    float mx = -INFINITY;
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if (e < n)
                            mx = fmaxf(mx, x[e]);
                    bool nan = false;
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        nan |= e < n && x[e] != x[e];
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
                            float* p = a.stat + (mrow * a.stat_n + tn * WN + wn) * 2;
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
                } else {
                    // d logits = dloss (softmax - one at the target), rounded to bf16 for the products that
                    // follow (each is a sum of many such terms; 2^-9 of each term is their input's own
                    // precision); padding columns of the buffer are zero
                    if (mrow < M && col < a.out.ldc) {
                        const int64_t y = a.targets[mrow];
                        const bool has = y >= 0 && y < a.vocab;
                        const float lse = a.lse[mrow], w = has ? a.dloss[mrow] : 0.0f;
                        const int64_t hit = y - a.col0 - col;
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            float p = fast_exp(x[e] - lse);
                            if (hit == e)
                                p -= 1.0f;
                            x[e] = (e < n && has) ? p * w : 0.0f;
                        }
                        bf16x8 o;
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            o[e] = (__bf16)x[e];
                        *reinterpret_cast<bf16x8*>(a.out.C + mrow * a.out.ldc + col) = o;
                    }
                }
            }
            __builtin_amdgcn_s_waitcnt(0xC07F);   // reads done before the slab is rewritten
            __builtin_amdgcn_wave_barrier();
        }
        __syncthreads();   // LDS is free for the next tile's loads
    }
}

}  // namespace lm
}  // namespace ag
