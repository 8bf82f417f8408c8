// qb_token_sums.h -- sums of a gradient's rows over the tokens of one id, in the
// order that k_order made (shared by the gradients of the plain and of the
// stable embedding).
#pragma once
#include "qb_rows.h"

namespace qb {

constexpr int kZeroRows = 16;           // table rows of a zero-filling workgroup

// sum[k] += dy of the units k * TPR + tid over the R tokens whose positions lanes
// i .. i + R - 1 hold, in order; the loads of all R rows are in flight together.
template <int GDT, int TAIL, int TPR, int VPT, int R>
__device__ __forceinline__ void add_tokens(int32_t pos, int32_t i, const void* dy, int tid, int units, int dim,
                                           float (&sum)[VPT][8])
{
    Unit<GDT> u[R][VPT];
#pragma unroll
    for (int q = 0; q < R; ++q) {
        const int32_t t = __builtin_amdgcn_readlane(pos, i + q);
        const char* const row = static_cast<const char*>(dy) + (int64_t)t * dim * elem_bytes(GDT);
#pragma unroll
        for (int k = 0; k < VPT; ++k) u[q][k] = load_row_unit<GDT, TAIL, true>(row, k * TPR + tid, units, dim);
    }
#pragma unroll
    for (int q = 0; q < R; ++q)
#pragma unroll
        for (int k = 0; k < VPT; ++k)
#pragma unroll
            for (int j = 0; j < 8; ++j) sum[k][j] += unit_at<GDT>(u[q][k], j);
}

// sum[k] += dy of the units k * TPR + tid over the tokens order[first .. last), in
// order.  Wave-uniform first and last: the positions are read 64 at a time, one
// per lane, and handed out by readlane.  Most ids have one to three tokens:
// each remainder has its own straight code, since a wave that reads a row it
// does not need waits as long as for one that it does.
template <int GDT, int TAIL, int TPR, int VPT, int UN>
__device__ __forceinline__ void sum_tokens(const int32_t* order, int32_t first, int32_t last, const void* dy, int tid,
                                           int units, int dim, float (&sum)[VPT][8])
{
    static_assert(UN == 4 || UN == 8, "remainders up to 7");
    const int lane = threadIdx.x % 64;
    for (int32_t b = first; b < last; b += 64) {
        const int32_t m = last - b < 64 ? last - b : 64;
        const int32_t pos = lane < m ? gld<int32_t>(order + b + lane) : 0;
        int32_t i = 0;
        for (; i + UN <= m; i += UN) add_tokens<GDT, TAIL, TPR, VPT, UN>(pos, i, dy, tid, units, dim, sum);
        if constexpr (UN == 8) {
            if (m - i >= 4) {
                add_tokens<GDT, TAIL, TPR, VPT, 4>(pos, i, dy, tid, units, dim, sum);
                i += 4;
            }
        }
        if (m - i == 1) add_tokens<GDT, TAIL, TPR, VPT, 1>(pos, i, dy, tid, units, dim, sum);
        else if (m - i == 2) add_tokens<GDT, TAIL, TPR, VPT, 2>(pos, i, dy, tid, units, dim, sum);
        else if (m - i == 3) add_tokens<GDT, TAIL, TPR, VPT, 3>(pos, i, dy, tid, units, dim, sum);
    }
}

// Row of the chunks' sums that holds chunk c's share of an id whose tokens begin at `first`.
__device__ __forceinline__ int64_t chunk_slot(int32_t c, int32_t first, int32_t chunk)
{
    return 2 * (int64_t)c + (first > c * chunk ? 1 : 0);
}

__device__ __forceinline__ int64_t slot_of(int64_t v, const OrderArgs& o)
{
    return (v & ((int64_t(1) << o.log2g) - 1)) * o.per + (v >> o.log2g);
}

// One column of the sum of an id's chunks c .. end - 1 (its tokens begin at `first`):
// a lane adds one binary32 per chunk, kJoinLoads in flight.
constexpr int kJoinWaves = 4, kJoinLoads = 16, kJoinAlone = 64;

__device__ __forceinline__ float sum_column(const float* part, int32_t chunk, int32_t first, int32_t c, int32_t end,
                                            int64_t padded, int64_t col)
{
    float sum = 0.0f;
    for (; c < end; c += kJoinLoads) {
        float v[kJoinLoads];
#pragma unroll
        for (int q = 0; q < kJoinLoads; ++q)
            v[q] = gld<float>(part + chunk_slot(c + q < end ? c + q : end - 1, first, chunk) * padded + col);
#pragma unroll
        for (int q = 0; q < kJoinLoads; ++q)
            if (c + q < end) sum += v[q];
    }
    return sum;
}

// The joined sums of all long ids, done(id, first, col, sum) once for each of their
// `padded` columns.  A wave takes 64 columns of an id; an id of more than kJoinAlone
// chunks (padding, a batch of one token) is left to all waves of the workgroup, which
// share its chunks evenly and add their sums in order (16384 tokens of one id, rows of
// 4096: 104 us for the whole gradient against 127 by single waves; with every id shared
// that way 16384 tokens of natural frequencies took 98 us against 93).
template <class Done>
__device__ __forceinline__ void join_long_ids(const OrderArgs& o, const float* part, int64_t padded, Done done)
{
    __shared__ float s_sum[kJoinWaves][64];
    __shared__ int64_t s_shared[kJoinWaves];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), lane = threadIdx.x % 64;
    const int64_t groups = (padded + 63) / 64, tasks = (int64_t)o.count[1] * groups;
    // neighbouring columns to the waves of one workgroup, unless that left workgroups without
    // any (natural frequencies: 93.4 against 94.1 us for the whole gradient)
    const bool near = tasks >= gridDim.x;
    const int64_t at = near ? (int64_t)blockIdx.x * kJoinWaves + wave : blockIdx.x + (int64_t)wave * gridDim.x;
    for (int64_t w0 = 0; w0 < tasks; w0 += (int64_t)gridDim.x * kJoinWaves) {
        const int64_t w = w0 + at;
        int64_t shared = -1;
        if (w < tasks) {
            const int64_t v = o.longs[w / groups], s = slot_of(v, o), col = w % groups * 64 + lane;
            const int32_t first = o.start[s], c0 = first / o.chunk, c1 = (o.start[s + 1] - 1) / o.chunk + 1;
            if (c1 - c0 > kJoinAlone) shared = w;
            else if (col < padded) done(v, first, col, sum_column(part, o.chunk, first, c0, c1, padded, col));
        }
        if (lane == 0) s_shared[wave] = shared;
        __syncthreads();
        for (int q = 0; q < kJoinWaves; ++q) {
            const int64_t wq = s_shared[q];
            if (wq < 0) continue;                      // (the same for all threads)
            const int64_t v = o.longs[wq / groups], s = slot_of(v, o), col = wq % groups * 64 + lane;
            const int32_t first = o.start[s], c0 = first / o.chunk, c1 = (o.start[s + 1] - 1) / o.chunk + 1;
            const int32_t per = (c1 - c0 + kJoinWaves - 1) / kJoinWaves, begin = c0 + wave * per;
            const int32_t end = begin + per < c1 ? begin + per : c1;
            s_sum[wave][lane] =
                col < padded ? sum_column(part, o.chunk, first, begin, end, padded, col) : 0.0f;
            __syncthreads();
            if (wave == 0 && col < padded) {
                float sum = s_sum[0][lane];
#pragma unroll
                for (int r = 1; r < kJoinWaves; ++r) sum += s_sum[r][lane];
                done(v, first, col, sum);
            }
            __syncthreads();
        }
        __syncthreads();                               // s_shared is written anew
    }
}

// ---------------------------------------------------------------------------
// few tokens: no ordering
// ---------------------------------------------------------------------------

// The ids of up to kDirectTokens tokens, held by every wave (lane l: tokens l and
// 64 + l); ids outside the table are -1.
struct DirectIds {
    int32_t id[2];

    __device__ __forceinline__ explicit DirectIds(const IdArgs& a)
    {
        const int lane = threadIdx.x % 64;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int t = h * 64 + lane;
            const int64_t v = t < a.n ? load_id(a.ids, a.id64, t) : -1;
            id[h] = (uint64_t)v < (uint64_t)a.rows ? (int32_t)v : -1;
        }
    }

    // id of token t (uniform)
    __device__ __forceinline__ int32_t of(int t) const
    {
        const int32_t a = __builtin_amdgcn_readlane(id[0], t & 63), b = __builtin_amdgcn_readlane(id[1], t & 63);
        return t < 64 ? a : b;
    }

    // tokens of id v
    __device__ __forceinline__ unsigned long long tokens(int h, int32_t v) const { return __ballot(id[h] == v); }
};

// sum[k] += dy of the units k * TPR + tid over the tokens of `mask` (bit l: token
// 64 h + l), in order, UN tokens in flight.
template <int GDT, int TAIL, int TPR, int VPT, int UN>
__device__ __forceinline__ void sum_masked(unsigned long long mask, int h, const void* dy, int tid, int units, int dim,
                                           float (&sum)[VPT][8])
{
    while (mask) {
        Unit<GDT> u[UN][VPT];
        const int m = (int)__popcll(mask);
        unsigned long long rest = mask;
        int t = 0;
#pragma unroll
        for (int q = 0; q < UN; ++q) {
            // (beyond the last token the last one again: no branch, the same lines)
            t = rest ? h * 64 + __builtin_ctzll(rest) : t;
            rest &= rest - 1;
#pragma unroll
            for (int k = 0; k < VPT; ++k)
                u[q][k] = load_row_unit<GDT, TAIL, true>(
                    static_cast<const char*>(dy) + (int64_t)t * dim * elem_bytes(GDT), k * TPR + tid, units, dim);
        }
#pragma unroll
        for (int q = 0; q < UN; ++q)
            if (q < m)
#pragma unroll
                for (int k = 0; k < VPT; ++k)
#pragma unroll
                    for (int j = 0; j < 8; ++j) sum[k][j] += unit_at<GDT>(u[q][k], j);
        mask = rest;
    }
}

// One workgroup of THREADS threads: zeros into the rows of kZeroRows that no
// token names, and into pad's.
template <int TAIL, int THREADS>
__device__ __forceinline__ void zero_unnamed(const IdArgs& a, const DirectIds& ids, int64_t v0, int64_t pad, void* dtable,
                                             int ddt)
{
    const int dim = a.dim, units = (dim + 7) >> 3;
    const float zero[8] = {};
    for (int i = 0; i < kZeroRows && v0 + i < a.rows; ++i) {
        const int64_t v = v0 + i;
        if (v != pad && (ids.tokens(0, (int32_t)v) | ids.tokens(1, (int32_t)v))) continue;
        char* const row = static_cast<char*>(dtable) + v * dim * (ddt == DT_F32 ? 4 : 2);
        for (int unit = threadIdx.x; unit < units; unit += THREADS)
            store_row_unit_rt<TAIL, true>(ddt, row, unit, units, dim, zero);
    }
}

// Workgroups that zero the table in such a launch (0 with accumulate).
inline int64_t direct_zero_wgs(int64_t rows, bool accumulate)
{
    return accumulate ? 0 : (rows + kZeroRows - 1) / kZeroRows;
}

}  // namespace qb
