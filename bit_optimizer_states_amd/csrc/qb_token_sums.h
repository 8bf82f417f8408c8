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

// One column of the joined sums of an id whose tokens are order[first .. last):
// a lane adds one binary32 per chunk, so that many waves share a row, 16 loads in flight.
__device__ __forceinline__ float join_column(const float* part, int32_t chunk, int32_t first, int32_t last,
                                             int64_t padded, int64_t col)
{
    constexpr int UN = 16;
    const int32_t c1 = (last - 1) / chunk;
    int32_t c = first / chunk;
    float sum = gld<float>(part + chunk_slot(c, first, chunk) * padded + col);
    ++c;
    const float* p = part + 2 * (int64_t)c * padded + col;         // later chunks begin with this id's tokens
    for (; c <= c1; c += UN, p += 2 * UN * padded) {
        float v[UN];
#pragma unroll
        for (int q = 0; q < UN; ++q) v[q] = gld<float>(p + 2 * (int64_t)(c + q <= c1 ? q : c1 - c) * padded);
#pragma unroll
        for (int q = 0; q < UN; ++q)
            if (c + q <= c1) sum += v[q];
    }
    return sum;
}

__device__ __forceinline__ int64_t slot_of(int64_t v, const OrderArgs& o)
{
    return (v & ((int64_t(1) << o.log2g) - 1)) * o.per + (v >> o.log2g);
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
