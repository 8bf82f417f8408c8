// qb_token_sums.h -- sums of a gradient's rows over the tokens of one id, in the
// order that k_order made (shared by the gradients of the plain and of the
// stable embedding).
#pragma once
#include "qb_rows.h"

namespace qb {

// sum[k] += dy of the units k * TPR + tid over the R tokens whose positions lanes
// i .. i + R - 1 hold, in order; the loads of all R rows are in flight together.
template <int GDT, bool TAIL, int TPR, int VPT, int R>
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
template <int GDT, bool TAIL, int TPR, int VPT, int UN>
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

}  // namespace qb
