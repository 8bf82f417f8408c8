// qb_token_sums.h -- sums of a gradient's rows over the tokens of one id, in the
// order that k_order made (shared by the gradients of the plain and of the
// stable embedding).
#pragma once
#include "qb_rows.h"

namespace qb {

// sum[8] += dy of unit `unit` over the tokens order[first .. last), in order.
// Wave-uniform first and last: the positions are read 64 at a time, one per
// lane, and handed out by readlane, so UN rows' loads are in flight together.
template <int GDT, bool TAIL, int UN>
__device__ __forceinline__ void sum_tokens(const int32_t* order, int32_t first, int32_t last, const void* dy, int unit,
                                           int units, int dim, float* sum)
{
    const int lane = threadIdx.x % 64;
    for (int32_t b = first; b < last; b += 64) {
        const int32_t m = last - b < 64 ? last - b : 64;
        const int32_t pos = lane < m ? gld<int32_t>(order + b + lane) : 0;
        for (int32_t i = 0; i < m; i += UN) {
            Unit<GDT> u[UN];
#pragma unroll
            for (int q = 0; q < UN; ++q) {
                const int32_t t = __builtin_amdgcn_readlane(pos, i + q < m ? i + q : m - 1);
                u[q] = load_row_unit<GDT, TAIL, true>(
                    static_cast<const char*>(dy) + (int64_t)t * dim * elem_bytes(GDT), unit, units, dim);
            }
#pragma unroll
            for (int q = 0; q < UN; ++q)
                if (i + q < m)
#pragma unroll
                    for (int j = 0; j < 8; ++j) sum[j] += unit_at<GDT>(u[q], j);
        }
    }
}

// Joins the chunks' sums of an id whose tokens are order[first .. last).
template <int UN>
__device__ __forceinline__ void sum_chunks(const float* part, int32_t chunk, int32_t first, int32_t last, int unit,
                                           int units, int64_t padded, float* sum)
{
    const int32_t c0 = first / chunk, c1 = (last - 1) / chunk;
    const int64_t col = (int64_t)(unit < units ? unit : 0) * 8;
    for (int32_t c = c0; c <= c1; c += UN) {
        f32x4 a[UN], b[UN];
#pragma unroll
        for (int q = 0; q < UN; ++q) {
            const int32_t cc = c + q <= c1 ? c + q : c1;
            const float* p = part + (2 * (int64_t)cc + (first > cc * chunk ? 1 : 0)) * padded + col;
            a[q] = gld<f32x4>(p);
            b[q] = gld<f32x4>(p + 4);
        }
#pragma unroll
        for (int q = 0; q < UN; ++q)
            if (c + q <= c1) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    sum[j] += a[q][j];
                    sum[4 + j] += b[q][j];
                }
            }
    }
}

__device__ __forceinline__ int64_t slot_of(int64_t v, const OrderArgs& o)
{
    return (v & ((int64_t(1) << o.log2g) - 1)) * o.per + (v >> o.log2g);
}

}  // namespace qb
