// qb_norm_kernels.h -- layer norm of rows held in registers, from a dense
// matrix or straight from the rows of an embedding table.
//
// Mathematics (page "Py之bitsandbytes", section 1, lists the stable embedding
// layer, an embedding followed by layer norm, next to the 8-bit optimizers):
//   mean = sum x / dim,  var = sum (x - mean)^2 / dim,  rstd = 1/sqrt(var + eps),
//   y = (x - mean) * rstd * gamma + beta.
// The statistics take two passes over the registers that hold the row: the
// sum, then the sums of d = x - mean and of d^2, from which the mean is
// corrected by the residue of its own rounding, m = sum d / dim (var = sum d^2
// / dim - m^2).  A row whose mean is large against its spread keeps its digits,
// which sum x^2 - (sum x)^2 would cancel.  All sums are binary32.
//
// One read and one write of every row: the kernel is bound by HBM.
#pragma once
#include "qb_rows.h"

namespace qb {

// Sum over the TPR threads that share a row: within a wave by DPP, over the
// row's waves through LDS (slot: TPR / 64 words that no other sum uses before
// the next-but-one barrier).
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float* slot)
{
    if constexpr (TPR <= 64) {
        return lanes_sum<TPR>(v);
    } else {
        constexpr int W = TPR / 64;
        v = lanes_sum<64>(v);
        const int w = (threadIdx.x % TPR) / 64;
        if (threadIdx.x % 64 == 0) slot[w] = v;
        lds_barrier();
        float s[W];
#pragma unroll
        for (int i = 0; i < W; ++i) s[i] = slot[i];
#pragma unroll
        for (int h = W / 2; h > 0; h /= 2)
#pragma unroll
            for (int i = 0; i < h; ++i) s[i] += s[i + h];
        return s[0];
    }
}

// Two sums with one barrier.
template <int TPR>
__device__ __forceinline__ void row_sum2(float& a, float& b, float* slot)
{
    if constexpr (TPR <= 64) {
        a = lanes_sum<TPR>(a);
        b = lanes_sum<TPR>(b);
    } else {
        constexpr int W = TPR / 64;
        a = lanes_sum<64>(a);
        b = lanes_sum<64>(b);
        const int w = (threadIdx.x % TPR) / 64;
        if (threadIdx.x % 64 == 0) {
            slot[2 * w] = a;
            slot[2 * w + 1] = b;
        }
        lds_barrier();
        float s[W], t[W];
#pragma unroll
        for (int i = 0; i < W; ++i) {
            s[i] = slot[2 * i];
            t[i] = slot[2 * i + 1];
        }
#pragma unroll
        for (int h = W / 2; h > 0; h /= 2)
#pragma unroll
            for (int i = 0; i < h; ++i) {
                s[i] += s[i + h];
                t[i] += t[i + h];
            }
        a = s[0];
        b = t[0];
    }
}

constexpr int row_slot_words(int tpr) { return tpr <= 64 ? 1 : 3 * (tpr / 64); }

// 1/sqrt(var + eps); a variance that rounding took below zero is zero, a NaN stays one.
__device__ __forceinline__ float inv_deviation(float var, float eps)
{
    return 1.0f / __builtin_sqrtf((var < 0.0f ? 0.0f : var) + eps);
}

// Mean and 1/sqrt(var + eps) of a row of `dim` elements spread over TPR
// threads, unit k * TPR + lane in x[k] (zeros beyond the row).
template <int TPR, int VPT>
__device__ __forceinline__ void row_stats(const float (&x)[VPT][8], int lane, int dim, float eps, float* slot,
                                          float* mean, float* rstd)
{
    float s = 0.0f;
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
        const float a = (x[k][0] + x[k][1]) + (x[k][2] + x[k][3]);
        const float b = (x[k][4] + x[k][5]) + (x[k][6] + x[k][7]);
        s += a + b;
    }
    const float m0 = row_sum<TPR>(s, slot) / (float)dim;
    float sd = 0.0f, sq = 0.0f;
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
        const int cnt = unit_count(k * TPR + lane, dim);
        float ud = 0.0f, uq = 0.0f;
        if (cnt == 8) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float d = x[k][j] - m0;
                ud += d;
                uq = __builtin_fmaf(d, d, uq);
            }
        } else {
#pragma unroll
            for (int j = 0; j < 7; ++j) {
                const float d = j < cnt ? x[k][j] - m0 : 0.0f;
                ud += d;
                uq = __builtin_fmaf(d, d, uq);
            }
        }
        sd += ud;
        sq += uq;
    }
    row_sum2<TPR>(sd, sq, slot + (TPR <= 64 ? 0 : TPR / 64));
    const float c = sd / (float)dim;
    *mean = m0 + c;
    *rstd = inv_deviation(sq / (float)dim - c * c, eps);
}

// One row per TPR threads, 256 threads a workgroup.  GATHER: row t is scale *
// table[ids[t]] (zeros out where the id is outside the table).
template <int XDT, int YDT, int WDT, int TPR, int VPT, bool TAIL, bool GATHER>
__global__ __launch_bounds__(256) void k_norm(const void* __restrict__ x, IdArgs a, float scale,
                                              const void* __restrict__ gamma, const void* __restrict__ beta, float eps,
                                              void* __restrict__ y, float* __restrict__ mean_out,
                                              float* __restrict__ rstd_out)
{
    constexpr int RPB = 256 / TPR;
    // gamma and beta are read with the row where registers allow, else after the statistics
    constexpr bool EARLY = VPT <= 2;
    __shared__ float s_slot[RPB][row_slot_words(TPR)];
    const int lane = threadIdx.x % TPR, grp = threadIdx.x / TPR;
    const int64_t t = (int64_t)blockIdx.x * RPB + grp;
    const int dim = a.dim, units = (dim + 7) >> 3;
    bool live = t < a.n;
    if constexpr (TPR >= 64) {
        if (!live) return;             // a whole wave, or the whole workgroup where its waves meet at barriers
    }
    char* const yrow = static_cast<char*>(y) + t * dim * elem_bytes(YDT);
    const char* xrow = nullptr;
    bool found = live;
    if constexpr (GATHER) {
        const int64_t id = live ? load_id(a.ids, a.id64, t) : -1;
        found = (uint64_t)id < (uint64_t)a.rows;
        if (found) xrow = static_cast<const char*>(x) + id * dim * elem_bytes(XDT);
    } else {
        if (found) xrow = static_cast<const char*>(x) + t * dim * elem_bytes(XDT);
    }

    float v[VPT][8];
    Unit<WDT> gu[VPT], bu[VPT];
    {
        Unit<XDT> xu[VPT];
        if (found) {
#pragma unroll
            for (int k = 0; k < VPT; ++k) xu[k] = load_row_unit<XDT, TAIL, !GATHER>(xrow, k * TPR + lane, units, dim);
        }
        if constexpr (EARLY) {
            if (gamma) {
#pragma unroll
                for (int k = 0; k < VPT; ++k)
                    gu[k] = load_row_unit<WDT, TAIL, false>(gamma, k * TPR + lane, units, dim);
            }
            if (beta) {
#pragma unroll
                for (int k = 0; k < VPT; ++k)
                    bu[k] = load_row_unit<WDT, TAIL, false>(beta, k * TPR + lane, units, dim);
            }
        }
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            const bool in = found && k * TPR + lane < units;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float w = unit_at<XDT>(xu[k], j);
                v[k][j] = in ? (GATHER ? w * scale : w) : 0.0f;
            }
        }
    }
    float mean, rstd;
    row_stats<TPR, VPT>(v, lane, dim, eps, s_slot[grp], &mean, &rstd);
    if (!live) return;
    if (lane == 0) {
        if (mean_out) mean_out[t] = mean;
        if (rstd_out) rstd_out[t] = rstd;
    }
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
        const int unit = k * TPR + lane;
        if constexpr (!EARLY) {
            if (gamma) gu[k] = load_row_unit<WDT, TAIL, false>(gamma, unit, units, dim);
            if (beta) bu[k] = load_row_unit<WDT, TAIL, false>(beta, unit, units, dim);
        }
        float o[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float g = gamma ? unit_at<WDT>(gu[k], j) : 1.0f;
            const float b = beta ? unit_at<WDT>(bu[k], j) : 0.0f;
            o[j] = __builtin_fmaf((v[k][j] - mean) * rstd, g, b);
            if (GATHER && !found) o[j] = 0.0f;
        }
        store_row_unit<YDT, TAIL, true>(yrow, unit, units, dim, o);
    }
}

// Threads and units per row.  Up to 128 elements 16 lanes share a row, up to
// 2048 one wave (no barrier), beyond that a workgroup.
template <int XDT, int YDT, int WDT, bool TAIL, bool GATHER>
hipError_t norm_as(const void* x, const IdArgs& a, float scale, const NormArgs& w, void* y, float* mean, float* rstd,
                   hipStream_t s)
{
    const int units = (a.dim + 7) / 8;
    auto go = [&](auto kernel, int tpr) {
        return launch_rows(a.n, 256 / tpr, [&](int64_t t0, int64_t m, int grid) {
            const void* const in = GATHER ? x : static_cast<const char*>(x) + t0 * a.dim * elem_bytes(XDT);
            return launch_kernel(kernel, grid, s, in, ids_from(a, t0, m), scale, w.gamma, w.beta, w.eps,
                                 static_cast<char*>(y) + t0 * a.dim * elem_bytes(YDT), mean ? mean + t0 : nullptr,
                                 rstd ? rstd + t0 : nullptr);
        });
    };
    if (units <= 16) return go(k_norm<XDT, YDT, WDT, 16, 1, TAIL, GATHER>, 16);
    if (units <= 64) return go(k_norm<XDT, YDT, WDT, 64, 1, TAIL, GATHER>, 64);
    if (units <= 128) return go(k_norm<XDT, YDT, WDT, 64, 2, TAIL, GATHER>, 64);
    if (units <= 256) return go(k_norm<XDT, YDT, WDT, 64, 4, TAIL, GATHER>, 64);
    if (units <= 512) return go(k_norm<XDT, YDT, WDT, 256, 2, TAIL, GATHER>, 256);
    if (units <= 1024) return go(k_norm<XDT, YDT, WDT, 256, 4, TAIL, GATHER>, 256);
    if (units <= 2048) return go(k_norm<XDT, YDT, WDT, 256, 8, TAIL, GATHER>, 256);
    return hipErrorInvalidValue;
}

template <int XDT, int YDT, int WDT, bool GATHER>
hipError_t norm_dim(const void* x, const IdArgs& a, float scale, const NormArgs& w, void* y, float* mean, float* rstd,
                    hipStream_t s)
{
    return a.dim % 8 ? norm_as<XDT, YDT, WDT, true, GATHER>(x, a, scale, w, y, mean, rstd, s)
                     : norm_as<XDT, YDT, WDT, false, GATHER>(x, a, scale, w, y, mean, rstd, s);
}

}  // namespace qb
