// qb_norm_kernels.h -- layer norm of rows held in registers, from a dense
// matrix or straight from the rows of an embedding table.
//
// Mathematics (page "Py之bitsandbytes", section 1, lists the stable embedding
// layer, an embedding followed by layer norm, next to the 8-bit optimizers):
//   mean = sum x / dim,  var = sum (x - mean)^2 / dim,  rstd = 1/sqrt(var + eps),
//   y = (x - mean) * rstd * gamma + beta.
// The statistics take two passes over the registers that hold the row, so that
// nothing cancels as sum x^2 - (sum x)^2 would.  All sums are binary32.
//
// One read and one write of every row: the kernel is bound by HBM (16384 rows of
// 4096 bf16 in 47 us, 5.8 TB/s; a copy of the same 268 MB takes 45), with the vector
// ALU close behind: about 265 instructions per wave and row there, active 0.68 of the
// time (42 of them for the correction of 16-bit rows' means and its check, 46.7 -> 47.1
// us); a first version of 550 was bound by them (50 us), so uniform conditions are kept out
// of the lanes and everything that depends on the row's length alone is computed once.  Gathering rows
// of a binary32 table ([32000, 4096], natural frequencies) 52 us: the 90 MB of used rows
// come to 167 MB, since each of the 8 L2s fetches the frequent ones.
#pragma once
#include <cfloat>
#include <type_traits>

#include "qb_rows.h"

namespace qb {

// Two sums over the TPR threads that share a row: within a wave by DPP, then
// over the row's waves through LDS (slot: 2 * TPR / 64 words that no other sum uses
// before the next-but-one barrier), in two parts with a barrier between them.
template <int TPR>
__device__ __forceinline__ void put_sum2(float& a, float& b, float* slot)
{
    constexpr int L = TPR < 64 ? TPR : 64;
    a = lanes_sum<L>(a);
    b = lanes_sum<L>(b);
    if (TPR > 64 && threadIdx.x % 64 == 0) {
        const int w = (threadIdx.x % TPR) / 64;
        slot[2 * w] = a;
        slot[2 * w + 1] = b;
    }
}

template <int TPR>
__device__ __forceinline__ void join_sum2(float& a, float& b, const float* slot)
{
    if constexpr (TPR > 64) {
        // lane l takes wave l % W's sums: two reads and log2 W steps for all of them
        constexpr int W = TPR / 64;
        const int l = threadIdx.x % W;
        a = group_sum<W>(slot[2 * l]);
        b = group_sum<W>(slot[2 * l + 1]);
    }
}

template <int TPR>
__device__ __forceinline__ void row_sum2(float& a, float& b, float* slot)
{
    put_sum2<TPR>(a, b, slot);
    if constexpr (TPR > 64) lds_barrier();
    join_sum2<TPR>(a, b, slot);
}

constexpr int row_slot_words(int tpr) { return tpr <= 64 ? 1 : 3 * (tpr / 64); }

// 1/sqrt(var + eps) by the hardware's reciprocal root (1 ulp); a variance that
// rounding took below zero is zero, a NaN stays one.
__device__ __forceinline__ float inv_deviation(float var, float eps)
{
    return __builtin_amdgcn_rsqf((var < 0.0f ? 0.0f : var) + eps);
}

// What depends on the length of a row alone: the numbers of elements that the
// TPR / 64 waves of a row hold, and reciprocals.
template <int TPR, int VPT>
struct RowShape {
    static constexpr int L = TPR < 64 ? TPR : 64, W = TPR < 64 ? 1 : TPR / 64;
    float held;              // elements of wave (lane % W)
    float inv_mine;          // 1 / elements of this wave (0 where it has none)
    float inv_dim;
    int wave;

    __device__ __forceinline__ RowShape(int lane, int dim)
    {
        wave = W == 1 ? 0 : __builtin_amdgcn_readfirstlane(lane / 64);
        float mine = 0.0f;
        held = 0.0f;
#pragma unroll
        for (int w = 0; w < W; ++w) {
            int n = 0;
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
                const int left = dim - (k * TPR + w * L) * 8;
                n += left < 0 ? 0 : left > L * 8 ? L * 8 : left;
            }
            held = w == lane % W ? (float)n : held;
            mine = w == wave ? (float)n : mine;
        }
        inv_mine = mine > 0.0f ? 1.0f / mine : 0.0f;
        inv_dim = 1.0f / (float)dim;
    }
};

// Whether all TPR lanes' units of step k are whole (uniform).
template <int TPR>
__device__ __forceinline__ bool whole_step(int k, int dim)
{
    return (k + 1) * TPR * 8 <= dim;
}

// Mean and 1/sqrt(var + eps) of a row spread over TPR threads, unit k * TPR +
// lane in x[k] (zeros beyond the row).  Each wave takes the mean and the squared
// deviation of its own elements (wave_stats), which are then joined over the row's
// waves (join_stats, behind one barrier) as those of parts of a sample:
//   mean = sum n_w mean_w / dim,  M2 = sum (M2_w + n_w (mean_w - mean)^2).
// A wave's mean is corrected by the mean of the differences, so that a row whose mean
// is large against its spread keeps its digits: the mean's first rounding would come
// out multiplied by up to 1/sqrt(eps), also in a row of equal 16-bit values (159
// values of 60000 were normalized to 0.78 instead of 0 without it).
struct WaveStats {
    float m0, c, m2;          // mean m0 + c (not rounded to one binary32), squared deviation
};

// Sums over a row's lanes of the differences from m and of their squares.
template <int TPR, int VPT>
__device__ __forceinline__ void deviations(const float (&x)[VPT][8], float m, int lane, int dim, float& sd, float& sq)
{
    constexpr int L = RowShape<TPR, VPT>::L;
    sd = sq = 0.0f;
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
        float ud = 0.0f, uq = 0.0f;
        if (whole_step<TPR>(k, dim)) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float d = x[k][j] - m;
                ud += d;
                uq = __builtin_fmaf(d, d, uq);
            }
        } else {
            const int cnt = unit_count(k * TPR + lane, dim);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float d = j < cnt ? x[k][j] - m : 0.0f;
                ud += d;
                uq = __builtin_fmaf(d, d, uq);
            }
        }
        sd += ud;
        sq += uq;
    }
    sq = lanes_sum<L>(sq);
    sd = lanes_sum<L>(sd);
}

// Whether the squares sq around a mean are more than half that mean's own error, share =
// sd * c: what would be left of them has lost digits, or both overflowed (inf - inf), or
// the row holds an infinity or NaN.
__device__ __forceinline__ bool mostly_rounding(float share, float sq)
{
    return !(__builtin_fmaf(-2.0f, share, sq) >= 0.0f);
}

// The correction of a mean: none where the row holds infinities or NaN, whose mean the
// first sum already is (inf - inf is no correction).
__device__ __forceinline__ float correction(float sd, float inv)
{
    const float c = sd * inv;
    return __builtin_fabsf(c) <= FLT_MAX ? c : 0.0f;
}

// The squares less the mean's share; infinite squares stay so.
__device__ __forceinline__ float without_mean(float sq, float share) { return sq <= FLT_MAX ? sq - share : sq; }

// A row (nearly) of equal values takes its squares a second time, around the corrected
// mean: its elements and that mean, rounded, are whole multiples of one last place, so
// that these differences are exact and at most half of their squares is the mean's.
template <int TPR, int VPT>
__device__ __forceinline__ WaveStats wave_stats(const float (&x)[VPT][8], const RowShape<TPR, VPT>& shape, int lane,
                                                int dim)
{
    constexpr int L = RowShape<TPR, VPT>::L;
    float s = 0.0f;
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
        const float a = (x[k][0] + x[k][1]) + (x[k][2] + x[k][3]);
        const float b = (x[k][4] + x[k][5]) + (x[k][6] + x[k][7]);
        s += a + b;
    }
    float m0 = lanes_sum<L>(s) * shape.inv_mine, sd, sq;
    deviations<TPR, VPT>(x, m0, lane, dim, sd, sq);
    float c = sd * shape.inv_mine, m2 = sq - sd * c;
    const bool again = mostly_rounding(sd * c, sq);
    if (__any(again)) {                                // (several rows may share the wave)
        m0 = again ? m0 + correction(sd, shape.inv_mine) : m0;
        deviations<TPR, VPT>(x, m0, lane, dim, sd, sq);
        c = correction(sd, shape.inv_mine);
        m2 = without_mean(sq, sd * c);
    }
    return WaveStats{m0, c, m2};
}

// Leaves a wave's share in the row's slot (row_slot_words(TPR) words).
template <int TPR, int VPT>
__device__ __forceinline__ void put_stats(const WaveStats& w, const RowShape<TPR, VPT>& shape, float* slot)
{
    if (RowShape<TPR, VPT>::W > 1 && threadIdx.x % 64 == 0) {
        slot[3 * shape.wave] = w.m0;
        slot[3 * shape.wave + 1] = w.m2;
        slot[3 * shape.wave + 2] = w.c;
    }
}

template <int TPR, int VPT>
__device__ __forceinline__ void join_stats(const WaveStats& w, const RowShape<TPR, VPT>& shape, float eps,
                                           const float* slot, float* mean, float* rstd)
{
    constexpr int W = RowShape<TPR, VPT>::W;
    float m = w.m0 + w.c, m2 = w.m2;
    if constexpr (W > 1) {
        // differences from wave 0's mean (it holds elements in every row): the join keeps
        // the digits that the waves' means share.  A wave without elements has mean 0, weight 0.
        // Lane l takes wave l % W.
        const int l = threadIdx.x % W;
        const float m00 = slot[0], c00 = slot[2];
        const float d = (slot[3 * l] - m00) + (slot[3 * l + 2] - c00);
        const float nd = shape.held * d;
        const float dm = group_sum<W>(nd), dq = group_sum<W>(nd * d), q = group_sum<W>(slot[3 * l + 1]);
        const float shift = dm * shape.inv_dim;
        float between = dq - dm * shift;
        m = m00 + (c00 + shift);
        if (between != between) {                      // squares beyond binary32, infinities, NaN
            between = without_mean(dq, dm * shift);
            if (!(__builtin_fabsf(shift) <= FLT_MAX))  // the mean of the waves' means
                m = group_sum<W>(slot[3 * l] * (shape.held * shape.inv_dim));
        }
        m2 = q + between;
    }
    *mean = m;
    *rstd = inv_deviation(m2 * shape.inv_dim, eps);
}

template <int TPR, int VPT>
__device__ __forceinline__ void row_stats(const float (&x)[VPT][8], const RowShape<TPR, VPT>& shape, int lane, int dim,
                                          float eps, float* slot, float* mean, float* rstd)
{
    const WaveStats w = wave_stats<TPR, VPT>(x, shape, lane, dim);
    put_stats<TPR, VPT>(w, shape, slot);
    if constexpr (TPR > 64) lds_barrier();
    join_stats<TPR, VPT>(w, shape, eps, slot, mean, rstd);
}

// Threads of a workgroup: a row that waves share has one to itself.
constexpr int norm_threads(int tpr) { return tpr > 64 ? tpr : 256; }

// TPR threads to a row; the workgroups walk the rows by the grid, gamma and beta
// stay in registers and the next row is read before the current one is
// reduced.  GATHER: row t is scale * table[ids[t]] (zeros out where the id is
// outside the table); the id is read one row further ahead.
template <int XDT, int YDT, int WDT, int TPR, int VPT, int TAIL, bool GATHER>
__global__ __launch_bounds__(norm_threads(TPR)) void k_norm(const void* __restrict__ x, IdArgs a, float scale,
                                                            const void* __restrict__ gamma,
                                                            const void* __restrict__ beta, float eps,
                                                            void* __restrict__ y, float* __restrict__ mean_out,
                                                            float* __restrict__ rstd_out)
{
    constexpr int RPB = norm_threads(TPR) / TPR;
    // two slots in turn: a wave may leave its share of the next row while another still
    // reads this row's (one barrier a row)
    __shared__ float s_slot[2][RPB][row_slot_words(TPR)];
    int buf = 0;
    const int lane = threadIdx.x % TPR, grp = threadIdx.x / TPR;
    const int dim = a.dim, units = (dim + 7) >> 3;
    const int64_t step = (int64_t)gridDim.x * RPB;

    // row t's id (its own number without GATHER), or -1 where it has no row to read
    auto id_of = [&](int64_t t) -> int64_t {
        if constexpr (GATHER) {
            const int64_t id = t < a.n ? load_id(a.ids, a.id64, t) : -1;
            return (uint64_t)id < (uint64_t)a.rows ? id : -1;
        } else {
            return t < a.n ? t : -1;
        }
    };
    Unit<XDT> xu[VPT] = {};
    auto load_row = [&](int64_t id) {
        if (id >= 0) {
            const char* const row = static_cast<const char*>(x) + id * dim * elem_bytes(XDT);
#pragma unroll
            for (int k = 0; k < VPT; ++k) xu[k] = load_row_unit<XDT, TAIL, !GATHER>(row, k * TPR + lane, units, dim);
        }
    };
    int64_t base = (int64_t)blockIdx.x * RPB;
    int64_t id = id_of(base + grp), id1 = GATHER ? id_of(base + step + grp) : 0;
    load_row(id);
    const RowShape<TPR, VPT> shape(lane, dim);
    float g[VPT][8], b[VPT][8];
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
        Unit<WDT> gu, bu;
        if (gamma) gu = load_row_unit<WDT, TAIL, false>(gamma, k * TPR + lane, units, dim);
        if (beta) bu = load_row_unit<WDT, TAIL, false>(beta, k * TPR + lane, units, dim);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            g[k][j] = gamma ? unit_at<WDT>(gu, j) : 1.0f;
            b[k][j] = beta ? unit_at<WDT>(bu, j) : 0.0f;
        }
    }
    for (; base < a.n; base += step) {
        const int64_t t = base + grp;
        const bool found = id >= 0;
        float v[VPT][8];
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float w = unit_at<XDT>(xu[k], j);
                v[k][j] = GATHER ? w * scale : w;
            }
            if (!whole_step<TPR>(k, dim) && k * TPR + lane >= units) {
#pragma unroll
                for (int j = 0; j < 8; ++j) v[k][j] = 0.0f;
            }
        }
        if constexpr (GATHER) {
            id = id1;
            id1 = id_of(base + 2 * step + grp);
        } else {
            id = id_of(base + step + grp);
        }
        load_row(id);
        float mean = 0.0f, rstd = 0.0f;
        if (TPR < 64 || found) {
            row_stats<TPR, VPT>(v, shape, lane, dim, eps, s_slot[buf][grp], &mean, &rstd);
            buf ^= 1;                    // (only behind a barrier)
        }
        if (t >= a.n) continue;
        if (lane == 0) {
            if (mean_out) mean_out[t] = mean;
            if (rstd_out) rstd_out[t] = rstd;
        }
        char* const yrow = static_cast<char*>(y) + t * dim * elem_bytes(YDT);
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            float o[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) o[j] = __builtin_fmaf((v[k][j] - mean) * rstd, g[k][j], b[k][j]);
            if (GATHER && !found) {
#pragma unroll
                for (int j = 0; j < 8; ++j) o[j] = 0.0f;
            }
            store_row_unit<YDT, TAIL, true>(yrow, k * TPR + lane, units, dim, o);
        }
    }
}

template <int N>
using threads_c = std::integral_constant<int, N>;

// Threads and units per row.  Up to 128 elements 16 lanes share a row, up to
// 1024 one wave (no barrier), beyond that a workgroup, two units a thread at most, so
// that gamma and beta fit in registers (one wave with four units up to 2048 elements,
// 16384 rows: of 2048 bf16 25.7 against 24.0 us, of 1500 32.3 against 23.9).
template <int XDT, int YDT, int WDT, int TAIL, bool GATHER>
hipError_t norm_as(const void* x, const IdArgs& a, float scale, const NormArgs& w, void* y, float* mean, float* rstd,
                   hipStream_t s)
{
    const int units = (a.dim + 7) / 8;
    auto go = [&](auto kernel, auto tpr) {
        constexpr int T = norm_threads(decltype(tpr)::value), RPB = T / decltype(tpr)::value;
        const int64_t tiles = (a.n + RPB - 1) / RPB;
        const int grid = tiles <= 256 ? (int)tiles : persistent_grid_of<T>(kernel, tiles);
        return launch_kernel_nt(kernel, grid, T, s, x, a, scale, w.gamma, w.beta, w.eps, y, mean, rstd);
    };
    if (units <= 16) return go(k_norm<XDT, YDT, WDT, 16, 1, TAIL, GATHER>, threads_c<16>{});
    if constexpr (TAIL != kShort) {
        if (units <= 64) return go(k_norm<XDT, YDT, WDT, 64, 1, TAIL, GATHER>, threads_c<64>{});
        if (units <= 128) return go(k_norm<XDT, YDT, WDT, 64, 2, TAIL, GATHER>, threads_c<64>{});
        if (units <= 256) return go(k_norm<XDT, YDT, WDT, 128, 2, TAIL, GATHER>, threads_c<128>{});
        if (units <= 512) return go(k_norm<XDT, YDT, WDT, 256, 2, TAIL, GATHER>, threads_c<256>{});
        if (units <= 1024) return go(k_norm<XDT, YDT, WDT, 512, 2, TAIL, GATHER>, threads_c<512>{});
        if (units <= 2048) return go(k_norm<XDT, YDT, WDT, 1024, 2, TAIL, GATHER>, threads_c<1024>{});
    }
    return hipErrorInvalidValue;
}

template <int XDT, int YDT, int WDT, bool GATHER>
hipError_t norm_dim(const void* x, const IdArgs& a, float scale, const NormArgs& w, void* y, float* mean, float* rstd,
                    hipStream_t s)
{
    const int tail = tail_of(a.dim);
    return tail == kWhole     ? norm_as<XDT, YDT, WDT, kWhole, GATHER>(x, a, scale, w, y, mean, rstd, s)
           : tail == kPartial ? norm_as<XDT, YDT, WDT, kPartial, GATHER>(x, a, scale, w, y, mean, rstd, s)
                              : norm_as<XDT, YDT, WDT, kShort, GATHER>(x, a, scale, w, y, mean, rstd, s);
}

}  // namespace qb
