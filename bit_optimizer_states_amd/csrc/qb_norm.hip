// qb_norm.hip -- layer norm (forward) and its backward pass with the reduction
// of the weight's gradient.
//
// Backward, with h = (x - mean) * rstd and g = dy * gamma:
//   dx = rstd * (g - mean(g) - h * mean(g h)),  dgamma = sum_rows dy h,
//   dbeta = sum_rows dy.
// One kernel reads dy and x once: a fixed set of workgroups walks the rows, each
// thread keeping binary32 sums of dy h and dy for its own columns in registers;
// at the end a workgroup joins its waves' sums in LDS and writes one partial
// row, and a second kernel adds the partial rows.  Every sum has a fixed order:
// the same bits on every run.  Bound by HBM: 16384 rows of 4096 bf16 in 69 us and 4.5
// us for the partial rows (403 MB: 5.5 TB/s together).  Few long rows are bound by the
// latency of a row or two per workgroup: 1023 rows of 5001 binary32 in 19 and 4 us (61 MB).
#include "qb_norm_kernels.h"

namespace qb {

namespace {

// Rows beyond the kernels of two units a thread (dim > kRowRegMax): one workgroup of
// 1024 threads per row reads it three times (the second and third time from L2): 2048 rows
// of 32768 bf16 in 64 us, 4.2 TB/s.  (16-bit rows of that length would fit registers as
// four raw units a thread; no such kernel was built.)
constexpr int kLongThreads = 1024;

template <int XDT, int WDT>
__global__ __launch_bounds__(kLongThreads) void k_norm_long(const void* __restrict__ x, int64_t dim,
                                                            const void* __restrict__ gamma,
                                                            const void* __restrict__ beta, float eps,
                                                            void* __restrict__ y, float* __restrict__ mean_out,
                                                            float* __restrict__ rstd_out)
{
    __shared__ float s_slot[6 * (kLongThreads / 64)];
    const int64_t t = blockIdx.x;
    const char* const xrow = static_cast<const char*>(x) + t * dim * elem_bytes(XDT);
    char* const yrow = static_cast<char*>(y) + t * dim * elem_bytes(XDT);
    const int64_t whole = dim / 8;
    const int left = (int)(dim % 8);

    float sum = 0.0f;
    for (int64_t u = threadIdx.x; u < whole; u += kLongThreads) {
        const Unit<XDT> w = load_unit8<XDT, false>(xrow, u * 8);
        float s = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) s += unit_at<XDT>(w, j);
        sum += s;
    }
    if ((int)threadIdx.x < left) sum += load1<XDT>(xrow, whole * 8 + threadIdx.x);
    float none = 0.0f;
    row_sum2<kLongThreads>(sum, none, s_slot);
    // differences from m and their squares, as deviations()
    float sd, sq;
    auto around = [&](float m, float* slot) {
        sd = sq = 0.0f;
        for (int64_t u = threadIdx.x; u < whole; u += kLongThreads) {
            const Unit<XDT> w = load_unit8<XDT, false>(xrow, u * 8);
            float a = 0.0f, b = 0.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float d = unit_at<XDT>(w, j) - m;
                a += d;
                b = __builtin_fmaf(d, d, b);
            }
            sd += a;
            sq += b;
        }
        if ((int)threadIdx.x < left) {
            const float d = load1<XDT>(xrow, whole * 8 + threadIdx.x) - m;
            sd += d;
            sq = __builtin_fmaf(d, d, sq);
        }
        row_sum2<kLongThreads>(sd, sq, slot);
    };
    float m0 = sum / (float)dim;
    const float inv = 1.0f / (float)dim;
    around(m0, s_slot + 2 * (kLongThreads / 64));
    float c = correction(sd, inv);
    if (mostly_rounding(sd * c, sq)) {                 // (the same for all threads)
        m0 += c;
        around(m0, s_slot + 4 * (kLongThreads / 64));
        c = correction(sd, inv);
    }
    const float mean = m0 + c;
    const float rstd = inv_deviation(without_mean(sq, sd * c) / (float)dim, eps);
    if (threadIdx.x == 0) {
        if (mean_out) mean_out[t] = mean;
        if (rstd_out) rstd_out[t] = rstd;
    }
    for (int64_t u = threadIdx.x; u < whole; u += kLongThreads) {
        const Unit<XDT> w = load_unit8<XDT, false>(xrow, u * 8);
        Unit<WDT> gu, bu;
        if (gamma) gu = load_unit8<WDT, false>(gamma, u * 8);
        if (beta) bu = load_unit8<WDT, false>(beta, u * 8);
        float o[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
            o[j] = __builtin_fmaf((unit_at<XDT>(w, j) - mean) * rstd, gamma ? unit_at<WDT>(gu, j) : 1.0f,
                                  beta ? unit_at<WDT>(bu, j) : 0.0f);
        store_unit8<XDT, true>(yrow, u * 8, o);
    }
    if ((int)threadIdx.x < left) {
        const int64_t i = whole * 8 + threadIdx.x;
        store1<XDT>(yrow, i,
                    __builtin_fmaf((load1<XDT>(xrow, i) - mean) * rstd, gamma ? load1<WDT>(gamma, i) : 1.0f,
                                   beta ? load1<WDT>(beta, i) : 0.0f));
    }
}

template <int XDT, int WDT>
hipError_t layer_norm_as(const void* x, int64_t n, int64_t dim, const NormArgs& w, void* y, float* mean, float* rstd,
                         hipStream_t s)
{
    if (dim > kRowRegMax)
        return launch_rows(n, 1, [&](int64_t t0, int64_t, int grid) {
            const int64_t at = t0 * dim * elem_bytes(XDT);
            return launch_kernel_nt(k_norm_long<XDT, WDT>, grid, kLongThreads, s, static_cast<const char*>(x) + at, dim,
                                    w.gamma, w.beta, w.eps, static_cast<char*>(y) + at, mean ? mean + t0 : nullptr,
                                    rstd ? rstd + t0 : nullptr);
        });
    const IdArgs a{nullptr, n, n, 0, (int32_t)dim};
    return norm_dim<XDT, XDT, WDT, false>(x, a, 1.0f, w, y, mean, rstd, s);
}

// Backward pass.  NT threads: NT / TPR rows at a time.  LDS (dynamic): gamma in
// binary32 while the rows are walked, then the joined sums, padded_dim floats.
template <int XDT, int WDT, int TPR, int VPT, int TAIL, int NT>
__global__ __launch_bounds__(NT) void k_norm_grad(const void* __restrict__ dy, const void* __restrict__ x, int64_t n,
                                                  int dim, const void* __restrict__ gamma,
                                                  const float* __restrict__ mean_in, const float* __restrict__ rstd_in,
                                                  void* __restrict__ dx, float* __restrict__ part)
{
    extern __shared__ __align__(16) float s_cols[];
    constexpr int GROUPS = NT / TPR;
    constexpr int SLOT = TPR <= 64 ? 1 : 2 * (TPR / 64);
    constexpr bool KEEP = VPT <= 2;          // h and g stay in registers for the second use
    __shared__ float s_slot[2][GROUPS][SLOT];
    const int lane = threadIdx.x % TPR, grp = threadIdx.x / TPR;
    const int units = (dim + 7) >> 3, padded = units * 8;
    float accg[VPT][8] = {}, accb[VPT][8] = {};
    const float inv = 1.0f / (float)dim;
    int buf = 0;
    const int64_t step = (int64_t)gridDim.x * GROUPS;
    Unit<XDT> xu[VPT], du[VPT];
    float m, r;
    auto load_next = [&](int64_t t) {
        const int64_t at = t < n ? t : n - 1;
        const char* const xrow = static_cast<const char*>(x) + at * dim * elem_bytes(XDT);
        const char* const grow = static_cast<const char*>(dy) + at * dim * elem_bytes(XDT);
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            du[k] = load_row_unit<XDT, TAIL, true>(grow, k * TPR + lane, units, dim);
            xu[k] = load_row_unit<XDT, TAIL, true>(xrow, k * TPR + lane, units, dim);
        }
        m = t < n ? mean_in[at] : 0.0f;
        r = t < n ? rstd_in[at] : 0.0f;
    };
    int64_t t0 = (int64_t)blockIdx.x * GROUPS;
    load_next(t0 + grp);
    for (int unit = threadIdx.x; unit < units; unit += NT) {
        Unit<WDT> u;
        if (gamma) u = load_row_unit<WDT, TAIL, false>(gamma, unit, units, dim);
#pragma unroll
        for (int j = 0; j < 8; ++j) s_cols[unit * 8 + j] = gamma ? unit_at<WDT>(u, j) : 1.0f;
    }
    lds_barrier();
    for (; t0 < n; t0 += step) {
        const int64_t t = t0 + grp;
        const bool live = t < n;
        const int64_t row = t * dim * elem_bytes(XDT);
        // Elements beyond the row, and rows beyond the last, take a dy and an h of zero ((0 - m) * r may
        // overflow).
        float s1 = 0.0f, s2 = 0.0f;
        float hk[KEEP ? VPT : 1][8], gk[KEEP ? VPT : 1][8];
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            const int unit = k * TPR + lane;
            if (!(whole_step<TPR>(k, dim) && t0 + GROUPS <= n) && (!live || unit >= units)) {
#pragma unroll
                for (int j = 0; j < (XDT == DT_F32 ? 8 : 4); ++j) du[k].w[j] = xu[k].w[j] = 0u;
            }
            const float* const gam = s_cols + (unit < units ? unit : 0) * 8;
            const bool whole = whole_step<TPR>(k, dim);
            const float rk = TAIL != kWhole || whole || unit < units ? r : 0.0f;
            const int cnt = unit_count(unit, dim);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float d = unit_at<XDT>(du[k], j);
                float h = (unit_at<XDT>(xu[k], j) - m) * rk;
                if (TAIL != kWhole && !whole) h = j < cnt ? h : 0.0f;
                const float g = d * gam[j];
                s1 += g;
                s2 = __builtin_fmaf(g, h, s2);
                accg[k][j] = __builtin_fmaf(d, h, accg[k][j]);
                accb[k][j] += d;
                if constexpr (KEEP) {
                    hk[k][j] = h;
                    gk[k][j] = g;
                }
            }
        }
        row_sum2<TPR>(s1, s2, s_slot[buf][grp]);
        buf ^= 1;
        if (dx && live) {
            const float c1 = s1 * inv, c2 = s2 * inv;
            char* const orow = static_cast<char*>(dx) + row;
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
                const int unit = k * TPR + lane;
                const float* const gam = s_cols + (unit < units ? unit : 0) * 8;
                float o[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    float h, g;
                    if constexpr (KEEP) {
                        h = hk[k][j];
                        g = gk[k][j];
                    } else {
                        h = (unit_at<XDT>(xu[k], j) - m) * r;
                        g = unit_at<XDT>(du[k], j) * gam[j];
                    }
                    o[j] = r * (g - __builtin_fmaf(h, c2, c1));
                }
                store_row_unit<XDT, TAIL, true>(orow, unit, units, dim, o);
            }
        }
        if (t0 + step < n) load_next(t + step);
    }
    if (!part) return;

    // Join: the threads that hold the same columns take turns, one unit each at a time.
    if constexpr (TPR == 16) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            accg[0][j] += __shfl_xor(accg[0][j], 16);
            accg[0][j] += __shfl_xor(accg[0][j], 32);
            accb[0][j] += __shfl_xor(accb[0][j], 16);
            accb[0][j] += __shfl_xor(accb[0][j], 32);
        }
    }
    constexpr int JT = TPR < 64 ? 64 : TPR;          // threads that hold one set of columns
    constexpr int SETS = NT / JT;
    const int set = threadIdx.x / JT;
    const bool mine = TPR >= 64 || threadIdx.x % 64 < TPR;
    float* const out = part + (int64_t)blockIdx.x * 2 * padded;
    auto join = [&](float (&acc)[VPT][8], float* dst) {
        __syncthreads();
#pragma unroll
        for (int turn = 0; turn < SETS; ++turn) {
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
                const int unit = k * TPR + lane;
                if (mine && unit < units && k % SETS == (set + turn) % SETS) {
                    float* const p = s_cols + unit * 8;
#pragma unroll
                    for (int j = 0; j < 8; ++j) p[j] = turn == 0 ? acc[k][j] : p[j] + acc[k][j];
                }
            }
            __syncthreads();
        }
        for (int c = threadIdx.x * 4; c < padded; c += NT * 4)
            *reinterpret_cast<float4*>(dst + c) = *reinterpret_cast<const float4*>(s_cols + c);
    };
    join(accg, out);
    join(accb, out + padded);
}

// Long rows: dx by one workgroup per row, which reads the row twice (2048 rows of
// 32768 bf16: 90 us, 4.5 TB/s of the 403 MB; 52 us more for the column sums) ...
template <int XDT, int WDT>
__global__ __launch_bounds__(kLongThreads) void k_norm_grad_long(const void* __restrict__ dy,
                                                                 const void* __restrict__ x, int64_t dim,
                                                                 const void* __restrict__ gamma,
                                                                 const float* __restrict__ mean_in,
                                                                 const float* __restrict__ rstd_in,
                                                                 void* __restrict__ dx)
{
    __shared__ float s_slot[2 * (kLongThreads / 64)];
    const int64_t t = blockIdx.x, row = t * dim * elem_bytes(XDT);
    const char* const xrow = static_cast<const char*>(x) + row;
    const char* const grow = static_cast<const char*>(dy) + row;
    char* const orow = static_cast<char*>(dx) + row;
    const float m = mean_in[t], r = rstd_in[t];
    const int64_t whole = dim / 8, i = whole * 8 + threadIdx.x;        // i: one of the last dim % 8 elements
    const bool last = i < dim;
    float s1 = 0.0f, s2 = 0.0f;
    for (int64_t u = threadIdx.x; u < whole; u += kLongThreads) {
        const Unit<XDT> xu = load_unit8<XDT, false>(xrow, u * 8), du = load_unit8<XDT, false>(grow, u * 8);
        Unit<WDT> gu;
        if (gamma) gu = load_unit8<WDT, false>(gamma, u * 8);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float g = unit_at<XDT>(du, j) * (gamma ? unit_at<WDT>(gu, j) : 1.0f);
            s1 += g;
            s2 = __builtin_fmaf(g, (unit_at<XDT>(xu, j) - m) * r, s2);
        }
    }
    const float gl = last ? load1<XDT>(grow, i) * (gamma ? load1<WDT>(gamma, i) : 1.0f) : 0.0f;
    const float hl = last ? (load1<XDT>(xrow, i) - m) * r : 0.0f;
    s1 += gl;
    s2 = __builtin_fmaf(gl, hl, s2);
    row_sum2<kLongThreads>(s1, s2, s_slot);
    const float c1 = s1 / (float)dim, c2 = s2 / (float)dim;
    for (int64_t u = threadIdx.x; u < whole; u += kLongThreads) {
        const Unit<XDT> xu = load_unit8<XDT, false>(xrow, u * 8), du = load_unit8<XDT, false>(grow, u * 8);
        Unit<WDT> gu;
        if (gamma) gu = load_unit8<WDT, false>(gamma, u * 8);
        float o[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float g = unit_at<XDT>(du, j) * (gamma ? unit_at<WDT>(gu, j) : 1.0f);
            o[j] = r * (g - __builtin_fmaf((unit_at<XDT>(xu, j) - m) * r, c2, c1));
        }
        store_unit8<XDT, true>(orow, u * 8, o);
    }
    if (last) store1<XDT>(orow, i, r * (gl - __builtin_fmaf(hl, c2, c1)));
}

// ... and the column sums apart: workgroup (b % parts) takes the rows t = part,
// part + parts, ... of 256 columns, four rows in flight.
template <int XDT>
__global__ __launch_bounds__(256) void k_norm_cols(const void* __restrict__ dy, const void* __restrict__ x, int64_t n,
                                                   int64_t dim, const float* __restrict__ mean_in,
                                                   const float* __restrict__ rstd_in, float* __restrict__ part,
                                                   int parts)
{
    const int p = blockIdx.x % parts;
    const int64_t c = (int64_t)(blockIdx.x / parts) * 256 + threadIdx.x, padded = (dim + 7) / 8 * 8;
    if (c >= padded) return;
    float sg = 0.0f, sb = 0.0f;
    if (c < dim) {
#pragma unroll 4
        for (int64_t t = p; t < n; t += parts) {
            const float d = load1<XDT>(dy, t * dim + c);
            sg = __builtin_fmaf(d, (load1<XDT>(x, t * dim + c) - mean_in[t]) * rstd_in[t], sg);
            sb += d;
        }
    }
    float* const out = part + (int64_t)p * 2 * padded;
    out[c] = sg;
    out[padded + c] = sb;
}

constexpr int kLongParts = 64;

// Threads and units per row: two units a thread where a row allows it, so that h and g
// stay in registers and 16 waves fit a CU (8192 rows: 5001 binary32 elements 127 -> 104
// us against four units a thread, 8192 bf16 83 -> 78).  Up to 2048 elements a wave
// with four units needs no barrier, which pays for whole units (16384 rows of 2048 bf16:
// 39.8 against 41.2 us), but not where shifting the last unit needs registers too
// (1500: 45.4 against 37.8).
template <int XDT, int WDT, int TAIL>
hipError_t grad_as(const void* dy, const void* x, int64_t n, int dim, const void* gamma, const float* mean,
                   const float* rstd, void* dx, float* part, hipStream_t s)
{
    const int units = (dim + 7) / 8;
    const int grid = layer_norm_parts(n, dim);
    const size_t lds = (size_t)units * 8 * sizeof(float);
    auto go = [&](auto kernel, int threads) {
        return launch_kernel_lds(kernel, grid, threads, lds, s, dy, x, n, dim, gamma, mean, rstd, dx, part);
    };
    if (units <= 16) return go(k_norm_grad<XDT, WDT, 16, 1, TAIL, 512>, 512);
    if constexpr (TAIL != kShort) {
        if (units <= 64) return go(k_norm_grad<XDT, WDT, 64, 1, TAIL, 512>, 512);
        if (units <= 128) return go(k_norm_grad<XDT, WDT, 64, 2, TAIL, 512>, 512);
        if constexpr (TAIL == kWhole) {
            if (units <= 256) return go(k_norm_grad<XDT, WDT, 64, 4, TAIL, 512>, 512);
        } else {
            if (units <= 256) return go(k_norm_grad<XDT, WDT, 128, 2, TAIL, 1024>, 1024);
        }
        if (units <= 512) return go(k_norm_grad<XDT, WDT, 256, 2, TAIL, 1024>, 1024);
        if (units <= 1024) return go(k_norm_grad<XDT, WDT, 512, 2, TAIL, 1024>, 1024);
        return go(k_norm_grad<XDT, WDT, 1024, 2, TAIL, 1024>, 1024);
    }
    return hipErrorInvalidValue;
}

template <int XDT, int WDT>
hipError_t layer_norm_grad_as(const void* dy, const void* x, int64_t n, int64_t dim, const void* gamma,
                              const float* mean, const float* rstd, void* dx, float* part, hipStream_t s)
{
    if (dim > kRowRegMax) {
        if (dx) {
            const hipError_t e = launch_rows(n, 1, [&](int64_t t0, int64_t, int grid) {
                const int64_t at = t0 * dim * elem_bytes(XDT);
                return launch_kernel_nt(k_norm_grad_long<XDT, WDT>, grid, kLongThreads, s,
                                        static_cast<const char*>(dy) + at, static_cast<const char*>(x) + at, dim,
                                        gamma, mean + t0, rstd + t0, static_cast<char*>(dx) + at);
            });
            if (e != hipSuccess) return e;
        }
        if (!part) return hipSuccess;
        const int parts = layer_norm_parts(n, dim);
        const int64_t grid = (padded_dim(dim) + 255) / 256 * parts;
        if (grid >= (int64_t(1) << 24)) return hipErrorInvalidValue;
        return launch_kernel(k_norm_cols<XDT>, (int)grid, s, dy, x, n, dim, mean, rstd, part, parts);
    }
    const int tail = tail_of(dim);
    return tail == kWhole     ? grad_as<XDT, WDT, kWhole>(dy, x, n, (int)dim, gamma, mean, rstd, dx, part, s)
           : tail == kPartial ? grad_as<XDT, WDT, kPartial>(dy, x, n, (int)dim, gamma, mean, rstd, dx, part, s)
                              : grad_as<XDT, WDT, kShort>(dy, x, n, (int)dim, gamma, mean, rstd, dx, part, s);
}

// dgamma, dbeta = the sum of the partial rows.  A workgroup takes 64 of the 2 *
// padded columns: 16 lanes of 4 columns, the partial rows dealt to 32 threads
// each (8 of 256 rows in flight at once), joined in LDS.
constexpr int kJoinRows = 32;

__global__ __launch_bounds__(16 * kJoinRows) void k_join_parts(const float* __restrict__ part, int parts, int64_t dim,
                                                               int64_t padded, int accumulate,
                                                               void* __restrict__ dgamma, void* __restrict__ dbeta,
                                                               int wdt)
{
    __shared__ f32x4 s_sum[kJoinRows][16];
    const int l = threadIdx.x % 16, q = threadIdx.x / 16;
    const int64_t c = (int64_t)blockIdx.x * 64 + l * 4;
    f32x4 sum = {0.0f, 0.0f, 0.0f, 0.0f};
    if (c < 2 * padded) {
        const float* p = part + c;
#pragma unroll 8
        for (int g = q; g < parts; g += kJoinRows) sum += gld<f32x4>(p + (int64_t)g * 2 * padded);
    }
    s_sum[q][l] = sum;
    __syncthreads();
    if (threadIdx.x < 64) {
        const int64_t cc = (int64_t)blockIdx.x * 64 + threadIdx.x;
        float v = 0.0f;
#pragma unroll
        for (int g = 0; g < kJoinRows; ++g) v += s_sum[g][threadIdx.x / 4][threadIdx.x % 4];
        if (cc < 2 * padded) {
            void* const out = cc < padded ? dgamma : dbeta;
            const int64_t i = cc < padded ? cc : cc - padded;
            if (out && i < dim) {
                if (accumulate) v += load1_rt(wdt, out, i);
                store1_rt(wdt, out, i, v);
            }
        }
    }
}

}  // namespace

// Rows a workgroup of the backward kernel takes at once.
int norm_grad_groups(int64_t dim)
{
    const int64_t units = (dim + 7) / 8;
    return units <= 16 ? 32 : units <= 256 ? 8 : units <= 512 ? 4 : units <= 1024 ? 2 : 1;
}

// One workgroup per CU at most, and two rows at least per group of threads:
// every workgroup writes two partial rows of binary32, which for few rows cost
// more than the rows (1024 rows of 8192 16-bit elements: 23.6 us with 512
// workgroups, 14.4 us of them without the partial rows).
int layer_norm_parts(int64_t n, int64_t dim)
{
    if (dim > kRowRegMax) return (int)(n < kLongParts ? n : kLongParts);
    const int64_t per = 2 * norm_grad_groups(dim), g = (n + per - 1) / per;
    return (int)(g < kNormPartsMax ? g : kNormPartsMax);
}

hipError_t launch_layer_norm(const void* x, int xdt, int64_t n, int64_t dim, const NormArgs& w, void* y, float* mean,
                             float* rstd, hipStream_t s)
{
    if (w.wdt == DT_F32) {
        if (xdt == DT_F32) return layer_norm_as<DT_F32, DT_F32>(x, n, dim, w, y, mean, rstd, s);
        if (xdt == DT_F16) return layer_norm_as<DT_F16, DT_F32>(x, n, dim, w, y, mean, rstd, s);
        return layer_norm_as<DT_BF16, DT_F32>(x, n, dim, w, y, mean, rstd, s);
    }
    if (w.wdt != xdt) return hipErrorInvalidValue;
    if (xdt == DT_F16) return layer_norm_as<DT_F16, DT_F16>(x, n, dim, w, y, mean, rstd, s);
    return layer_norm_as<DT_BF16, DT_BF16>(x, n, dim, w, y, mean, rstd, s);
}

hipError_t launch_layer_norm_grad(const void* dy, const void* x, int xdt, int64_t n, int64_t dim, const void* gamma,
                                  int wdt, const float* mean, const float* rstd, void* dx, float* part, hipStream_t s)
{
    if (wdt == DT_F32) {
        if (xdt == DT_F32) return layer_norm_grad_as<DT_F32, DT_F32>(dy, x, n, dim, gamma, mean, rstd, dx, part, s);
        if (xdt == DT_F16) return layer_norm_grad_as<DT_F16, DT_F32>(dy, x, n, dim, gamma, mean, rstd, dx, part, s);
        return layer_norm_grad_as<DT_BF16, DT_F32>(dy, x, n, dim, gamma, mean, rstd, dx, part, s);
    }
    if (wdt != xdt) return hipErrorInvalidValue;
    if (xdt == DT_F16) return layer_norm_grad_as<DT_F16, DT_F16>(dy, x, n, dim, gamma, mean, rstd, dx, part, s);
    return layer_norm_grad_as<DT_BF16, DT_BF16>(dy, x, n, dim, gamma, mean, rstd, dx, part, s);
}

hipError_t launch_join_parts(const float* part, int parts, int64_t dim, bool accumulate, void* dgamma, void* dbeta,
                             int wdt, hipStream_t s)
{
    if (!dgamma && !dbeta) return hipSuccess;
    const int64_t padded = padded_dim(dim), grid = (2 * padded + 63) / 64;
    if (grid >= (int64_t(1) << 24)) return hipErrorInvalidValue;
    return launch_kernel_nt(k_join_parts, (int)grid, 16 * kJoinRows, s, part, parts, dim, padded, accumulate ? 1 : 0, dgamma, dbeta,
                         wdt);
}

}  // namespace qb
