// qb_linear_grad.hip -- the elementwise half of the 4-bit layers' gradients: the gradient
// at the pre-activation, padded to the tiled product's steps, and the bias's.
//
//   linear: dz = dy act'(z), db = sum over rows of dz;
//   gated:  dg = dh u act'(g), du = dh act(g).
// dz, dg and du are rounded to the compute dtype, which the matrix instructions take; db
// sums the unrounded values in binary32, rows in a fixed order.  Bound by HBM.
#include "qb_act.h"
#include "qb_linear.h"
#include "qb_rows.h"

namespace qb {

namespace {

constexpr int kCols = kDzCols, kGradWaves = kDzWaves;     // a workgroup: a wave's 64 units of 8 columns, 4 waves

// A unit at row `row` of an array padded to `pitch` columns (a multiple of 8).
template <int XDT>
__device__ __forceinline__ void store_padded(void* p, int64_t row, int64_t pitch, int unit, const float* v)
{
    if ((int64_t)unit * 8 < pitch)
        store_unit8<XDT, false>(static_cast<char*>(p) + row * pitch * elem_bytes(XDT), (int64_t)unit * 8, v);
}

template <int XDT>
__device__ __forceinline__ void store_plain(void* p, int64_t row, int64_t N, int unit, const float* v)
{
    char* const q = static_cast<char*>(p) + row * N * elem_bytes(XDT);
    const int64_t i = (int64_t)unit * 8;
    if (i + 8 <= N) {
        store_unit8<XDT, false>(q, i, v);
    } else {
#pragma unroll
        for (int j = 0; j < 7; ++j)
            if (i + j < N) store1<XDT>(q, i + j, v[j]);
    }
}

// Row `row` of an array of N columns.
template <int XDT>
__device__ __forceinline__ const char* row_of(const void* p, int64_t row, int64_t N)
{
    return static_cast<const char*>(p) + row * N * elem_bytes(XDT);
}

// A unit's values, zeros beyond the row.
template <int XDT, int TAIL>
__device__ __forceinline__ void unit_values(const Unit<XDT>& u, int unit, int N, float* v)
{
    const int cnt = unit_count(unit, N);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = j < cnt ? unit_at<XDT>(u, j) : 0.0f;
}

// Workgroup (block of columns, slice of rows); its waves take the slice's rows in turn, the
// next row in flight.
template <int XDT, int TAIL>
__global__ __launch_bounds__(64 * kGradWaves) void k_linear_dz(const void* __restrict__ dy, const void* __restrict__ z,
                                                               int act, int64_t M, int64_t N, void* __restrict__ dz,
                                                               int64_t pitch, void* __restrict__ dz_out,
                                                               float* __restrict__ part, int slices)
{
    __shared__ float s_sum[kGradWaves][kCols];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int slice = blockIdx.x % slices;
    const int64_t block = blockIdx.x / slices;
    const int units = (int)((N + 7) / 8), unit = (int)(block * 64 + lane);
    const int64_t step = (int64_t)slices * kGradWaves;
    float sum[8] = {};
    Unit<XDT> du, zu;
    auto load_row = [&](int64_t m) {
        if (m >= M) return;
        du = load_row_unit<XDT, TAIL, false>(row_of<XDT>(dy, m, N), unit, units, (int)N);
        if (z) zu = load_row_unit<XDT, TAIL, false>(row_of<XDT>(z, m, N), unit, units, (int)N);
    };
    int64_t m = slice * kGradWaves + wave;
    load_row(m);
    for (; m < M; m += step) {
        float d[8];
        unit_values<XDT, TAIL>(du, unit, (int)N, d);
        if (z) {
            float zv[8];
            unit_values<XDT, TAIL>(zu, unit, (int)N, zv);
            load_row(m + step);
            times_act_slopes<8>(act, zv, d);
        } else {
            load_row(m + step);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) sum[j] += d[j];
        if (dz) store_padded<XDT>(dz, m, pitch, unit, d);
        if (dz_out) store_plain<XDT>(dz_out, m, N, unit, d);
    }
    if (!part) return;
#pragma unroll
    for (int j = 0; j < 8; ++j) s_sum[wave][lane * 8 + j] = sum[j];
    __syncthreads();
    for (int c = threadIdx.x; c < kCols; c += 64 * kGradWaves) {
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < kGradWaves; ++w) v += s_sum[w][c];
        if (block * kCols + c < N) part[(int64_t)slice * N + block * kCols + c] = v;
    }
}

// 64 columns a workgroup; the slices dealt to 16 waves, joined in wave order (4096 columns
// of 128 slices: one thread a column takes 7 us).
constexpr int kSumWaves = 16;

__global__ __launch_bounds__(64 * kSumWaves) void k_bias_sum(const float* __restrict__ part, int slices, int64_t N,
                                                             int accumulate, void* __restrict__ db, int bias_dt)
{
    __shared__ float s_sum[kSumWaves][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t n = (int64_t)blockIdx.x * 64 + lane;
    float v = 0.0f;
    if (n < N) {
#pragma unroll 8
        for (int s = wave; s < slices; s += kSumWaves) v += part[(int64_t)s * N + n];
    }
    s_sum[wave][lane] = v;
    __syncthreads();
    if (wave != 0 || n >= N) return;
    float sum = 0.0f;
#pragma unroll
    for (int w = 0; w < kSumWaves; ++w) sum += s_sum[w][lane];
    if (accumulate) sum += load1_rt(bias_dt, db, n);
    store1_rt(bias_dt, db, n, sum);
}

template <int XDT, int TAIL>
__global__ __launch_bounds__(256) void k_gated_dz(const void* __restrict__ dh, const void* __restrict__ g,
                                                  const void* __restrict__ u, int act, int64_t M, int64_t N,
                                                  void* __restrict__ dz, int64_t pitch, void* __restrict__ dg_out,
                                                  void* __restrict__ du_out, int blocks)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t block = blockIdx.x % blocks;
    const int64_t rows = (int64_t)gridDim.x / blocks * 4;
    const int units = (int)((N + 7) / 8), unit = (int)(block * 64 + lane);
    Unit<XDT> du, gu, uu;
    auto load_row = [&](int64_t m) {
        if (m >= M) return;
        du = load_row_unit<XDT, TAIL, true>(row_of<XDT>(dh, m, N), unit, units, (int)N);
        gu = load_row_unit<XDT, TAIL, true>(row_of<XDT>(g, m, N), unit, units, (int)N);
        uu = load_row_unit<XDT, TAIL, true>(row_of<XDT>(u, m, N), unit, units, (int)N);
    };
    int64_t m = (int64_t)(blockIdx.x / blocks) * 4 + wave;
    load_row(m);
    for (; m < M; m += rows) {
        float d[8], gv[8], uv[8], a[8];
        unit_values<XDT, TAIL>(du, unit, (int)N, d);
        unit_values<XDT, TAIL>(gu, unit, (int)N, gv);
        unit_values<XDT, TAIL>(uu, unit, (int)N, uv);
        load_row(m + rows);
        // d u act'(g) and d act(g)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            a[j] = d[j] * uv[j];
            uv[j] = d[j];
        }
        times_act_both<8>(act, gv, a, uv);
        if (dz) {
            store_padded<XDT>(dz, m, pitch, unit, a);
            store_padded<XDT>(static_cast<char*>(dz) + M * pitch * elem_bytes(XDT), m, pitch, unit, uv);
        }
        if (dg_out) store_plain<XDT>(dg_out, m, N, unit, a);
        if (du_out) store_plain<XDT>(du_out, m, N, unit, uv);
    }
}

// Blocks of kCols columns that cover N columns and the padding.
int64_t column_blocks(int64_t N, int64_t pitch) { return ((pitch > N ? pitch : N) + kCols - 1) / kCols; }

template <int XDT, int TAIL>
hipError_t linear_dz_as(const void* dy, const void* z, int act, int64_t M, int64_t N, void* dz, int64_t pitch,
                        void* dz_out, float* part, int slices, hipStream_t s)
{
    return launch_kernel(k_linear_dz<XDT, TAIL>, (int)(column_blocks(N, dz ? pitch : 0) * slices), s, dy, z, act, M, N,
                         dz, pitch, dz_out, part, slices);
}

template <int XDT>
hipError_t linear_dz_dt(const void* dy, const void* z, int act, int64_t M, int64_t N, void* dz, int64_t pitch,
                        void* dz_out, float* part, int slices, hipStream_t s)
{
    const int tail = tail_of(N);
    return tail == kWhole     ? linear_dz_as<XDT, kWhole>(dy, z, act, M, N, dz, pitch, dz_out, part, slices, s)
           : tail == kPartial ? linear_dz_as<XDT, kPartial>(dy, z, act, M, N, dz, pitch, dz_out, part, slices, s)
                              : linear_dz_as<XDT, kShort>(dy, z, act, M, N, dz, pitch, dz_out, part, slices, s);
}

template <int XDT, int TAIL>
hipError_t gated_dz_as(const void* dh, const void* g, const void* u, int act, int64_t M, int64_t N, void* dz,
                       int64_t pitch, void* dg_out, void* du_out, hipStream_t s)
{
    const int64_t blocks = column_blocks(N, dz ? pitch : 0), row_groups = (M + 3) / 4;
    const int64_t want = (4096 + blocks - 1) / blocks, take = row_groups < want ? row_groups : want;
    return launch_kernel(k_gated_dz<XDT, TAIL>, (int)(blocks * take), s, dh, g, u, act, M, N, dz, pitch, dg_out,
                         du_out, (int)blocks);
}

template <int XDT>
hipError_t gated_dz_dt(const void* dh, const void* g, const void* u, int act, int64_t M, int64_t N, void* dz,
                       int64_t pitch, void* dg_out, void* du_out, hipStream_t s)
{
    const int tail = tail_of(N);
    return tail == kWhole     ? gated_dz_as<XDT, kWhole>(dh, g, u, act, M, N, dz, pitch, dg_out, du_out, s)
           : tail == kPartial ? gated_dz_as<XDT, kPartial>(dh, g, u, act, M, N, dz, pitch, dg_out, du_out, s)
                              : gated_dz_as<XDT, kShort>(dh, g, u, act, M, N, dz, pitch, dg_out, du_out, s);
}

}  // namespace

hipError_t launch_linear_dz(int xdt, const void* dy, const void* z, int act, int64_t M, int64_t N, void* dz,
                            int64_t pitch, void* dz_out, float* part, int slices, hipStream_t s)
{
    switch (xdt) {
    case DT_F32: return linear_dz_dt<DT_F32>(dy, z, act, M, N, dz, pitch, dz_out, part, slices, s);
    case DT_F16: return linear_dz_dt<DT_F16>(dy, z, act, M, N, dz, pitch, dz_out, part, slices, s);
    default: return linear_dz_dt<DT_BF16>(dy, z, act, M, N, dz, pitch, dz_out, part, slices, s);
    }
}

hipError_t launch_bias_sum(const float* part, int slices, int64_t N, bool accumulate, void* db, int bias_dt,
                           hipStream_t s)
{
    return launch_kernel_nt(k_bias_sum, (int)((N + 63) / 64), 64 * kSumWaves, s, part, slices, N, accumulate ? 1 : 0, db, bias_dt);
}

hipError_t launch_gated_dz(int xdt, const void* dh, const void* g, const void* u, int act, int64_t M, int64_t N,
                           void* dz, int64_t pitch, void* dg_out, void* du_out, hipStream_t s)
{
    switch (xdt) {
    case DT_F32: return gated_dz_dt<DT_F32>(dh, g, u, act, M, N, dz, pitch, dg_out, du_out, s);
    case DT_F16: return gated_dz_dt<DT_F16>(dh, g, u, act, M, N, dz, pitch, dg_out, du_out, s);
    default: return gated_dz_dt<DT_BF16>(dh, g, u, act, M, N, dz, pitch, dg_out, du_out, s);
    }
}

}  // namespace qb
