// qb_linear_grad.hip -- what the product of the 4-bit layers' gradients takes: the gradient
// at the pre-activation, padded to the product's steps, and the weights transposed, by one
// launch of two kinds of workgroups (neither needs the other); and the bias's gradient.
//
//   linear: dz = dy act'(z), db = sum over rows of dz;
//   gated:  dg = dh u act'(g), du = dh act(g).
// dz, dg and du are rounded to the compute dtype, which the matrix instructions take; db
// sums the unrounded values in binary32, rows in a fixed order.  Bound by HBM.
#include <type_traits>

#include "qb_act.h"
#include "qb_linear.h"
#include "qb_mm_device.h"
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

struct LinearDz {
    const void *dy, *z;
    void *dz, *dz_out;
    float* part;
    int64_t M, N, pitch;
    int32_t act, slices;
};

struct GatedDz {
    const void *dh, *g, *u;
    void *dz, *dg_out, *du_out;
    int64_t M, N, pitch;
    int32_t act, blocks;
};

// Transposed, into out[k][n]: a workgroup takes 64 rows n and 128 columns k, 8 weights of two
// neighbouring rows a thread at a time into LDS, and writes rows k of 64 n (128 bytes, 256 in
// binary32).  16-byte chunk c of LDS row k lies at chunk c ^ spread(k): the threads of a
// wave, which hold 16 k eight apart and 4 row pairs, write to different banks but for two
// each.  (Rows padded by 16 bytes instead fell into one bank: 4096 x 4096 15.1 us.)
template <int XDT, bool DQ>
__device__ __forceinline__ void unpack_transposed(const TransposedWeights& t, int64_t bx, int64_t by, int bz, char* s_t,
                                                  const QbTables* tab)
{
    constexpr int ES = XDT == DT_F32 ? 4 : 2;
    constexpr int LP = 64 * ES, CPR = LP / 16;                // bytes and chunks of an LDS row of 64 n
    __shared__ float s_val[16];
    __shared__ float s_dyn[DQ ? 256 : 1];
    const int tid = threadIdx.x, kl = (tid & 15) * 8;
    const int64_t k0 = bx * 128, n0 = by * 64, N = t.N, K = t.K, np = t.np, pitch = t.np * t.count;
    const Weight4 w = t.w[bz];
    const Weight4Format f = t.f;
    // row pairs tid / 16 and tid / 16 + 16 of the tile: codes and constants of 8 weights of each row
    uint32_t code[2][2], c2[2][2];
    float a[2][2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int64_t n = n0 + 2 * ((tid >> 4) + 16 * i) + h, e = n * K + k0 + kl, blk = e >> f.log2B;
            code[i][h] = c2[i][h] = 0u;
            a[i][h] = 0.0f;
            if (n < N && k0 + kl < K) {
                code[i][h] = gld<uint32_t>(w.codes + e / 2);
                if constexpr (DQ) {
                    c2[i][h] = gld<uint8_t>(w.c2 + blk);
                    a[i][h] = gld<float>(w.absmax2 + (blk >> f.log2B2));
                } else {
                    a[i][h] = gld<float>(w.absmax + blk);
                }
            }
        }
    const float mu = DQ ? gld<float>(w.offset) : 0.0f;
    if (tid < 16) s_val[tid] = (f.code4 == 0 ? tab->nf4 : tab->fp4)[tid];
    if constexpr (DQ) s_dyn[tid] = tab->dyn8[tid];
    __syncthreads();
    auto spread = [](int k) { return XDT == DT_F32 ? ((k >> 3) & 7) * 2 : (k >> 3) & 7; };
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int pr = (tid >> 4) + 16 * i;
        Frag<DT_F32> v[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int64_t n = n0 + 2 * pr + h;
            const float c = DQ ? s_dyn[c2[i][h]] * a[i][h] + mu : a[i][h];       // two rounded operations
            dequant_frag<DT_F32>(code[i][h], n < N ? c : 0.0f, s_val, v[h]);     // zeros beyond the last row
        }
        const int at = 2 * pr * ES;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            char* const p = s_t + (kl + j) * LP + ((at / 16) ^ spread(kl)) * 16 + at % 16;
            if constexpr (XDT == DT_F32) {
                typedef float f32x2_t __attribute__((ext_vector_type(2)));
                *reinterpret_cast<f32x2_t*>(p) = f32x2_t{v[0].w[j], v[1].w[j]};
            } else {
                *reinterpret_cast<uint32_t*>(p) = pack_two<XDT>(v[0].w[j], v[1].w[j]);
            }
        }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 128 * CPR / 256; ++i) {
        const int o = tid + 256 * i, row = o / CPR, c = o % CPR;
        if (k0 + row < K && n0 + c * (16 / ES) < np)
            gst<u32x4>(static_cast<char*>(t.out) + ((k0 + row) * pitch + bz * np + n0) * ES + 16 * c,
                       *reinterpret_cast<const u32x4*>(s_t + row * LP + (c ^ spread(row)) * 16));
    }
}

// Workgroup (block of columns, slice of rows); its waves take the slice's rows in turn, the
// next row in flight.
template <int XDT, int TAIL>
__device__ __forceinline__ void linear_dz(const LinearDz& a, int group, float (*s_sum)[kCols])
{
    const void *const dy = a.dy, *const z = a.z;
    void *const dz = a.dz, *const dz_out = a.dz_out;
    float* const part = a.part;
    const int act = a.act, slices = a.slices;
    const int64_t M = a.M, N = a.N, pitch = a.pitch;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int slice = group % slices;
    const int64_t block = group / slices;
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
__device__ __forceinline__ void gated_dz(const GatedDz& a, int group, int groups)
{
    const void *const dh = a.dh, *const g = a.g, *const u = a.u;
    void *const dz = a.dz, *const dg_out = a.dg_out, *const du_out = a.du_out;
    const int act = a.act, blocks = a.blocks;
    const int64_t M = a.M, N = a.N, pitch = a.pitch;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t block = group % blocks;
    const int64_t rows = (int64_t)groups / blocks * 4;
    const int units = (int)((N + 7) / 8), unit = (int)(block * 64 + lane);
    Unit<XDT> du, gu, uu;
    auto load_row = [&](int64_t m) {
        if (m >= M) return;
        du = load_row_unit<XDT, TAIL, true>(row_of<XDT>(dh, m, N), unit, units, (int)N);
        gu = load_row_unit<XDT, TAIL, true>(row_of<XDT>(g, m, N), unit, units, (int)N);
        uu = load_row_unit<XDT, TAIL, true>(row_of<XDT>(u, m, N), unit, units, (int)N);
    };
    int64_t m = (int64_t)(group / blocks) * 4 + wave;
    load_row(m);
    for (; m < M; m += rows) {
        float d[8], gv[8], uv[8], ad[8];
        unit_values<XDT, TAIL>(du, unit, (int)N, d);
        unit_values<XDT, TAIL>(gu, unit, (int)N, gv);
        unit_values<XDT, TAIL>(uu, unit, (int)N, uv);
        load_row(m + rows);
        // d u act'(g) and d act(g)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            ad[j] = d[j] * uv[j];
            uv[j] = d[j];
        }
        times_act_both<8>(act, gv, ad, uv);
        if (dz) {
            store_padded<XDT>(dz, m, pitch, unit, ad);
            store_padded<XDT>(static_cast<char*>(dz) + M * pitch * elem_bytes(XDT), m, pitch, unit, uv);
        }
        if (dg_out) store_plain<XDT>(dg_out, m, N, unit, ad);
        if (du_out) store_plain<XDT>(du_out, m, N, unit, uv);
    }
}

// The first `groups` workgroups of grid plane 0, by rows of gridDim.x, take dz, the rows of the
// grid behind them (dz_rows on) the weights; plane i the i-th weight.  One launch instead of two, in
// which the weights' latencies hide: 301 rows of 1056 x 2731 in binary32 16.6 -> 11.6 us, 2048 rows of
// 4096 x 4096 in bf16 26.1 -> 21.4, a gated block of 4096 rows, 4096 x 2 x 11008, 130 -> 120.
template <int XDT>
constexpr int kGradLds = 128 * 64 * (XDT == DT_F32 ? 4 : 2);       // the transposed tile; dz's sums take 8 KB

template <int XDT, bool DQ, int TAIL, class Dz>
__global__ __launch_bounds__(256) void k_grad_inputs(const Dz a, int groups, int dz_rows, const TransposedWeights t,
                                                     const QbTables* __restrict__ tab)
{
    __shared__ __attribute__((aligned(16))) char s_mem[kGradLds<XDT>];
    static_assert(kGradLds<XDT> >= kGradWaves * kCols * 4, "the sums of dz");
    if ((int)blockIdx.y < dz_rows) {
        const int group = (int)(blockIdx.y * gridDim.x + blockIdx.x);
        if (blockIdx.z != 0 || group >= groups) return;
        if constexpr (std::is_same_v<Dz, LinearDz>)
            linear_dz<XDT, TAIL>(a, group, reinterpret_cast<float(*)[kCols]>(s_mem));
        else
            gated_dz<XDT, TAIL>(a, group, groups);
    } else {
        unpack_transposed<XDT, DQ>(t, blockIdx.x, (int64_t)blockIdx.y - dz_rows, blockIdx.z, s_mem, tab);
    }
}

// Blocks of kCols columns that cover N columns and the padding.
int64_t column_blocks(int64_t N, int64_t pitch) { return ((pitch > N ? pitch : N) + kCols - 1) / kCols; }

template <int XDT, bool DQ, int TAIL, class Dz>
hipError_t grad_inputs_as(const Dz& a, int groups, const TransposedWeights& t, hipStream_t s)
{
    const QbTables* tab = device_tables();
    if (!tab) return hipErrorNotInitialized;
    const int64_t x = t.out ? (t.K + 127) / 128 : groups, rows = (groups + x - 1) / x, y = t.out ? (t.np + 63) / 64 : 0;
    if (x == 0) return hipSuccess;
    return launch_grid(k_grad_inputs<XDT, DQ, TAIL, Dz>, dim3((unsigned)x, (unsigned)(rows + y), t.out ? t.count : 1), 256,
                       0, s, a, groups, (int)rows, t, tab);
}

template <int XDT, int TAIL, class Dz>
hipError_t grad_inputs_tail(const Dz& a, int groups, const TransposedWeights& t, hipStream_t s)
{
    return t.out && t.f.nested ? grad_inputs_as<XDT, true, TAIL>(a, groups, t, s)
                               : grad_inputs_as<XDT, false, TAIL>(a, groups, t, s);
}

template <int XDT, class Dz>
hipError_t grad_inputs_dt(const Dz& a, int groups, const TransposedWeights& t, hipStream_t s)
{
    const int tail = tail_of(a.N);
    return tail == kWhole     ? grad_inputs_tail<XDT, kWhole>(a, groups, t, s)
           : tail == kPartial ? grad_inputs_tail<XDT, kPartial>(a, groups, t, s)
                              : grad_inputs_tail<XDT, kShort>(a, groups, t, s);
}

template <class Dz>
hipError_t grad_inputs(int xdt, const Dz& a, int64_t groups, const TransposedWeights* t, hipStream_t s)
{
    const TransposedWeights none{};
    switch (xdt) {
    case DT_F32: return grad_inputs_dt<DT_F32>(a, (int)groups, t ? *t : none, s);
    case DT_F16: return grad_inputs_dt<DT_F16>(a, (int)groups, t ? *t : none, s);
    default: return grad_inputs_dt<DT_BF16>(a, (int)groups, t ? *t : none, s);
    }
}

}  // namespace

hipError_t launch_linear_grad(int xdt, bool dz_too, const void* dy, const void* z, int act, int64_t M, int64_t N, void* dz,
                              int64_t pitch, void* dz_out, float* part, int slices, const TransposedWeights* t,
                              hipStream_t s)
{
    const LinearDz a{dy, z, dz, dz_out, part, M, N, pitch, act, slices};
    return grad_inputs(xdt, a, dz_too ? column_blocks(N, dz ? pitch : 0) * slices : 0, t, s);
}

hipError_t launch_gated_grad(int xdt, const void* dh, const void* g, const void* u, int act, int64_t M, int64_t N,
                             void* dz, int64_t pitch, void* dg_out, void* du_out, const TransposedWeights* t,
                             hipStream_t s)
{
    const int64_t blocks = column_blocks(N, dz ? pitch : 0), row_groups = (M + 3) / 4;
    const int64_t want = (4096 + blocks - 1) / blocks, take = row_groups < want ? row_groups : want;
    const GatedDz a{dh, g, u, dz, dg_out, du_out, M, N, pitch, act, (int32_t)blocks};
    return grad_inputs(xdt, a, blocks * take, t, s);
}

hipError_t launch_bias_sum(const float* part, int slices, int64_t N, bool accumulate, void* db, int bias_dt,
                           hipStream_t s)
{
    return launch_kernel_nt(k_bias_sum, (int)((N + 63) / 64), 64 * kSumWaves, s, part, slices, N, accumulate ? 1 : 0, db, bias_dt);
}

}  // namespace qb
