// qb_linear_grad.hip -- what the product of the 4-bit layers' gradients takes: the gradient
// at the pre-activation, padded to the product's steps, and the weights transposed, by one
// launch of two kinds of workgroups (neither needs the other).
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

// 64 rows n and 128 columns k of a weight, transposed into LDS rows k of 64 n (128 bytes, 256 in
// binary32), by 256 threads: 8 weights of two neighbouring rows a thread at a time.  16-byte
// chunk c of LDS row k lies at chunk c ^ spread(k): the threads of a wave, which hold 16 k eight
// apart and 4 row pairs, write to different banks but for two each, and 16 rows' equal chunks
// (16-bit types) are in different banks too.  (Rows padded by 16 bytes instead fell into one
// bank: 4096 x 4096 15.1 us for 9.6.)
template <int XDT, bool DQ>
struct TransposedTile {
    static constexpr int ES = XDT == DT_F32 ? 4 : 2;
    static constexpr int LP = 64 * ES, CPR = LP / 16;          // bytes and chunks of an LDS row
    uint32_t code[2][2], c2[2][2];                             // row pairs tid / 16 and tid / 16 + 16
    float a[2][2], mu;

    static __device__ __forceinline__ int spread(int k)
    {
        return XDT == DT_F32 ? ((k >> 3) & 7) * 2 : ((k >> 3) ^ k) & 7;
    }
    // Codes and constants of rows n0 .., columns k0 ..
    __device__ __forceinline__ void load(const TransposedWeights& t, const Weight4& w, int64_t n0, int64_t k0)
    {
        const int tid = threadIdx.x, kl = (tid & 15) * 8;
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int64_t n = n0 + 2 * ((tid >> 4) + 16 * i) + h, e = n * t.K + k0 + kl, blk = e >> t.f.log2B;
                code[i][h] = c2[i][h] = 0u;
                a[i][h] = 0.0f;
                if (n < t.N && k0 + kl < t.K) {
                    code[i][h] = gld<uint32_t>(w.codes + e / 2);
                    if constexpr (DQ) {
                        c2[i][h] = gld<uint8_t>(w.c2 + blk);
                        a[i][h] = gld<float>(w.absmax2 + (blk >> t.f.log2B2));
                    } else {
                        a[i][h] = gld<float>(w.absmax + blk);
                    }
                }
            }
        mu = DQ ? gld<float>(w.offset) : 0.0f;
    }
    // .. into s_t, zeros beyond the last row.
    __device__ __forceinline__ void fill(int64_t left, char* s_t, const float* s_val, const float* s_dyn) const
    {
        const int tid = threadIdx.x, kl = (tid & 15) * 8;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int pr = (tid >> 4) + 16 * i;
            Frag<DT_F32> v[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float c = DQ ? s_dyn[c2[i][h]] * a[i][h] + mu : a[i][h];       // two rounded operations
                dequant_frag<DT_F32>(code[i][h], 2 * pr + h < left ? c : 0.0f, s_val, v[h]);
            }
            const int at = 2 * pr * ES;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                char* const p = s_t + (kl + j) * LP + ((at / 16) ^ spread(kl + j)) * 16 + at % 16;
                if constexpr (XDT == DT_F32) {
                    typedef float f32x2_t __attribute__((ext_vector_type(2)));
                    *reinterpret_cast<f32x2_t*>(p) = f32x2_t{v[0].w[j], v[1].w[j]};
                } else {
                    *reinterpret_cast<uint32_t*>(p) = pack_two<XDT>(v[0].w[j], v[1].w[j]);
                }
            }
        }
    }
};

template <bool DQ>
__device__ __forceinline__ void stage_tables(const Weight4Format& f, const QbTables* tab, float* s_val, float* s_dyn)
{
    const int tid = threadIdx.x;
    if (tid < 16) s_val[tid] = (f.code4 == 0 ? tab->nf4 : tab->fp4)[tid];
    if constexpr (DQ) s_dyn[tid] = tab->dyn8[tid];
}

// A tile into out[k][n].
template <int XDT, bool DQ>
__device__ __forceinline__ void unpack_transposed(const TransposedWeights& t, int64_t bx, int64_t by, int bz, char* s_t,
                                                  const QbTables* tab)
{
    using Tile = TransposedTile<XDT, DQ>;
    constexpr int ES = Tile::ES, LP = Tile::LP, CPR = Tile::CPR;
    __shared__ float s_val[16];
    __shared__ float s_dyn[DQ ? 256 : 1];
    const int tid = threadIdx.x;
    const int64_t k0 = bx * 128, n0 = by * 64, pitch = t.np * t.count;
    Tile tile;
    tile.load(t, t.w[bz], n0, k0);
    stage_tables<DQ>(t.f, tab, s_val, s_dyn);
    __syncthreads();
    tile.fill(t.N - n0, s_t, s_val, s_dyn);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 128 * CPR / 256; ++i) {
        const int o = tid + 256 * i, row = o / CPR, c = o % CPR;
        if (k0 + row < t.K && n0 + c * (16 / ES) < t.np)
            gst<u32x4>(static_cast<char*>(t.out) + ((k0 + row) * pitch + bz * t.np + n0) * ES + 16 * c,
                       *reinterpret_cast<const u32x4*>(s_t + row * LP + (c ^ Tile::spread(row)) * 16));
    }
}

// Few rows (16 MT, 16-bit types): dx = dz W without the transposed weights in memory.  A workgroup
// takes 128 columns k of dx and a slice of the n (of both weights' n in a row): 64 of them at a time
// it transposes the weights' tile into LDS as above, beside it dz's rows, by direct loads, and its
// four waves multiply 32 columns each.  The slices' sums go to part[slice][M][K].  One row through
// 4096 x 4096 17 us in all (26 with the transposed weights in memory and the tiled product), 16 through
// a gated block of 4096 x 2 x 11008 43 (86), 64 through it 52 (92).
struct FewRows {
    const void* dz[2];
    int64_t M, ldz;
    float* part;
    int32_t tiles, per_slice;            // tiles of 64 n, of all weights; of a slice
};

template <int XDT, bool DQ, int MT>
__global__ __launch_bounds__(256) void k_few_rows_back(const FewRows a, const TransposedWeights t,
                                                       const QbTables* __restrict__ tab)
{
    using Tile = TransposedTile<XDT, DQ>;
    __shared__ __attribute__((aligned(16))) char s_t[128 * 128], s_a[16 * MT * 128];
    __shared__ float s_val[16];
    __shared__ float s_dyn[DQ ? 256 : 1];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int r = lane & 15, g = lane >> 4;
    const int64_t k0 = (int64_t)blockIdx.x * 128, M = a.M, K = t.K;
    const int per_weight = (int)(t.np / 64), begin = blockIdx.y * a.per_slice,
              end = a.tiles - begin < a.per_slice ? a.tiles : begin + a.per_slice;
    stage_tables<DQ>(t.f, tab, s_val, s_dyn);
    f32x4 acc[2][MT];
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int m = 0; m < MT; ++m) acc[j][m] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    for (int i = begin; i < end; ++i) {
        const int bz = i / per_weight;
        const int64_t n0 = (int64_t)(i - bz * per_weight) * 64;
        Tile tile;
        tile.load(t, t.w[bz], n0, k0);
        __syncthreads();                                 // the tile before has been read
        const char* const dz = static_cast<const char*>(a.dz[bz]) + n0 * 2;
#pragma unroll
        for (int l = 0; l < (2 * MT + 3) / 4; ++l) {     // 8 rows a load; chunk p of row i holds chunk p ^ (i % 8)
            const int at = l * 4 + wave;
            if (at < 2 * MT) {
                const int row = at * 8 + (lane >> 3), c = (lane & 7) ^ (row & 7);
                const int64_t m = row < M ? row : M - 1;
                __builtin_amdgcn_global_load_lds((gptr_t)(dz + m * a.ldz * 2 + c * 16), (lptr_t)(s_a + at * 1024), 16, 0, 0);
            }
        }
        tile.fill(t.N - n0, s_t, s_val, s_dyn);
        wait_loads<0>();
        __syncthreads();
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) {
            u32x4 b[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int row = 32 * wave + 16 * j + r;
                b[j] = *reinterpret_cast<const u32x4*>(s_t + row * 128 + ((4 * kk + g) ^ Tile::spread(row)) * 16);
            }
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                Frag<XDT> fa, fb;
                __builtin_memcpy(fa.w, s_a + (16 * m + r) * 128 + ((4 * kk + g) ^ (r & 7)) * 16, 16);
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    __builtin_memcpy(fb.w, &b[j], 16);
                    mma<XDT>(fb, fa, acc[j][m]);         // a lane's four sums: four columns of one row
                }
            }
        }
    }
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int64_t row = 16 * m + r, k = k0 + 32 * wave + 16 * j + 4 * g;
            if (row < M && k < K) gst<f32x4>(a.part + ((int64_t)blockIdx.y * M + row) * K + k, acc[j][m]);
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
    if (groups == 0 && !t.out) return hipSuccess;
    const int64_t x = t.out ? (t.K + 127) / 128 : groups, rows = (groups + x - 1) / x, y = t.out ? (t.np + 63) / 64 : 0;
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

namespace {

template <int XDT, bool DQ>
hipError_t few_rows_as(const FewRows& a, const TransposedWeights& t, dim3 grid, const QbTables* tab, hipStream_t s)
{
    if (a.M <= 16) return launch_grid(k_few_rows_back<XDT, DQ, 1>, grid, 256, 0, s, a, t, tab);
    if (a.M <= 32) return launch_grid(k_few_rows_back<XDT, DQ, 2>, grid, 256, 0, s, a, t, tab);
    return launch_grid(k_few_rows_back<XDT, DQ, 4>, grid, 256, 0, s, a, t, tab);
}

template <int XDT>
hipError_t few_rows_dq(const FewRows& a, const TransposedWeights& t, dim3 grid, const QbTables* tab, hipStream_t s)
{
    return t.f.nested ? few_rows_as<XDT, true>(a, t, grid, tab, s) : few_rows_as<XDT, false>(a, t, grid, tab, s);
}

}  // namespace

hipError_t launch_few_rows_back(int xdt, const void* dz0, const void* dz1, int64_t ldz, int64_t M,
                                const TransposedWeights& t, float* part, int* slices, hipStream_t s)
{
    const QbTables* tab = device_tables();
    if (!tab) return hipErrorNotInitialized;
    const int64_t tiles = t.np / 64 * t.count, x = (t.K + 127) / 128, fit = gemm_part_floats(M, t.K) / (M * t.K);
    // four workgroups a CU, as far as the slices go
    int64_t n = 1024 / x < tiles ? 1024 / x : tiles;
    n = n < 1 ? 1 : n > kSplitMax ? kSplitMax : n;
    n = n < fit ? n : fit;
    const int64_t per = (tiles + n - 1) / n;
    *slices = (int)((tiles + per - 1) / per);
    const FewRows a{{dz0, dz1}, M, ldz, part, (int32_t)tiles, (int32_t)per};
    const dim3 grid((unsigned)x, (unsigned)*slices);
    return xdt == DT_F16 ? few_rows_dq<DT_F16>(a, t, grid, tab, s) : few_rows_dq<DT_BF16>(a, t, grid, tab, s);
}

}  // namespace qb
