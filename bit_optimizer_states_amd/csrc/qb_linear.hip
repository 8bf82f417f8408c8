// qb_linear.hip -- 4-bit layers of few rows: y = epilogue(x W^T), the weights dequantized
// in registers straight into MFMA operands, one weight (linear layer) or two that share x
// (gated block).
//
// One workgroup of 8 waves per 16 weight rows (of each weight) and up to 64 rows of x.
// A lane owns weight row n0 + lane % 16 and, per step of 128 k, the 32 consecutive k of its
// lane group (lane / 16): one 16-byte load of codes, one block constant, four 16x16x32
// MFMAs.  The waves take the steps of K in turn; their partial sums are added in wave order
// through LDS and finished there (same bits on every run).  Up to 8 rows of x are staged in
// LDS once per workgroup; a gated block's two weights share the fragments of x.
#include "qb_epilogue.h"
#include "qb_linear.h"
#include "qb_mm_device.h"

namespace qb {

namespace {

constexpr int kStepK = 128;                   // k of a wave's step: 4 lane groups x 32
constexpr int kXsPad = 4;                     // u32x4 of padding per staged row: 64 bytes
constexpr int kXsRows = 8;                    // rows of x that are staged in LDS ...
constexpr int64_t kXsBytes = 65536;           // ... while they take no more than this

struct RowsArgs {
    const void* x;
    int64_t M, K;
    Weight4 w[2];
    Weight4Format f;
    Epilogue e;
};

// Output (m, n) of one sum.
template <int XDT>
__device__ __forceinline__ void finish_linear1(const Epilogue& e, int64_t m, int64_t n, float z)
{
    const int64_t at = m * e.N + n;
    if (e.bias) z += e.bias_dt == DT_F32 ? load1<DT_F32>(e.bias, n) : e.bias_dt == DT_F16 ? load1<DT_F16>(e.bias, n)
                                                                                          : load1<DT_BF16>(e.bias, n);
    if (e.z) store1<XDT>(e.z, at, z);
    float y = act_value(e.act, z);
    if (e.residual) y += load1<XDT>(e.residual, at);
    store1<XDT>(e.y, at, y);
}

template <int XDT>
__device__ __forceinline__ void finish_gated1(const Epilogue& e, int64_t m, int64_t n, float g, float u)
{
    const int64_t at = m * e.N + n;
    if (e.z) store1<XDT>(e.z, at, g);
    if (e.u) store1<XDT>(e.u, at, u);
    store1<XDT>(e.y, at, act_value(e.act, g) * u);
}

// G weights; MT tiles of 16 rows of x; STAGED: x in LDS (rows of whole steps); WAVES waves
// share a column tile and take the steps in turn, the next step's codes in flight.
// LDS (dynamic): the staged rows, later the waves' sums.
// No load depends on a condition, so that the waits count loads exactly: steps past the
// last read the last one again (and are not multiplied), rows of x past M and weight rows
// past N read the last row (their sums are never stored), and in a last step that K fills
// in part the lanes behind K read their row's beginning of that step against zeros of x.
// Four waves a SIMD at least: at 131 VGPRs, three waves, the gated block of 8 rows (4096
// inputs, 2 x 11008 outputs) took 26.5 us instead of 21.3.  With conditional loads, which the
// waits cannot count, it took 26; with all of a wave's steps loaded at once 26; with pairs
// of neighbouring steps to a wave 28; two steps ahead 28.
template <int XDT, bool DQ, int G, int MT, bool STAGED, int WAVES>
__global__ __launch_bounds__(64 * WAVES, MT == 1 && XDT != DT_F32 ? 4 : 2) void k_linear_rows(const RowsArgs a, const QbTables* __restrict__ tab)
{
    static_assert(!STAGED || (MT == 1 && XDT != DT_F32), "staged rows: 16-bit, one tile");
    constexpr int ES = XDT == DT_F32 ? 4 : 2, NT = 64 * WAVES;
    __shared__ float s_val[16];
    __shared__ float s_dyn[DQ ? 256 : 1];
    extern __shared__ u32x4 s_x[];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int r = lane & 15, g = lane >> 4;
    const int64_t n0 = (int64_t)blockIdx.x * 16, m0 = (int64_t)blockIdx.y * (16 * MT), M = a.M, K = a.K, N = a.e.N;
    const int steps = (int)((K + kStepK - 1) / kStepK), last = steps - 1;
    const bool behind = last * kStepK + 32 * g >= (int)K;       // this lane in the last step
    // the lane's first weight of step 0, from the tile's first one
    const uint32_t e_lane = (uint32_t)((n0 + r < N ? r : (int)(N - 1 - n0)) * K + 32 * g);

    struct Codes {
        u32x4 cw;
        uint32_t c;
        float a;
    };
    // (element and block numbers are a uniform part, a whole number of blocks, and a 32-bit rest)
    auto load_codes = [&](Codes (&p)[G], int step) {
        const int s = step < last ? step : last;
        const int64_t e0 = n0 * K + (int64_t)s * kStepK, blk0 = e0 >> a.f.log2B;
        const uint32_t el = s == last && behind ? e_lane - 32 * g : e_lane;
        const uint32_t blk = (el + (uint32_t)(e0 - (blk0 << a.f.log2B))) >> a.f.log2B;
        const uint32_t blk2 = ((uint32_t)blk0 + blk) >> a.f.log2B2;
#pragma unroll
        for (int i = 0; i < G; ++i) {
            p[i].cw = ldo<u32x4>(a.w[i].codes + e0 / 2, el / 2);
            if constexpr (DQ) {
                p[i].c = ldo<uint8_t>(a.w[i].c2 + blk0, blk);
                p[i].a = ldo<float>(a.w[i].absmax2, blk2 * 4u);
            } else {
                p[i].a = ldo<float>(a.w[i].absmax + blk0, blk * 4u);
            }
        }
    };
    Codes codes[2][G];
    load_codes(codes[0], wave);

    // x: its rows staged (zeros behind K), or this lane's rows' beginnings
    const int xs_row = steps * (kStepK / 8) + kXsPad;          // u32x4 of a staged row
    const int mine = m0 + r < M ? r : (int)(M - 1 - m0);
    uint32_t x_off[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) {
        const int row = m0 + 16 * t + r < M ? 16 * t + r : (int)(M - 1 - m0);
        x_off[t] = (uint32_t)((row * K + 32 * g) * ES);
    }
    const char* const x_base = static_cast<const char*>(a.x) + m0 * K * ES;
    if constexpr (STAGED) {
        const int kc = (int)(K / 8);
        for (int i = tid; i < (int)M * xs_row; i += NT) {
            const int row = i / xs_row, c = i - row * xs_row;
            s_x[i] = c < kc ? ldo<u32x4>(a.x, (uint32_t)((row * kc + c) * 16)) : u32x4{0u, 0u, 0u, 0u};
        }
    }
    if (tid < 16) s_val[tid] = (a.f.code4 == 0 ? tab->nf4 : tab->fp4)[tid];
    if constexpr (DQ) {
        if (tid < 256) s_dyn[tid] = tab->dyn8[tid];
    }
    float mu[G];
#pragma unroll
    for (int i = 0; i < G; ++i) mu[i] = DQ ? gld<float>(a.w[i].offset) : 0.0f;
    __syncthreads();

    f32x4 acc[G][MT];
#pragma unroll
    for (int i = 0; i < G; ++i)
#pragma unroll
        for (int t = 0; t < MT; ++t) acc[i][t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

    auto load_x = [&](Frag<XDT> (&xf)[MT][4], int step) {
        const int s = step < last ? step : last;
        const char* const xs = x_base + (int64_t)s * kStepK * ES;
        const uint32_t back = s == last && behind ? 32u * g * ES : 0u;
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
            for (int q = 0; q < 4; ++q) load_frag_o<XDT>(xs, x_off[t] - back + (uint32_t)(8 * ES) * q, xf[t][q]);
    };
    auto multiply = [&](int s, const Codes (&cur)[G], Frag<XDT> (&xf)[MT][4]) {
        if constexpr (STAGED) {
            const u32x4* const xr = s_x + mine * xs_row + s * (kStepK / 8) + 4 * g;
#pragma unroll
            for (int q = 0; q < 4; ++q) __builtin_memcpy(xf[0][q].w, &xr[q], 16);
        } else if (s == last && (K % kStepK) != 0) {
#pragma unroll
            for (int t = 0; t < MT; ++t)
#pragma unroll
                for (int q = 0; q < 4; ++q)
#pragma unroll
                    for (int j = 0; j < (XDT == DT_F32 ? 8 : 4); ++j)
                        xf[t][q].w[j] = behind ? 0 : xf[t][q].w[j];
        }
#pragma unroll
        for (int i = 0; i < G; ++i) {
            const float c = DQ ? s_dyn[cur[i].c] * cur[i].a + mu[i] : cur[i].a;    // two rounded operations
            Frag<XDT> b[4];
            dequant_chunk<XDT>(cur[i].cw, c, s_val, b);
#pragma unroll
            for (int t = 0; t < MT; ++t)
#pragma unroll
                for (int q = 0; q < 4; ++q) mma<XDT>(xf[t][q], b[q], acc[i][t]);
        }
    };
    // (the barriers keep the loads in front of the products, behind which the compiler moves them)
    Frag<XDT> xf[MT][4];
    int s = wave;
    for (; s + 2 * WAVES < steps; s += 2 * WAVES) {
#pragma unroll
        for (int d = 0; d < 2; ++d) {
            if constexpr (!STAGED) load_x(xf, s + d * WAVES);
            load_codes(codes[d ^ 1], s + (d + 1) * WAVES);
            __builtin_amdgcn_sched_barrier(0);
            multiply(s + d * WAVES, codes[d], xf);
        }
    }
    if (s + WAVES < steps) {
        if constexpr (!STAGED) load_x(xf, s);
        load_codes(codes[1], s + WAVES);
        __builtin_amdgcn_sched_barrier(0);
        multiply(s, codes[0], xf);
        s += WAVES;
        if constexpr (!STAGED) load_x(xf, s);
        multiply(s, codes[1], xf);
    } else if (s < steps) {
        if constexpr (!STAGED) load_x(xf, s);
        multiply(s, codes[0], xf);
    }

    // the waves' partial tiles in wave order
    float* const s_red = reinterpret_cast<float*>(s_x);      // [WAVES][G * MT][4][64]
    if constexpr (STAGED) __syncthreads();
#pragma unroll
    for (int i = 0; i < G; ++i)
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
            for (int j = 0; j < 4; ++j) s_red[((wave * G * MT + i * MT + t) * 4 + j) * 64 + lane] = acc[i][t][j];
    __syncthreads();
    for (int o = tid; o < MT * 256; o += NT) {
        const int ml = o >> 4, nl = o & 15, t = ml >> 4, mm = ml & 15;
        const int l = (mm >> 2) * 16 + nl, j = mm & 3;      // C[m][n] of the tile: lane, element
        if (m0 + ml >= M || n0 + nl >= N) continue;
        float sum[G];
#pragma unroll
        for (int i = 0; i < G; ++i) {
            sum[i] = 0.0f;
#pragma unroll
            for (int w = 0; w < WAVES; ++w) sum[i] += s_red[((w * G * MT + i * MT + t) * 4 + j) * 64 + l];
        }
        if constexpr (G == 1) finish_linear1<XDT>(a.e, m0 + ml, n0 + nl, sum[0]);
        else finish_gated1<XDT>(a.e, m0 + ml, n0 + nl, sum[0], sum[1]);
    }
}

template <int XDT, bool DQ, int G>
hipError_t rows_as(const RowsArgs& a, const QbTables* tab, hipStream_t s)
{
    const int64_t gx = (a.e.N + 15) / 16, steps = (a.K + kStepK - 1) / kStepK;
    // the staged rows, and at least the waves' sums
    auto lds_bytes = [&](bool staged, int waves, int mt) {
        const size_t x = staged ? (size_t)(a.M * (steps * (kStepK / 8) + kXsPad) * 16) : 0, sums = (size_t)waves * G * mt * 1024;
        return x > sums ? x : sums;
    };
    if constexpr (XDT != DT_F32) {
        if (a.M <= kXsRows && a.M * steps * kStepK * 2 <= kXsBytes) {
            // fewer column tiles than 1.5 a CU take twice the waves each
            if (gx < 384)
                return launch_grid(k_linear_rows<XDT, DQ, G, 1, true, 16>, dim3((unsigned)gx), 1024,
                                   lds_bytes(true, 16, 1), s, a, tab);
            return launch_grid(k_linear_rows<XDT, DQ, G, 1, true, 8>, dim3((unsigned)gx), 512, lds_bytes(true, 8, 1), s,
                               a, tab);
        }
    }
    if (a.M <= 16)
        return launch_grid(k_linear_rows<XDT, DQ, G, 1, false, 8>, dim3((unsigned)gx), 512, lds_bytes(false, 8, 1), s,
                           a, tab);
    if (a.M <= 32)
        return launch_grid(k_linear_rows<XDT, DQ, G, 2, false, 8>, dim3((unsigned)gx), 512, lds_bytes(false, 8, 2), s,
                           a, tab);
    // 64 rows a workgroup; rows beyond a grid's in launches of their own
    constexpr int64_t kMost = 32768 * 64;
    constexpr int ES = XDT == DT_F32 ? 4 : 2;
    for (int64_t m = 0; m < a.M; m += kMost) {
        RowsArgs b = a;
        b.M = a.M - m < kMost ? a.M - m : kMost;
        b.x = static_cast<const char*>(a.x) + m * a.K * ES;
        b.e = epilogue_rows(a.e, m, ES);
        const dim3 grid((unsigned)gx, (unsigned)((b.M + 63) / 64));
        const hipError_t e = launch_grid(k_linear_rows<XDT, DQ, G, 4, false, 8>, grid, 512, lds_bytes(false, 8, 4), s, b, tab);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

template <int XDT>
hipError_t rows_dq(const RowsArgs& a, int count, const QbTables* tab, hipStream_t s)
{
    if (a.f.nested) return count == 2 ? rows_as<XDT, true, 2>(a, tab, s) : rows_as<XDT, true, 1>(a, tab, s);
    return count == 2 ? rows_as<XDT, false, 2>(a, tab, s) : rows_as<XDT, false, 1>(a, tab, s);
}

}  // namespace

hipError_t launch_linear_rows(int xdt, const void* x, int64_t M, int64_t K, const Weight4* w, int count,
                              const Weight4Format& f, const Epilogue& e, hipStream_t s)
{
    const QbTables* tab = device_tables();
    if (!tab) return hipErrorNotInitialized;
    const RowsArgs a{x, M, K, {w[0], w[count - 1]}, f, e};
    switch (xdt) {
    case DT_F32: return rows_dq<DT_F32>(a, count, tab, s);
    case DT_F16: return rows_dq<DT_F16>(a, count, tab, s);
    default: return rows_dq<DT_BF16>(a, count, tab, s);
    }
}

}  // namespace qb
