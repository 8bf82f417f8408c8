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

constexpr int kWaves = 8;
constexpr int kThreadsRows = 64 * kWaves;
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

// G weights; MT tiles of 16 rows of x; STAGED: x in LDS (dynamic, rows of whole steps).
template <int XDT, bool DQ, int G, int MT, bool STAGED>
__global__ __launch_bounds__(kThreadsRows) void k_linear_rows(const RowsArgs a, const QbTables* __restrict__ tab)
{
    static_assert(!STAGED || (MT == 1 && XDT != DT_F32), "staged rows: 16-bit, one tile");
    __shared__ float s_val[16];
    __shared__ float s_dyn[DQ ? 256 : 1];
    __shared__ float s_red[kWaves][G * MT][4][64];
    extern __shared__ u32x4 s_x[];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int r = lane & 15, g = lane >> 4;
    const int64_t n0 = (int64_t)blockIdx.x * 16, m0 = (int64_t)blockIdx.y * (16 * MT), M = a.M, K = a.K, N = a.e.N;
    // weight rows past N read row N - 1 (their sums are never stored)
    const int64_t rn = n0 + r < N ? n0 + r : N - 1;
    const int64_t e_lane = rn * K + 32 * g;             // the lane's first weight of step 0
    const int64_t steps = (K + kStepK - 1) / kStepK;

    struct Codes {
        u32x4 cw;
        uint32_t c;
        float a;
    };
    auto in_k = [&](int64_t s) { return s * kStepK + 32 * g < K; };
    auto load_codes = [&](Codes& p, const Weight4& w, int64_t s) {
        if (s >= steps || !in_k(s)) return;
        const int64_t e = e_lane + s * kStepK, blk = e >> a.f.log2B;
        p.cw = gld<u32x4>(w.codes + e / 2);
        if constexpr (DQ) {
            p.c = gld<uint8_t>(w.c2 + blk);
            p.a = gld<float>(w.absmax2 + (blk >> a.f.log2B2));
        } else {
            p.a = gld<float>(w.absmax + blk);
        }
    };
    Codes cur[G], next[G];
#pragma unroll
    for (int i = 0; i < G; ++i) load_codes(cur[i], a.w[i], wave);

    const int xs_row = (int)steps * (kStepK / 8) + kXsPad;     // staged: u32x4 of a row
    if constexpr (STAGED) {
        const int kc = (int)(K / 8);
        for (int i = tid; i < (int)M * xs_row; i += kThreadsRows) {
            const int row = i / xs_row, c = i - row * xs_row;
            s_x[i] = c < kc ? gld<u32x4>(static_cast<const char*>(a.x) + ((int64_t)row * kc + c) * 16)
                            : u32x4{0u, 0u, 0u, 0u};
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

    for (int64_t s = wave; s < steps; s += kWaves) {
#pragma unroll
        for (int i = 0; i < G; ++i) load_codes(next[i], a.w[i], s + kWaves);
        const bool kin = in_k(s);
        // rows of x past M, and k past K, are zero
        Frag<XDT> xf[MT][4];
#pragma unroll
        for (int t = 0; t < MT; ++t) {
            const int64_t m = m0 + 16 * t + r;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                if constexpr (STAGED) {
                    u32x4 v = {0u, 0u, 0u, 0u};
                    if (m < M) v = s_x[r * xs_row + s * (kStepK / 8) + 4 * g + q];
                    xf[t][q].w[0] = v.x; xf[t][q].w[1] = v.y; xf[t][q].w[2] = v.z; xf[t][q].w[3] = v.w;
                } else if (m < M && kin) {
                    load_frag<XDT>(a.x, m * K + s * kStepK + 32 * g + 8 * q, xf[t][q]);
                } else {
                    frag_zero<XDT>(xf[t][q]);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < G; ++i) {
            Frag<XDT> b[4];
            if (kin) {
                const float c = DQ ? s_dyn[cur[i].c] * cur[i].a + mu[i] : cur[i].a;    // two rounded operations
                dequant_chunk<XDT>(cur[i].cw, c, s_val, b);
            } else {
#pragma unroll
                for (int q = 0; q < 4; ++q) frag_zero<XDT>(b[q]);
            }
#pragma unroll
            for (int t = 0; t < MT; ++t)
#pragma unroll
                for (int q = 0; q < 4; ++q) mma<XDT>(xf[t][q], b[q], acc[i][t]);
            cur[i] = next[i];
        }
    }

    // the waves' partial tiles in wave order
#pragma unroll
    for (int i = 0; i < G; ++i)
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
            for (int j = 0; j < 4; ++j) s_red[wave][i * MT + t][j][lane] = acc[i][t][j];
    __syncthreads();
    for (int o = tid; o < MT * 256; o += kThreadsRows) {
        const int ml = o >> 4, nl = o & 15, t = ml >> 4, mm = ml & 15;
        const int l = (mm >> 2) * 16 + nl, j = mm & 3;      // C[m][n] of the tile: lane, element
        if (m0 + ml >= M || n0 + nl >= N) continue;
        float sum[G];
#pragma unroll
        for (int i = 0; i < G; ++i) {
            sum[i] = 0.0f;
#pragma unroll
            for (int w = 0; w < kWaves; ++w) sum[i] += s_red[w][i * MT + t][j][l];
        }
        if constexpr (G == 1) finish_linear1<XDT>(a.e, m0 + ml, n0 + nl, sum[0]);
        else finish_gated1<XDT>(a.e, m0 + ml, n0 + nl, sum[0], sum[1]);
    }
}

template <int XDT, bool DQ, int G>
hipError_t rows_as(const RowsArgs& a, const QbTables* tab, hipStream_t s)
{
    const int64_t gx = (a.e.N + 15) / 16, steps = (a.K + kStepK - 1) / kStepK;
    auto go = [&](auto kernel, size_t lds) {
        return launch_grid(kernel, dim3((unsigned)gx), kThreadsRows, lds, s, a, tab);
    };
    if constexpr (XDT != DT_F32) {
        if (a.M <= kXsRows && a.M * steps * kStepK * 2 <= kXsBytes)
            return go(k_linear_rows<XDT, DQ, G, 1, true>, (size_t)(a.M * (steps * (kStepK / 8) + kXsPad) * 16));
    }
    if (a.M <= 16) return go(k_linear_rows<XDT, DQ, G, 1, false>, 0);
    if (a.M <= 32) return go(k_linear_rows<XDT, DQ, G, 2, false>, 0);
    // 64 rows a workgroup; rows beyond a grid's in launches of their own
    constexpr int64_t kMost = 32768 * 64;
    constexpr int ES = XDT == DT_F32 ? 4 : 2;
    for (int64_t m = 0; m < a.M; m += kMost) {
        RowsArgs b = a;
        b.M = a.M - m < kMost ? a.M - m : kMost;
        b.x = static_cast<const char*>(a.x) + m * a.K * ES;
        b.e = epilogue_rows(a.e, m, ES);
        const dim3 grid((unsigned)gx, (unsigned)((b.M + 63) / 64));
        const hipError_t e = launch_grid(k_linear_rows<XDT, DQ, G, 4, false>, grid, kThreadsRows, 0, s, b, tab);
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
