// qb_linear.hip -- 4-bit layers of few rows: y = epilogue(x W^T), the weights dequantized
// in registers straight into MFMA operands, one weight (linear layer) or two that share x
// (gated block).
//
// One workgroup of 8 or 16 waves per 16 weight rows (of each weight) and up to 64 rows of x.
// A lane owns weight row n0 + lane % 16 and, per step of 128 k, the 32 consecutive k of its
// lane group (lane / 16): 16 bytes of codes, one block constant, four 16x16x32 MFMAs.  The
// waves take the steps of K in turn; their partial sums are added in wave order through LDS
// and finished there (same bits on every run).  A gated block's two weights share the
// fragments of x.
//
// Codes and x reach LDS by direct global-to-LDS loads, a step ahead, into a slot that each
// wave keeps for itself: four lanes a row of codes, 16 a row of x, where loads into the
// fragments' lanes touch 16 rows at once and the address unit takes them one row at a time (64
// rows of 11008 x 4096: 47 us with loads to registers, 25 so; one row 10.0 both ways).  The
// block constants of the tile's rows are decoded into LDS once, for up to 12288 k.  What
// bounds it now: one row of 11008 x 4096 takes 10.2 us, 23.3 MB at 2.3 TB/s (from HBM hardly more than
// from the cache: 9.8 and 9.6 us a call), where the lookups and products of the 4-bit codes alone, 3 vector
// instructions and one LDS read a weight, take 5 us of the SIMDs; at 64 rows of 4096 x 11008 (28 us, 32 with
// the weights from HBM) it is x through LDS, 688 times over.
#include "qb_epilogue.h"
#include "qb_linear.h"
#include "qb_mm_device.h"

namespace qb {

namespace {

constexpr int kStepK = 128;                   // k of a wave's step: 4 lane groups x 32

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

// Block constants of a row and `part` (or all K) k in LDS: one more where the row begins
// inside a block; an odd number.
__host__ __device__ inline int const_pitch(int64_t K, int part, int log2B)
{
    const int64_t k = K < part ? K : part;
    return (int)(((k + (int64_t(1) << log2B) - 1) >> log2B) + 1) | 1;
}

template <int XDT, int G, int XR, int WAVES>
struct RowsShape {
    static constexpr int MT = XR < 16 ? 1 : XR / 16;
    static constexpr int ES = XDT == DT_F32 ? 4 : 2;
    static constexpr int XL = XR * kStepK * ES / 1024;               // loads of a step's rows of x
    static constexpr int SLOT = (G + XL) * 1024, SLOTS = WAVES * SLOT;
    // k whose block constants (blocks of 64) are in LDS at once, beside the slots: 160 KB in all
    static constexpr int PART = SLOTS + G * 16 * (12288 / 64 + 1) * 4 <= 160000 ? 12288 : 6144;
    static_assert(SLOTS + G * 16 * (PART / 64 + 1) * 4 <= 160000, "LDS");
    static_assert(PART % (kStepK * WAVES) == 0, "whole turns of the waves");
    static_assert(SLOTS >= WAVES * G * MT * 1024, "the waves' sums take the slots' place");
};

// Waves a SIMD that the registers must leave room for.  Six of one weight hold three workgroups
// of 8 waves a CU: the 688 tiles of 11008 outputs all at once (16 rows of 4096 inputs: 13.3 us
// with four, 12.2 so).  Two weights do not fit (23.7 us for 18.7).
constexpr int rows_waves(int xdt, int G, int XR, int WAVES)
{
    return G == 1 && XR <= 16 && WAVES == 8 && xdt != DT_F32 ? 6 : WAVES == 16 || (XR <= 16 && xdt != DT_F32) ? 4 : 2;
}

template <int XDT, bool DQ, int G, int XR, int WAVES>
__global__ __launch_bounds__(64 * WAVES, rows_waves(XDT, G, XR, WAVES)) void k_linear_rows(const RowsArgs a, const QbTables* __restrict__ tab)
{
    using Shape = RowsShape<XDT, G, XR, WAVES>;
    constexpr int MT = Shape::MT, ES = Shape::ES, NT = 64 * WAVES, XL = Shape::XL;
    constexpr int CPR = kStepK * ES / 16, RPL = 64 / CPR;    // 16-byte chunks of a row's step; rows of a load
    constexpr int PART = Shape::PART / kStepK / WAVES;
    __shared__ float s_val[16];
    __shared__ float s_dyn[DQ ? 256 : 1];
    __shared__ __attribute__((aligned(16))) char s_zero[16];
    extern __shared__ __attribute__((aligned(16))) char s_mem[];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int r = lane & 15, g = lane >> 4;
    const int64_t n0 = (int64_t)blockIdx.x * 16, m0 = (int64_t)blockIdx.y * XR, M = a.M, K = a.K, N = a.e.N;
    const int steps = (int)((K + kStepK - 1) / kStepK), last = steps - 1;
    // the last row of the tile and of x, from the first one
    const int rows_n = N - n0 < 16 ? (int)(N - n0) - 1 : 15, rows_m = M - m0 < XR ? (int)(M - m0) - 1 : XR - 1;
    const int pitch = const_pitch(K, Shape::PART, a.f.log2B);
    char* const slot = s_mem + wave * Shape::SLOT;
    float* const s_const = reinterpret_cast<float*>(s_mem + Shape::SLOTS);     // [G][16][pitch]

    // A wave's loads: of a column tile's step one of 16 rows (4 lanes a row), of x RPL rows each.
    // Chunk p of row i holds chunk p ^ (i / 4) (codes), p ^ (i % 16) (x) of the row's step, so that
    // 16 rows' equal chunks lie in different banks.  Rows past the end are the last one again; chunks
    // past K the step's first one (x and the weights are taken as zeros there).
    const int cc = (lane & 3) ^ (lane >> 4);
    const uint32_t c_off = (uint32_t)min(lane >> 2, rows_n) * (uint32_t)(K / 2) + 16 * cc;
    uint32_t x_off[XL];
#pragma unroll
    for (int i = 0; i < XL; ++i) {
        const int row = i * RPL + lane / CPR;
        x_off[i] = (uint32_t)min(row, rows_m) * (uint32_t)(K * ES) + ((lane % CPR) ^ (row & 15)) * 16;
    }
    const char* const x_base = static_cast<const char*>(a.x) + m0 * K * ES;
    auto load = [&](int s) {
        const int left = (int)(K - (int64_t)s * kStepK);                      // k of the step
#pragma unroll
        for (int i = 0; i < G; ++i)
            __builtin_amdgcn_global_load_lds(
                (gptr_t)(a.w[i].codes + (n0 * K + (int64_t)s * kStepK) / 2 + (32 * cc < left ? c_off : c_off - 16 * cc)),
                (lptr_t)(slot + i * 1024), 16, 0, 0);
        const char* const xs = x_base + (int64_t)s * kStepK * ES;
#pragma unroll
        for (int i = 0; i < XL; ++i) {
            const int c = (lane % CPR) ^ ((i * RPL + lane / CPR) & 15);
            __builtin_amdgcn_global_load_lds((gptr_t)(xs + (c * 16 < left * ES ? x_off[i] : x_off[i] - c * 16)),
                                             (lptr_t)(slot + (G + i) * 1024), 16, 0, 0);
        }
    };
    // The constants of the k from k0 on, of all rows of the tile, NT / 16 threads to a row: AHEAD
    // of them a thread are asked for at once, and decoded when they are there.
    constexpr int TPR = NT / 16, AHEAD = 3;
    struct Constant {
        uint32_t c;
        float a;
    };
    float mu[G];
#pragma unroll
    for (int i = 0; i < G; ++i) mu[i] = DQ ? gld<float>(a.w[i].offset) : 0.0f;
    const int c_row = tid / TPR, c_at = tid % TPR;
    Constant ahead[G][AHEAD];
    int64_t blk0;                  // this thread's row's first block of the part,
    int blocks;                    // and how many there are
    auto ask = [&](int i, int j, Constant& v) {
        const Weight4& w = a.w[i];
        const int64_t blk = blk0 + min(j, blocks - 1);
        if constexpr (DQ) {
            v.c = gld<uint8_t>(w.c2 + blk);
            v.a = gld<float>(w.absmax2 + (blk >> a.f.log2B2));
        } else {
            v.a = gld<float>(w.absmax + blk);
        }
    };
    auto keep = [&](int i, int j, const Constant& v) {
        if (j < blocks)
            s_const[(i * 16 + c_row) * pitch + j] = DQ ? s_dyn[v.c] * v.a + mu[i] : v.a;    // two rounded operations
    };
    auto ask_first = [&](int64_t k0) {
        const int64_t part = K - k0 < Shape::PART ? K - k0 : Shape::PART;
        const int64_t e = (n0 + min(c_row, rows_n)) * K + k0;
        blk0 = e >> a.f.log2B;
        blocks = (int)(((e + part - 1) >> a.f.log2B) - blk0) + 1;
#pragma unroll
        for (int i = 0; i < G; ++i)
#pragma unroll
            for (int j = 0; j < AHEAD; ++j) ask(i, c_at + j * TPR, ahead[i][j]);
    };
    auto keep_all = [&]() {
#pragma unroll
        for (int i = 0; i < G; ++i) {
#pragma unroll
            for (int j = 0; j < AHEAD; ++j) keep(i, c_at + j * TPR, ahead[i][j]);
#pragma unroll 1
            for (int j = c_at + AHEAD * TPR; j < blocks; j += TPR) {
                Constant v;
                ask(i, j, v);
                keep(i, j, v);
            }
        }
    };
    // a wave takes the steps wave, wave + WAVES, ..: `mine` of them
    const int mine = wave < steps ? (steps - wave + WAVES - 1) / WAVES : 0;
    float tables[2];
    if (tid < 16) tables[0] = (a.f.code4 == 0 ? tab->nf4 : tab->fp4)[tid];
    if constexpr (DQ) {
        if (tid < 256) tables[1] = tab->dyn8[tid];
    }
    ask_first(0);
    __builtin_amdgcn_sched_barrier(0);
    load(wave < last ? wave : last);
    __builtin_amdgcn_sched_barrier(0);
    if (tid < 4) reinterpret_cast<uint32_t*>(s_zero)[tid] = 0u;
    if (tid < 16) s_val[tid] = tables[0];
    if constexpr (DQ) {
        if (tid < 256) s_dyn[tid] = tables[1];
        pipeline_barrier();
    }

    f32x4 acc[G][MT];
#pragma unroll
    for (int i = 0; i < G; ++i)
#pragma unroll
        for (int t = 0; t < MT; ++t) acc[i][t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

    // every wave takes `turns` turns (the last one may find no step left)
    const int turns = (steps + WAVES - 1) / WAVES;
    const int xr = r & (XR < 16 ? XR - 1 : 15);
    uint32_t first = 0;            // of the lane's weights among the part's constants, in elements
#pragma unroll 1
    for (int turn = 0, in_part = 0; turn < turns; ++turn) {
        if (in_part == 0) {
            const int64_t k0 = (int64_t)turn * WAVES * kStepK;
            if (turn) {
                ask_first(k0);
                pipeline_barrier();
            }
            keep_all();
            first = ((uint32_t)((n0 + min(r, rows_n)) * K + k0) & ((1u << a.f.log2B) - 1)) + wave * kStepK + 32 * g;
            pipeline_barrier();
        }
        const int s = turn * WAVES + wave;
        if (turn < mine) {
            const bool zeros = s == last && s * kStepK + 32 * g >= (int)K;
            wait_loads<0>();
            asm volatile("" ::: "memory");
            u32x4 code[G];
            float constant[G];
            Frag<XDT> xf[MT][4];
#pragma unroll
            for (int i = 0; i < G; ++i) {
                code[i] = *reinterpret_cast<const u32x4*>(slot + i * 1024 + r * 64 + (g ^ (r >> 2)) * 16);
                // lanes past K: weights of zero too (an infinite constant times x's zero would be NaN)
                const float c = s_const[(i * 16 + r) * pitch + ((zeros ? first - 32 * g : first) >> a.f.log2B)];
                constant[i] = zeros ? 0.0f : c;
            }
#pragma unroll
            for (int t = 0; t < MT; ++t)
#pragma unroll
                for (int q = 0; q < 4; ++q)
#pragma unroll
                    for (int h = 0; h < ES / 2; ++h) {
                        const char* const at = slot + G * 1024 + ((16 * t + xr) * CPR + (((g * 4 + q) * (ES / 2) + h) ^ xr)) * 16;
                        __builtin_memcpy(&xf[t][q].w[4 * h], zeros ? s_zero : at, 16);
                    }
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");       // read before they are overwritten
            if (turn + 1 < mine) load(s + WAVES);
            // the next eight weights' values are looked up while these are multiplied
            float value[2][8];
            code_values(code[0][0], s_val, value[0]);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int q = 0; q < 4 * G; ++q) {
                if (q + 1 < 4 * G) code_values(code[(q + 1) / 4][(q + 1) % 4], s_val, value[(q + 1) & 1]);
                __builtin_amdgcn_sched_barrier(0);
                Frag<XDT> b;
                scaled<XDT>(value[q & 1], constant[q / 4], b);
#pragma unroll
                for (int t = 0; t < MT; ++t) mma<XDT>(xf[t][q % 4], b, acc[q / 4][t]);
            }
        }
        in_part = in_part + 1 == PART ? 0 : in_part + 1;
        first += WAVES * kStepK;
    }

    wait_loads<0>();               // (a wave without a step asked for one all the same)
    // the waves' partial tiles in wave order
    float* const s_red = reinterpret_cast<float*>(s_mem);     // [WAVES][G * MT][4][64]
    __syncthreads();
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

// XR rows of x to a workgroup: 4 and 8 where there are no more (they load less), else whole tiles
// of 16.
template <int XDT, bool DQ, int G, int XR, int WAVES>
hipError_t rows_launch(const RowsArgs& a, const QbTables* tab, hipStream_t s)
{
    using Shape = RowsShape<XDT, G, XR, WAVES>;
    const size_t lds = Shape::SLOTS + (size_t)G * 16 * const_pitch(a.K, Shape::PART, a.f.log2B) * 4;
    // rows beyond a grid's in launches of their own
    constexpr int64_t kMost = 32768 * XR;
    for (int64_t m = 0; m < a.M; m += kMost) {
        RowsArgs b = a;
        b.M = a.M - m < kMost ? a.M - m : kMost;
        b.x = static_cast<const char*>(a.x) + m * a.K * Shape::ES;
        b.e = epilogue_rows(a.e, m, Shape::ES);
        const dim3 grid((unsigned)((a.e.N + 15) / 16), (unsigned)((b.M + XR - 1) / XR));
        const hipError_t e = launch_grid(k_linear_rows<XDT, DQ, G, XR, WAVES>, grid, 64 * WAVES, lds, s, b, tab);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

// Beyond 32 rows: blocks of 48 where those of 64 are not fewer.
int rows_of_block(int64_t M) { return (M + 47) / 48 == (M + 63) / 64 ? 48 : 64; }

template <int XDT, bool DQ, int G>
hipError_t rows_as(const RowsArgs& a, const QbTables* tab, hipStream_t s)
{
    const int64_t gx = (a.e.N + 15) / 16;
    if constexpr (XDT == DT_F32) {
        if (a.M <= 16) return rows_launch<XDT, DQ, G, 16, 8>(a, tab, s);
        return rows_launch<XDT, DQ, G, 32, 8>(a, tab, s);
    } else {
        // fewer column tiles than 1.5 a CU take twice the waves each (16 rows of 11008 x 4096, 256 tiles: 13.3 us
        // with 8, 11.2 with 16; of 4096 x 11008, 688 tiles, one row 10.4 and 13.6).  Beyond 16 rows their slots
        // leave no room.
        if (gx < 384) {
            if (a.M <= 4) return rows_launch<XDT, DQ, G, 4, 16>(a, tab, s);
            if (a.M <= 8) return rows_launch<XDT, DQ, G, 8, 16>(a, tab, s);
            if (a.M <= 16) return rows_launch<XDT, DQ, G, 16, 16>(a, tab, s);
        }
        if (a.M <= 4) return rows_launch<XDT, DQ, G, 4, 8>(a, tab, s);
        if (a.M <= 8) return rows_launch<XDT, DQ, G, 8, 8>(a, tab, s);
        if (a.M <= 16) return rows_launch<XDT, DQ, G, 16, 8>(a, tab, s);
        if (a.M <= 32) return rows_launch<XDT, DQ, G, 32, 8>(a, tab, s);
        if (rows_of_block(a.M) == 48) return rows_launch<XDT, DQ, G, 48, 8>(a, tab, s);
        return rows_launch<XDT, DQ, G, 64, 8>(a, tab, s);
    }
}

template <int XDT>
hipError_t rows_dq(const RowsArgs& a, int count, const QbTables* tab, hipStream_t s)
{
    if (a.f.nested) return count == 2 ? rows_as<XDT, true, 2>(a, tab, s) : rows_as<XDT, true, 1>(a, tab, s);
    return count == 2 ? rows_as<XDT, false, 2>(a, tab, s) : rows_as<XDT, false, 1>(a, tab, s);
}

}  // namespace

// A launch, and rounds of one workgroup a CU (fitted to 65 .. 384 rows of layers of 512 .. 11008
// inputs and 1001 .. 11008 outputs).
double rows_us(int xdt, int64_t M, int64_t K, int64_t N, int count)
{
    const int block = xdt == DT_F32 ? 32 : rows_of_block(M);
    const double fixed = xdt == DT_F32 ? 2.4 : count == 2 ? 4.0 : 2.5,
                 each = (xdt == DT_F32 ? 2.9 * count : count == 2 ? 2.05 : 1.8) * K / 1024;
    const int64_t rounds = ((N + 15) / 16 * ((M + block - 1) / block) + 255) / 256;
    return 3.0 + rounds * (fixed + each) * (block == 48 ? 0.87 : 1.0);
}

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
