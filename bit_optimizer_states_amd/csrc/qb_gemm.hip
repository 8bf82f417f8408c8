// qb_gemm.hip -- the tiled matrix product behind the 4-bit layers of many rows.
//
// From a few hundred rows on the products bound the layer, not the weights: each
// weight is dequantized once into a workspace in the compute dtype (N K elements written
// and read back), and C = A B^T runs at the matrix instructions' rate, with the layer's
// epilogue on the binary32 sums.
#include "qb_linear.h"
#include "qb_mm_device.h"
#include "qb_epilogue.h"

namespace qb {

namespace {

int64_t tiles_over(int64_t n, int64_t tile) { return (n + tile - 1) / tile; }

// ---------------------------------------------------------------------------
// C = A B^T
// ---------------------------------------------------------------------------
//
// A workgroup of WM x WN waves computes BM rows (of A) by BN columns (rows of B), each
// wave BM / WM by BN / WN of them in 16x16 tiles.  A step is 128 bytes of every row (64
// 16-bit elements, 32 binary32 ones), staged in LDS by direct global-to-LDS loads of 16
// bytes a lane, STAGES buffers in turn: the next steps load while one is multiplied.  16-byte
// chunk p of an LDS row holds chunk p ^ (row % 8) of the operand's row, so that the rows
// of one fragment lie in different banks.  A fragment is one chunk a lane: row lane % 16,
// chunk 4 kk + lane / 16; with binary32 its four elements go to four instructions, the same
// k order in both operands.  A step's first half of fragments is in registers when it begins;
// the second half's reads are dealt among the first half's products, then the waves meet, and
// the next step's first half and the loads are dealt among the second half's.
// The whole layer of 4096 x 11008 x 4096 bf16 takes 312 us so, 24 of them the dequantization.
// Beside runs of 308: 319 with the waves meeting at the beginning of a step, all fragments read before the products
// 8 us more, the loads first and each half read before its products 28 more.  The matrix pipes
// are busy 78% of the cycles (67% with the waves meeting at the beginning), and the clock falls
// as that rises, 1.75 to 1.6 GHz: what is left is power.  32x32x16 instructions 330; steps of half the
// length in four buffers, four waves of 128 x 128 each, two groups of waves kept half a step apart:
// equal or slower.
// B's fragment is the first operand, so that a lane's four sums are four neighbouring
// columns of C.

struct GemmParams {
    GemmArgs g;
    Epilogue e;
    float* part;                 // partial sums [split][M][R] of a product split over its length
    int32_t steps, steps0, half, tiles_m, tiles_n, split, per_split;
    int64_t n_first;             // first row of B
};

template <int XDT>
__device__ __forceinline__ void mma_chunk(const u32x4& a, const u32x4& b, f32x4& acc)
{
    if constexpr (XDT == DT_BF16) {
        bf16x8 av, bv;
        __builtin_memcpy(&av, &a, 16);
        __builtin_memcpy(&bv, &b, 16);
        acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(av, bv, acc, 0, 0, 0);
    } else if constexpr (XDT == DT_F16) {
        f16x8 av, bv;
        __builtin_memcpy(&av, &a, 16);
        __builtin_memcpy(&bv, &b, 16);
        acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(av, bv, acc, 0, 0, 0);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) acc = __builtin_amdgcn_mfma_f32_16x16x4f32(ffrom(a[i]), ffrom(b[i]), acc, 0, 0, 0);
    }
}

// Binary32 word of column group n4 (four columns) of row m of a staged tile of BN columns:
// groups are exchanged within eight by the row, so that neither the lanes that write a
// column group of 16 rows nor those that read a row meet in a bank.
template <int BN>
__device__ __forceinline__ int staged_word(int m, int n4)
{
    return m * BN + 4 * (n4 ^ (m & 7));
}

// The epilogue of `rows` staged rows (m0 onwards) of BN columns (of B: n0 onwards), 8
// outputs a thread at a time; a thread stays in its columns, and the residual is read
// two turns ahead.
template <int XDT, int BN, int NT, bool GATED>
__device__ __forceinline__ void finish_rows(const Epilogue& e, const float* tile, int rows, int64_t m0, int64_t n0,
                                            int64_t M)
{
    constexpr int TPR = BN / (GATED ? 16 : 8), STEP = NT / TPR;     // threads of a row, rows at a time
    const int tid = threadIdx.x, q = tid % TPR;
    const int64_t n = GATED ? n0 / 2 + q * 8 : n0 + q * 8;
    const int cnt = columns_left8(n, e.N);
    if (cnt == 0) return;
    const int last = M - m0 < rows ? (int)(M - m0) : rows;
    if constexpr (GATED) {
        const int g4 = (q >> 1) * 8 + (q & 1) * 2;         // the gate's column group; the up's is 4 further
#pragma unroll 1
        for (int row = tid / TPR; row < last; row += STEP) {
            float g[8], u[8];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                *reinterpret_cast<f32x4*>(g + 4 * h) = *reinterpret_cast<const f32x4*>(tile + staged_word<BN>(row, g4 + h));
                *reinterpret_cast<f32x4*>(u + 4 * h) =
                    *reinterpret_cast<const f32x4*>(tile + staged_word<BN>(row, g4 + 4 + h));
            }
            finish_gated8<XDT>(e, m0 + row, n, cnt, g, u);
        }
    } else {
        float bias[8];
        load_bias8(e, n, cnt, bias);
        float r0[8], r1[8];
        auto residual = [&](int row, float* r) {
            if (e.residual && row < last) load_up_to8<XDT>(e.residual, (m0 + row) * e.N + n, cnt, r);
        };
        residual(tid / TPR, r0);
        residual(tid / TPR + STEP, r1);
#pragma unroll 1
        for (int row = tid / TPR; row < last; row += STEP) {
            float z[8], r[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                r[j] = r0[j];
                r0[j] = r1[j];
            }
            residual(row + 2 * STEP, r1);
#pragma unroll
            for (int h = 0; h < 2; ++h)
                *reinterpret_cast<f32x4*>(z + 4 * h) = *reinterpret_cast<const f32x4*>(tile + staged_word<BN>(row, 2 * q + h));
            finish_linear8<XDT>(e, m0 + row, n, cnt, z, bias, r);
        }
    }
}

template <int XDT, int BM, int BN, int WM, int WN, int STAGES, bool GATED>
__global__ __launch_bounds__(64 * WM * WN) void k_gemm(const GemmParams p)
{
    constexpr int NW = WM * WN, NT = 64 * NW;          // waves, threads
    constexpr int TM = BM / WM / 16, TN = BN / WN / 16;   // 16x16 tiles of a wave
    constexpr int A_PER = BM / 8 / NW, B_PER = BN / 8 / NW;   // loads (8 rows each) of a wave and step
    static_assert(A_PER * NW * 8 == BM && B_PER * NW * 8 == BN, "whole loads");
    constexpr int BUF = (BM + BN) * 128;
    // the epilogue stages the tile in the same memory, the rows of WM / PASSES waves at once
    constexpr int PASSES = BM * BN * 4 <= STAGES * BUF ? 1 : 2;
    static_assert(WM % PASSES == 0 && BM * BN * 4 <= PASSES * STAGES * BUF, "whole waves' rows per pass");
    __shared__ __attribute__((aligned(16))) char s_ab[STAGES * BUF];   // buffers: A's rows, then B's
    constexpr int ES = XDT == DT_F32 ? 4 : 2;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / WN, wn = wave % WN;
    const int r = lane & 15, g = lane >> 4;

    // each XCD takes a contiguous range of tiles, numbered so that 8 rows of tiles are
    // walked column by column: the tiles that run together share A and B in its L2
    const int tiles = p.tiles_m * p.tiles_n;
    const int64_t item = tile_of<true>(blockIdx.x, gridDim.x);
    const int piece = (int)(item / tiles);
    const int64_t tile = item - (int64_t)piece * tiles;
    const int64_t band = tile / (8 * p.tiles_n), in_band = tile - band * 8 * p.tiles_n;
    const int rows_here = p.tiles_m - band * 8 < 8 ? (int)(p.tiles_m - band * 8) : 8;
    const int64_t m0 = (band * 8 + in_band % rows_here) * BM, n0 = p.n_first + in_band / rows_here * BN;
    const int begin = piece * p.per_split, end = p.steps - begin < p.per_split ? p.steps : begin + p.per_split;

    // rows past the end read the last row (their sums are never stored)
    uint32_t a_off[A_PER], b_off[B_PER];
    {
        const int row8 = lane >> 3, c = (lane & 7) ^ row8;
#pragma unroll
        for (int i = 0; i < A_PER; ++i) {
            int64_t row = (i * NW + wave) * 8 + row8;
            row = m0 + row < p.g.M ? row : p.g.M - 1 - m0;
            a_off[i] = (uint32_t)(row * p.g.lda * ES + c * 16);
        }
#pragma unroll
        for (int i = 0; i < B_PER; ++i) {
            int64_t row = (i * NW + wave) * 8 + row8;
            if constexpr (GATED) {                     // rows 16 g .. of one weight, then of the other
                row = row / 32 * 16 + row % 16;
                row = n0 / 2 + row < p.e.N ? row : p.e.N - 1 - n0 / 2;
            } else {
                row = n0 + row < p.g.R ? row : p.g.R - 1 - n0;
            }
            b_off[i] = (uint32_t)(row * p.g.ldb * ES + c * 16);
        }
    }
    const char* const a0 = static_cast<const char*>(p.g.a0) + m0 * p.g.lda * ES;
    const char* const a1 = static_cast<const char*>(p.g.a1) + m0 * p.g.lda * ES - (int64_t)p.steps0 * 128;
    // a gated block's waves load 8 rows of 16 alternately from the two weights, each always from the same one
    static_assert(!GATED || NW % 4 == 0, "a wave's loads are of one weight");
    const char* const b0 = GATED ? static_cast<const char*>((wave >> 1) & 1 ? p.g.b1 : p.g.b) + n0 / 2 * p.g.ldb * ES
                                 : static_cast<const char*>(p.g.b) + n0 * p.g.ldb * ES;

    // a length of half a step too many: its last step begins half a step early, and only its
    // upper half is multiplied
    constexpr int PER = A_PER + B_PER;
    auto load_one = [&](int s, int buffer, int i) {
        char* const dst = s_ab + buffer * BUF;
        const int64_t at = (int64_t)s * 128 - (p.half && s + 1 == p.steps ? 64 : 0);
        if (i < A_PER) {
            const char* const as = (s < p.steps0 ? a0 : a1) + at;
            __builtin_amdgcn_global_load_lds((gptr_t)(as + a_off[i]), (lptr_t)(dst + (i * NW + wave) * 1024), 16, 0, 0);
        } else {
            const char* const bs = b0 + at;
            __builtin_amdgcn_global_load_lds((gptr_t)(bs + b_off[i - A_PER]),
                                             (lptr_t)(dst + BM * 128 + ((i - A_PER) * NW + wave) * 1024), 16, 0, 0);
        }
    };
    auto load_step = [&](int s, int buffer) {
#pragma unroll
        for (int i = 0; i < PER; ++i) load_one(s, buffer, i);
    };

    f32x4 acc[TN][TM];
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
        for (int t = 0; t < TM; ++t) acc[j][t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

    const int a_row = (wm * (BM / WM) + r) * 128, b_row = BM * 128 + (wn * (BN / WN) + r) * 128;
    u32x4 bf[2][TN], af[2][TM];
    auto read_one = [&](const char* buf, int kk, int i) {
        const int c = ((4 * kk + g) ^ (r & 7)) * 16;
        if (i < TN) bf[kk][i] = *reinterpret_cast<const u32x4*>(buf + b_row + i * 16 * 128 + c);
        else af[kk][i - TN] = *reinterpret_cast<const u32x4*>(buf + a_row + (i - TN) * 16 * 128 + c);
    };
    auto read_half = [&](const char* buf, int kk) {
#pragma unroll
        for (int i = 0; i < TN + TM; ++i) read_one(buf, kk, i);
    };
    auto multiply_half = [&](int kk) {
#pragma unroll
        for (int t = 0; t < TM; ++t)
#pragma unroll
            for (int j = 0; j < TN; ++j) mma_chunk<XDT>(bf[kk][j], af[kk][t], acc[j][t]);
    };
    const int full = end - (p.half && end == p.steps ? 1 : 0);      // steps of the whole length
#pragma unroll
    for (int i = 0; i < STAGES; ++i)
        if (begin + i < end) load_step(begin + i, i);
    int now = 0;
    // Step s with its first half's fragments in registers.  Behind the barrier step s + 1 has landed
    // and every wave has read what it takes of step s: its buffer goes to step s + STAGES.
    auto step = [&](int s, bool more, bool next) {
        read_half(s_ab + now * BUF, 1);
        multiply_half(0);
        // the reads are dealt among the products
#pragma unroll
        for (int i = 0; i < TM + TN; ++i) {
            __builtin_amdgcn_sched_group_barrier(0x008, XDT == DT_F32 ? 8 : 2, 0);      // matrix instructions
            __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);                          // an LDS read
        }
        __builtin_amdgcn_sched_group_barrier(0x008, TM * TN * (XDT == DT_F32 ? 4 : 1), 0);
        __builtin_amdgcn_sched_barrier(0);
        if (more) wait_loads<(STAGES - 2) * PER>();
        else wait_loads<0>();
        pipeline_barrier();
        // A load, some of the next step's reads and of the products in turn: the address unit takes a load of
        // 64 lanes 16 cycles, and the eight waves' loads in a row would keep the products waiting
        const int freed = now;
        now = now + 1 == STAGES ? 0 : now + 1;
        const char* const ahead = s_ab + now * BUF;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            if (more) load_one(s + STAGES, freed, i);
            if (next) {
#pragma unroll
                for (int k = 0; k < TM + TN; ++k)
                    if (k * PER / (TM + TN) == i) read_one(ahead, 0, k);
            }
#pragma unroll
            for (int k = 0; k < TM * TN; ++k)
                if (k * PER / (TM * TN) == i) mma_chunk<XDT>(bf[1][k % TN], af[1][k / TN], acc[k % TN][k / TN]);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    if (begin + STAGES <= end) wait_loads<(STAGES - 1) * PER>();
    else wait_loads<0>();
    pipeline_barrier();
    if (begin < full) read_half(s_ab, 0);
    int s = begin;
    for (; s + STAGES < end; ++s) step(s, true, true);
    for (; s + 1 < full; ++s) step(s, false, true);
    if (s < full) step(s, false, false);
    if (full < end) {
        read_half(s_ab + now * BUF, 1);
        multiply_half(1);
    }

    // lane: its column r of a 16x16 tile is C's row, its elements 4 g + i are C's columns
    if (p.split > 1) {
        float* const out = p.part + (int64_t)piece * p.g.M * p.g.R;
#pragma unroll
        for (int t = 0; t < TM; ++t) {
            const int64_t m = m0 + wm * (BM / WM) + 16 * t + r;
            if (m >= p.g.M) continue;
#pragma unroll
            for (int j = 0; j < TN; ++j) {
                const int64_t n = n0 + wn * (BN / WN) + 16 * j + 4 * g;
                const int cnt = columns_left(n, p.g.R);
                if (cnt > 0) store_up_to4<DT_F32>(out, m * p.g.R + n, cnt, acc[j][t]);
            }
        }
        return;
    }
    float* const staged = reinterpret_cast<float*>(s_ab);
#pragma unroll
    for (int pass = 0; pass < PASSES; ++pass) {
        __syncthreads();
        if (wm / (WM / PASSES) == pass) {
#pragma unroll
            for (int t = 0; t < TM; ++t)
#pragma unroll
                for (int j = 0; j < TN; ++j) {
                    const int m = (wm % (WM / PASSES)) * (BM / WM) + 16 * t + r, n4 = (wn * (BN / WN) + 16 * j) / 4 + g;
                    *reinterpret_cast<f32x4*>(staged + staged_word<BN>(m, n4)) = acc[j][t];
                }
        }
        __syncthreads();
        finish_rows<XDT, BN, NT, GATED>(p.e, staged, BM / PASSES, m0 + pass * (BM / PASSES), n0, p.g.M);
    }
}

// 64 columns of the bias's gradient: the slices dealt to 16 sums, joined in order; WAVES waves (4 or
// 16, with the same result) keep 16 / WAVES of them each.
template <int WAVES>
__device__ __forceinline__ void bias_sum(const BiasSum& b, int64_t group)
{
    constexpr int EACH = 16 / WAVES;
    __shared__ float s_sum[16][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t n = group * 64 + lane;
    float v[EACH] = {};
    if (n < b.N) {
        // (slices past the last read it again, so that no load waits for another)
#pragma unroll 4
        for (int s = wave; s < b.slices; s += 16)
#pragma unroll
            for (int q = 0; q < EACH; ++q) {
                const int at = s + q * WAVES;
                const float x = b.part[(int64_t)(at < b.slices ? at : b.slices - 1) * b.N + n];
                v[q] += at < b.slices ? x : 0.0f;
            }
    }
#pragma unroll
    for (int q = 0; q < EACH; ++q) s_sum[wave + q * WAVES][lane] = v[q];
    __syncthreads();
    if (wave != 0 || n >= b.N) return;
    float sum = 0.0f;
#pragma unroll
    for (int w = 0; w < 16; ++w) sum += s_sum[w][lane];
    if (b.dt == DT_F32) store1<DT_F32>(b.db, n, b.accumulate ? sum + load1<DT_F32>(b.db, n) : sum);
    else if (b.dt == DT_F16) store1<DT_F16>(b.db, n, b.accumulate ? sum + load1<DT_F16>(b.db, n) : sum);
    else store1<DT_BF16>(b.db, n, b.accumulate ? sum + load1<DT_BF16>(b.db, n) : sum);
}

// (4096 columns of 128 slices: with one thread a column 7 us, with four waves 5.5, with 16 4.7)
__global__ __launch_bounds__(1024) void k_bias_sum(const BiasSum b) { bias_sum<16>(b, blockIdx.x); }

// The pieces of a split product added in order, then the epilogue: four columns a thread.  The
// workgroups from `blocks` on take the bias's gradient (a launch of its own 3 us more).
template <int XDT, bool GATED>
__global__ __launch_bounds__(256) void k_join_split(const GemmParams p, int64_t groups, int blocks, const BiasSum b)
{
    if ((int)blockIdx.x >= blocks) {
        bias_sum<4>(b, blockIdx.x - blocks);
        return;
    }
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t m = i / groups, n = (i - m * groups) * 4;
    if (m >= p.g.M) return;
    auto sum = [&](int64_t column) {
        const int cnt = columns_left(column, p.g.R);
        f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
        for (int s = 0; s < p.split; ++s) v += load_up_to4<DT_F32>(p.part, ((int64_t)s * p.g.M + m) * p.g.R + column, cnt);
        return v;
    };
    if constexpr (GATED) {
        const int64_t column = n / 16 * 32 + n % 16;
        const f32x4 g = sum(column), u = sum(column + 16);
        finish_gated4<XDT>(p.e, m, n, g, u);
    } else {
        finish_linear4<XDT>(p.e, m, n, sum(n));
    }
}

template <int XDT, bool GATED>
hipError_t join_as(const GemmParams& p, const BiasSum* b, hipStream_t s)
{
    const int64_t groups = (p.e.N + 3) / 4;
    const int blocks = (int)tiles_over(p.g.M * groups, 256), more = b ? (int)tiles_over(b->N, 64) : 0;
    return launch_kernel(k_join_split<XDT, GATED>, blocks + more, s, p, groups, blocks, b ? *b : BiasSum{});
}

// `rows` rows of an array of `width` elements further on.
const void* further(const void* p, int64_t rows, int64_t width, int es)
{
    return p ? static_cast<const char*>(p) + rows * width * es : nullptr;
}

// Rows m .. m + rows - 1 of the product.
template <int XDT>
GemmParams rows_of(const GemmParams& all, int64_t m, int64_t rows)
{
    constexpr int ES = XDT == DT_F32 ? 4 : 2;
    GemmParams p = all;
    p.g.M = rows;
    p.g.a0 = further(all.g.a0, m, p.g.lda, ES);
    p.g.a1 = further(all.g.a1, m, p.g.lda, ES);
    p.e = epilogue_rows(all.e, m, ES);
    return p;
}

// Columns n_first .. R - 1 of B in BN-wide tiles (`columns` tiles of them at most), the length
// in p.split pieces.
template <int XDT, int BM, int BN, int WM, int WN, int STAGES, bool GATED>
hipError_t gemm_as(GemmParams p, int64_t n_first, int64_t columns, hipStream_t s)
{
    p.n_first = n_first;
    const int64_t all = tiles_over(p.g.R - n_first, BN);
    p.tiles_n = (int)(all < columns ? all : columns);
    p.tiles_m = (int)tiles_over(p.g.M, BM);
    return launch_kernel_nt(k_gemm<XDT, BM, BN, WM, WN, STAGES, GATED>, p.tiles_m * p.tiles_n * p.split, 64 * WM * WN,
                            s, p);
}

constexpr int64_t kEveryColumn = int64_t(1) << 40;

// Tile shapes (the cases of gemm_shape), and the time in us of a step of a workgroup where 1, 2, ..
// of them share a CU: fitted to layers of 4096 and 11008 inputs and outputs with 1 .. 4096
// rows, their weights just dequantized (bf16).  A CU's only workgroup waits for memory:
// 256 rows of 4096 x 4096 take 48 us in all in 64 x 64 tiles with three buffers, 35 with five; many
// small workgroups a CU hide it as well (with two buffers: 30).  Binary32 is bound by the matrix
// instructions and takes the third or the fourth (4096 x 4096 x 4096 1009 us and 1085; in the
// first 979).  128 x 256 tiles are not built: with three buffers they save 2 to 4% of the few products of 512 and
// 1024 rows where they are the best (the gradient of 1024 rows of 4096 x 4096 split in two 55 us, 57 in 128 x 128
// tiles).  The estimate's own choice can be further off: 61 there, 40 and not 34 for 300 rows (128 x 128 in two), 193 and
// not 177 for 2048 rows of 4096 x 11008 (256 x 256 in two).
struct TileShape {
    int bm, bn, per_cu;
    double us[5];
};
constexpr int kShapeCount = 5, kCus = 256;
constexpr TileShape kShapes[kShapeCount] = {
    {256, 256, 1, {1.6}}, {128, 128, 1, {0.77}}, {128, 128, 2, {0.80, 0.95}},
    {64, 64, 2, {0.38, 0.44}}, {64, 64, 5, {0.50, 0.56, 0.70, 0.89, 0.93}}};

// Estimated time of `groups` workgroups of `steps` steps: rounds that fill every CU, then the
// rest.  Binary32 is bound by the matrix instructions (0.55 TFLOP/s a CU, 0.51 in 64 x 64 tiles) where
// several share a CU.
// (32-bit numbers, since the host takes this estimate at every call.)
double rounds_us(int xdt, const TileShape& t, uint32_t groups, uint32_t steps)
{
    auto step_us = [&](uint32_t k) {
        const double flops = 2.0 * t.bm * t.bn * gemm_step(DT_F32) * k / (t.bm == 64 ? 0.51e6 : 0.55e6);
        return xdt == DT_F32 && flops > t.us[k - 1] ? flops : t.us[k - 1];
    };
    const uint32_t round = kCus * t.per_cu, full = groups / round, rest = groups - full * round;
    return (full * step_us(t.per_cu) + (rest ? step_us((rest + kCus - 1) / kCus) : 0.0)) * steps;
}

struct GemmPlan {
    int shape, split;
    double us;
};

// The best shape and number of pieces for M x R of `steps` steps.  A split product's partial
// sums are written and read once (3.5 TB/s) and cost a launch; four steps a piece at least.
// (gemm_rows keeps the number of tiles below 2^24.)
GemmPlan gemm_plan(int xdt, int64_t M, int64_t R, uint32_t steps, bool may_split)
{
    GemmPlan best{0, 1, 1e300};
    const double sums = (double)M * (double)R;
    const uint32_t fit = sums * kSplitMax <= (double)kPartMax ? (uint32_t)kSplitMax : (uint32_t)((double)kPartMax / sums);
    const uint32_t most = may_split ? (steps / 4 < fit ? steps / 4 : fit) : 1;
    const int first = xdt == DT_F32 ? 2 : 0, end = xdt == DT_F32 ? 4 : kShapeCount;
    for (int i = first; i < end; ++i) {
        const TileShape& t = kShapes[i];
        const uint32_t tiles = (uint32_t)((M + t.bm - 1) / t.bm * ((R + t.bn - 1) / t.bn));
        for (uint32_t split = 1; split == 1 || (split <= most && split * tiles <= 5u * kCus); ++split) {
            const double us = rounds_us(xdt, t, tiles * split, (steps + split - 1) / split) + 4.0 +
                              (split > 1 ? 4.0 + 8.0 * split * sums / 3.5e6 : 0.0);
            if (us < best.us) best = GemmPlan{i, (int)split, us};
        }
    }
    return best;
}

template <int XDT, bool GATED>
hipError_t gemm_shape(int shape, const GemmParams& p, int64_t n_first, int64_t columns, hipStream_t s)
{
    if constexpr (XDT == DT_F32) {
        return shape == 2 ? gemm_as<XDT, 128, 128, 2, 4, 2, GATED>(p, n_first, columns, s)
                          : gemm_as<XDT, 64, 64, 2, 2, 5, GATED>(p, n_first, columns, s);
    } else {
        switch (shape) {
        case 0: return gemm_as<XDT, 256, 256, 2, 4, 2, GATED>(p, n_first, columns, s);
        case 1: return gemm_as<XDT, 128, 128, 2, 4, 4, GATED>(p, n_first, columns, s);
        case 2: return gemm_as<XDT, 128, 128, 2, 4, 2, GATED>(p, n_first, columns, s);
        case 3: return gemm_as<XDT, 64, 64, 2, 2, 5, GATED>(p, n_first, columns, s);
        default: return gemm_as<XDT, 64, 64, 2, 2, 2, GATED>(p, n_first, columns, s);
        }
    }
}

// bias: the gradient that the call computes as well, or nullptr.
template <int XDT, bool GATED>
hipError_t gemm_tiles(GemmParams p, const BiasSum* bias, hipStream_t s)
{
    const int64_t M = p.g.M, R = p.g.R;
    const GemmPlan plan = gemm_plan(XDT, M, R, p.steps, p.part != nullptr);
    // or: the columns that whole rounds of 256 x 256 tiles cover, and the rest in the shape that suits it best (4096
    // rows of a gated block of 2 x 11008, 5.4 rounds: 709 us in 256 x 256 tiles alone, 662 so)
    const int64_t rows = tiles_over(M, 256), columns = tiles_over(R, 256), whole = rows * columns / kCus * kCus / rows;
    if (XDT != DT_F32 && whole > 0 && whole < columns) {
        p.split = 1;
        p.per_split = p.steps;
        const GemmPlan rest = gemm_plan(XDT, M, R - whole * 256, p.steps, false);
        if (rounds_us(XDT, kShapes[0], (uint32_t)(rows * whole), p.steps) + 4.0 + rest.us < plan.us && rest.shape != 0) {
            hipError_t e = gemm_shape<XDT, GATED>(0, p, 0, whole, s);
            if (e == hipSuccess) e = gemm_shape<XDT, GATED>(rest.shape, p, whole * 256, kEveryColumn, s);
            return e == hipSuccess && bias ? launch_bias_sum(*bias, s) : e;
        }
    }
    p.per_split = (int)tiles_over(p.steps, plan.split);
    p.split = (int)tiles_over(p.steps, p.per_split);
    const hipError_t e = gemm_shape<XDT, GATED>(plan.shape, p, 0, kEveryColumn, s);
    if (e != hipSuccess) return e;
    if (p.split > 1) return join_as<XDT, GATED>(p, bias, s);
    return bias ? launch_bias_sum(*bias, s) : hipSuccess;
}

// One product, or several of fewer rows where a grid would not hold them.
template <int XDT, bool GATED>
hipError_t gemm_rows(const GemmParams& p, const BiasSum* bias, hipStream_t s)
{
    const int64_t M = p.g.M, most = (int64_t(1) << 21) / tiles_over(p.g.R, 64) * 256;
    for (int64_t m = 0; m < M; m += most) {
        const hipError_t e = gemm_tiles<XDT, GATED>(rows_of<XDT>(p, m, M - m < most ? M - m : most), m == 0 ? bias : nullptr, s);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace

hipError_t launch_unpack(int xdt, const Weight4* w, int count, int64_t N, int64_t K, const Weight4Format& f, void* out,
                         size_t each, hipStream_t s)
{
    DequantDesc d[2];
    for (int i = 0; i < count; ++i)
        d[i] = DequantDesc{w[i].codes,   w[i].absmax, w[i].c2, w[i].absmax2,
                           w[i].offset, static_cast<char*>(out) + i * each, N * K, 0};
    return launch_dequant4_kept(d, count, f.code4, 1 << f.log2B, 1 << f.log2B2, f.nested != 0, xdt, s);
}

hipError_t launch_bias_sum(const BiasSum& b, hipStream_t s)
{
    return launch_kernel_nt(k_bias_sum, (int)tiles_over(b.N, 64), 1024, s, b);
}

hipError_t launch_join(int xdt, const float* part, int pieces, int64_t M, const Epilogue& e, const BiasSum* bias,
                       hipStream_t s)
{
    GemmParams p{};
    p.g.M = M;
    p.g.R = e.N;
    p.e = e;
    p.part = const_cast<float*>(part);
    p.split = pieces;
    return xdt == DT_F16 ? join_as<DT_F16, false>(p, bias, s) : join_as<DT_BF16, false>(p, bias, s);
}

double gemm_us(int xdt, int64_t M, int64_t R, int64_t len)
{
    return gemm_plan(xdt, M, R, (uint32_t)tiles_over(len, gemm_step(xdt)), true).us;
}

hipError_t launch_gemm(int xdt, bool gated, const GemmArgs& g, const Epilogue& e, float* part, const BiasSum* bias,
                       hipStream_t s)
{
    const int64_t step = gemm_step(xdt);
    GemmParams p{};
    p.g = g;
    p.e = e;
    p.part = part;
    p.steps = (int32_t)((g.len + step - 1) / step);
    p.steps0 = (int32_t)((g.len0 + step - 1) / step);
    p.half = g.len % step ? 1 : 0;
    switch (xdt) {
    case DT_F32: return gated ? gemm_rows<DT_F32, true>(p, bias, s) : gemm_rows<DT_F32, false>(p, bias, s);
    case DT_F16: return gated ? gemm_rows<DT_F16, true>(p, bias, s) : gemm_rows<DT_F16, false>(p, bias, s);
    default: return gated ? gemm_rows<DT_BF16, true>(p, bias, s) : gemm_rows<DT_BF16, false>(p, bias, s);
    }
}

}  // namespace qb
