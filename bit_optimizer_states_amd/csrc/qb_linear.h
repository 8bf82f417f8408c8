// qb_linear.h -- internal launchers of the 4-bit layers with a fused epilogue: the linear
// layer (bias, activation, residual), the gated block (two projections, activation,
// product) and their gradients.  Argument checks are done by the callers in
// qb_linear_api.cpp.
#pragma once
#include "qb_launch.h"

namespace qb {

// A weight [N, K] in 4 bits: codes and block constants, plain (absmax) or nested (c2,
// absmax2, offset).
struct Weight4 {
    const uint8_t* codes;
    const float* absmax;
    const uint8_t* c2;
    const float* absmax2;
    const float* offset;
};

// The code and block sizes that the weights of a call share.
struct Weight4Format {
    int32_t log2B, log2B2, code4, nested;
};

// What becomes of a sum z of products, in binary32 and rounded once per output.
//   linear: z += bias (each optional); z out; y = act(z) + residual.
//   gated:  the sums g and u of one column: g, u out (z, u); y = act(g) * u.
// y [M, N], as are z, u and residual (which may be y itself).
struct Epilogue {
    const void* bias;        // [N] of dtype bias_dt
    const void* residual;
    void* z;
    void* u;
    void* y;
    int64_t N;
    int32_t bias_dt, act;
};

// The epilogue of the rows m onwards (of types of `es` bytes).
inline Epilogue epilogue_rows(Epilogue e, int64_t m, int es)
{
    const int64_t at = m * e.N * es;
    if (e.residual) e.residual = static_cast<const char*>(e.residual) + at;
    if (e.z) e.z = static_cast<char*>(e.z) + at;
    if (e.u) e.u = static_cast<char*>(e.u) + at;
    e.y = static_cast<char*>(e.y) + at;
    return e;
}

// Rows of x up to which the products are always taken straight from the codes, and without a
// workspace; beyond, by an estimate, or after the weights are dequantized (which takes a length
// of a step of the tiled product at least).
constexpr int64_t kRowsMax = 64;
constexpr bool takes_rows(int64_t M, int64_t K) { return M <= kRowsMax || K < 64; }

// y = epilogue(x W^T) straight from the codes (count 1: linear, 2: gated).
hipError_t launch_linear_rows(int xdt, const void* x, int64_t M, int64_t K, const Weight4* w, int count,
                              const Weight4Format& f, const Epilogue& e, hipStream_t s);

// Elements of a step of the tiled product, and of the multiples that the reduced dimension
// of a gradient is padded to: 128 bytes.
constexpr int64_t gemm_step(int dt) { return dt == 0 ? 32 : 64; }
constexpr int64_t gemm_pitch(int dt, int64_t k) { return (k + gemm_step(dt) - 1) / gemm_step(dt) * gemm_step(dt); }
// Columns of a gated block's product: those of the two weights, dealt in groups of 16.
constexpr int64_t gated_rows(int64_t n) { return (n + 15) / 16 * 32; }

// One or two weights in the compute dtype, [n][k] (as qb_dequantize), the second `each` bytes
// behind the first.
hipError_t launch_unpack(int xdt, const Weight4* w, int count, int64_t N, int64_t K, const Weight4Format& f, void* out,
                         size_t each, hipStream_t s);
// One or two weights [N, K] transposed: out[k][n], the second's columns n at np + n, np =
// gemm_pitch(N); the pitch is count * np, its padding zero.
struct TransposedWeights {
    Weight4 w[2];
    Weight4Format f;
    void* out;
    int64_t N, K, np;
    int32_t count;
};

// C = epilogue(A B^T).  A [M, len] in one or two pieces of columns (a0: the first len0, a1
// the others; both of `lda` elements a row, 16-byte aligned rows), B [R, len] of ldb
// elements a row; gated: B is dealt from b and b1, of N rows each, and R = gated_rows(N).  len is at least a step and a multiple of half a step, len0 of a step
// unless it is len.
struct GemmArgs {
    const void* a0;
    const void* a1;
    const void* b;
    const void* b1;
    int64_t M, R, len0, len, lda, ldb;
};
// The gradient of a bias from dz's sums over slices of rows: db[n] = the sum of part[.][n] in order
// (plus what it holds).
struct BiasSum {
    const float* part;
    void* db;
    int64_t N;
    int32_t slices, accumulate, dt;
};
hipError_t launch_bias_sum(const BiasSum& b, hipStream_t s);

// part: room for the partial sums of a product split over its length, gemm_part_floats()
// (a product of few tiles is not split without it).  bias: computed as well, nullptr none.
hipError_t launch_gemm(int xdt, bool gated, const GemmArgs& g, const Epilogue& e, float* part, const BiasSum* bias,
                       hipStream_t s);

// The join of a split product alone: the epilogue of the sum of `pieces` pieces, part[piece][M][e.N],
// 16-bit types.
hipError_t launch_join(int xdt, const float* part, int pieces, int64_t M, const Epilogue& e, const BiasSum* bias,
                       hipStream_t s);

// Estimated times in us: of launch_linear_rows, and of launch_gemm of M x R x len.
double rows_us(int xdt, int64_t M, int64_t K, int64_t N, int count);
double gemm_us(int xdt, int64_t M, int64_t R, int64_t len);

// A product is split into kSplitMax pieces at most, and into as many as have their partial
// sums (M R each) in kPartMax: never less room for more rows or columns.
constexpr int64_t kSplitMax = 16, kPartMax = int64_t(20) << 20;
constexpr int64_t gemm_part_floats(int64_t M, int64_t R)
{
    return kSplitMax * M * R < kPartMax ? kSplitMax * M * R : kPartMax;
}

// dz = dy act'(z) [M, N] into `dz` of pitch `pitch` (its padding zero; nullptr: not
// wanted) and into `dz_out` [M, N] (nullptr: not wanted), and per slice of rows the sums of
// dz over its rows, part[slice][N] (nullptr: not wanted).  z == nullptr: dz = dy.  dz_too false:
// none of this.  And the weights `t` (nullptr: not wanted).
hipError_t launch_linear_grad(int xdt, bool dz_too, const void* dy, const void* z, int act, int64_t M, int64_t N, void* dz,
                              int64_t pitch, void* dz_out, float* part, int slices, const TransposedWeights* t,
                              hipStream_t s);
constexpr int kDzCols = 512, kDzWaves = 4;
// Slices of rows: enough workgroups for the chip (2048 over the blocks of columns), four rows a
// wave at least, two where that leaves fewer than 64 slices (301 rows of 2731 columns in binary32:
// 9.7 us in 19 slices, 7.0 in 38).
inline int linear_dz_slices(int64_t M, int64_t N)
{
    const int64_t blocks = (N + kDzCols - 1) / kDzCols, want = (2048 + blocks - 1) / blocks;
    const int64_t fours = (M + 4 * kDzWaves - 1) / (4 * kDzWaves), twos = (M + 2 * kDzWaves - 1) / (2 * kDzWaves);
    const int64_t most = fours > 64 ? fours : twos < 64 ? twos : 64, n = want < most ? want : most;
    return (int)(n < 1 ? 1 : n);
}
// dg = dh u act'(g) and du = dh act(g) into `dz` ([M, pitch] each, du behind dg; nullptr:
// not wanted) and into dg_out, du_out [M, N] (nullptr: not wanted).  And the weights `t`
// (nullptr: not wanted).
hipError_t launch_gated_grad(int xdt, const void* dh, const void* g, const void* u, int act, int64_t M, int64_t N,
                             void* dz, int64_t pitch, void* dg_out, void* du_out, const TransposedWeights* t,
                             hipStream_t s);

// dz W for up to kRowsMax rows in a 16-bit type, the weights from their codes: part[slice][M][K] of
// `*slices` slices of the n (t.out is not used).
hipError_t launch_few_rows_back(int xdt, const void* dz0, const void* dz1, int64_t ldz, int64_t M,
                                const TransposedWeights& t, float* part, int* slices, hipStream_t s);

}  // namespace qb
