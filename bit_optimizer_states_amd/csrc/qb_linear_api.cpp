// qb_linear_api.cpp -- the C ABI of the 4-bit layers with an epilogue, their gradients,
// and the gradient norm (declared in include/qb.h): argument validation, workspace layout and
// dispatch.  Nothing is enqueued unless every argument checks out.
#include <hip/hip_runtime.h>

#include <cmath>

#include "qb.h"
#include "qb_clip.h"
#include "qb_linear.h"

namespace {

using namespace qb;

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool valid_dtype(qb_dtype d) { return d == QB_F32 || d == QB_F16 || d == QB_BF16; }
bool valid_act(qb_act a) { return a >= QB_ACT_NONE && a <= QB_ACT_SILU; }
bool pow2_block(int32_t b) { return b >= 64 && b <= 4096 && (b & (b - 1)) == 0; }
size_t round_up(size_t v, size_t a) { return (v + a - 1) / a * a; }
int dtype_bytes(int d) { return d == QB_F32 ? 4 : 2; }

constexpr int64_t kRowMax = int64_t(1) << 31;        // rows of x
constexpr int64_t kGradMax = int64_t(1) << 33;       // elements of a gradient: 2^22 tiles at most
constexpr int64_t kWidthMax = int64_t(1) << 21;      // inputs, outputs of a layer

qb_status hip_status(hipError_t e)
{
    if (e == hipSuccess) return QB_OK;
    if (e == hipErrorNotInitialized) return QB_EINIT;
    return QB_EHIP;
}

bool valid_sizes(qb_dtype xdt, int64_t M, int64_t K, int64_t N)
{
    return valid_dtype(xdt) && M >= 0 && M < kRowMax && K > 0 && K % 32 == 0 && K < kWidthMax && N >= 0 && N < kWidthMax;
}

int log2_of(int32_t v)
{
    int l = 0;
    while ((int32_t(1) << l) < v) ++l;
    return l;
}

// Checks one weight; nested: -1 = not fixed yet, 0 plain, 1 nested (the weights of a
// call must agree).
qb_status check_weight(const Weight4& w, int* nested)
{
    if (!w.codes) return QB_EINVAL;
    const int mode = w.c2 ? 1 : 0;
    if (*nested >= 0 && *nested != mode) return QB_EUNSUPPORTED;
    *nested = mode;
    if (mode) {
        if (w.absmax || !w.absmax2 || !w.offset) return QB_EINVAL;
        if (!aligned16(w.c2) || !aligned16(w.absmax2) || !aligned16(w.offset)) return QB_EALIGN;
    } else if (!w.absmax || w.absmax2 || w.offset) {     // (nested constants without their codes)
        return QB_EINVAL;
    }
    return aligned16(w.codes) && aligned16(w.absmax) ? QB_OK : QB_EALIGN;
}

// The shared format of a call's weights [N, K].
qb_status check_format(qb_code code, int32_t blocksize, int32_t blocksize2, int64_t N, int64_t K, Weight4Format* f)
{
    if ((code != QB_NF4 && code != QB_FP4) || !pow2_block(blocksize)) return QB_EINVAL;
    if (f->nested && !pow2_block(blocksize2)) return QB_EINVAL;
    if ((N * K + blocksize - 1) / blocksize >= (int64_t(1) << 31)) return QB_EINVAL;
    f->log2B = log2_of(blocksize);
    f->log2B2 = f->nested ? log2_of(blocksize2) : 0;
    f->code4 = code == QB_FP4 ? 1 : 0;
    return QB_OK;
}

Weight4 weight_of(const uint8_t* codes, const float* absmax, const qb_dq* dq)
{
    return Weight4{codes, absmax, dq ? dq->codes : nullptr, dq ? dq->absmax2 : nullptr, dq ? dq->offset : nullptr};
}

// A qb_dq without codes is not a plain weight.
bool broken_dq(const qb_dq* dq) { return dq && !dq->codes; }

Weight4 weight_of(const qb_weight& w) { return Weight4{w.codes, w.absmax, w.c2, w.absmax2, w.offset}; }

qb_status check_ws(size_t need, const void* ws, size_t ws_bytes)
{
    if (need == 0) return QB_OK;
    if (!ws) return QB_EINVAL;
    if (!aligned16(ws)) return QB_EALIGN;
    return ws_bytes < need ? QB_EWORKSPACE : QB_OK;
}

// Workspace of a forward call that dequantizes its weights first: these, then the partial
// sums of a split product of R columns.
size_t unpacked_bytes(int xdt, int64_t K, int64_t N)
{
    return round_up((size_t)N * (size_t)K * dtype_bytes(xdt), 256);
}

size_t forward_bytes(int xdt, int64_t M, int64_t K, int64_t N, int count)
{
    if (takes_rows(M, K)) return 0;
    return count * unpacked_bytes(xdt, K, N) +
           (size_t)gemm_part_floats(M, count == 2 ? gated_rows(N) : N) * sizeof(float);
}

// The rows kernel, where it is needed or the faster one by the estimates: each reads the
// codes once a block of rows and needs one launch; two launches and the dequantized weights
// (5.6 TB/s) in the other.  bf16, us: 77 rows of 992 x 1001 14.4 dequantized, 9.8 so; 128 rows
// of 4096 x 4096 25 and 21, 256 rows 30 and 40; 128 rows of 4096 x 11008 50 and 57, of a gated block
// of them 81 and 70.
bool rows_win(int xdt, int64_t M, int64_t K, int64_t N, int count)
{
    if (takes_rows(M, K)) return true;
    if (M > 1024) return false;
    const double rows = rows_us(xdt, M, K, N, count);
    if (rows < 13.0) return true;               // two launches take that much in any case
    const double unpack = 3.0 + count * (double)N * (double)K * (0.5 + dtype_bytes(xdt)) / 5.6e6;
    return rows < 0.9 * (unpack + gemm_us(xdt, M, count == 2 ? gated_rows(N) : N, K));
}

// y = epilogue(x W^T) through the workspace.
hipError_t unpack_and_multiply(int xdt, const void* x, int64_t M, int64_t K, const Weight4* w, int count, int64_t N,
                               const Weight4Format& f, const Epilogue& e, void* ws, hipStream_t s)
{
    const size_t each = unpacked_bytes(xdt, K, N);
    char* const b = static_cast<char*>(ws);
    const hipError_t err = launch_unpack(xdt, w, count, N, K, f, b, each, s);
    if (err != hipSuccess) return err;
    const GemmArgs g{x, nullptr, b, b + (count - 1) * each, M, count == 2 ? gated_rows(N) : N, K, K, K, K};
    return launch_gemm(xdt, count == 2, g, e, reinterpret_cast<float*>(b + count * each), nullptr, s);
}

// Whether dx is taken from the codes, without the transposed weights in the workspace: up to 48 rows,
// and up to 64 of a layer of more than 2^24 weights (64 rows, us: 1024 x 1000 17.6 so and 14.8 by the
// tiled product, 4096 x 4096 24.8 and 24.3, 4096 x 11008 34.5 and 46).  Its slices' sums have to fit
// the room for partial sums.
constexpr int64_t kFewWeights = int64_t(1) << 24;
bool may_be_few(int xdt, int64_t M, int64_t K) { return xdt != QB_F32 && M <= kRowsMax && M * K <= kPartMax; }
bool few_rows(int xdt, int64_t M, int64_t K, int64_t N, int count)
{
    return may_be_few(xdt, M, K) && (M <= 48 || count * N * K > kFewWeights);
}

// Room for a gradient's transposed weights: none up to 48 rows of few; up to 64, where the smaller layers
// take them, no more than the largest of these does (rows of N padded by less than a step), so that
// it never shrinks.
size_t transposed_bytes(int xdt, int64_t M, int64_t K, int64_t N, int count)
{
    const size_t all = (size_t)K * (size_t)gemm_pitch(xdt, N) * count * dtype_bytes(xdt);
    if (!may_be_few(xdt, M, K)) return all;
    if (M <= 48) return 0;
    const size_t most = (size_t)(kFewWeights + gemm_step(xdt) * K * count) * dtype_bytes(xdt);
    return all < most ? all : most;
}

// Workspace of a gradient: the weights transposed, dz (dg and du) padded, the partial
// sums of a split product and of the bias's gradient.
struct BackwardLayout {
    size_t dz, split, part, bytes;
};

BackwardLayout backward_layout(int xdt, int64_t M, int64_t K, int64_t N, int count)
{
    const size_t pitch = (size_t)gemm_pitch(xdt, N) * count * dtype_bytes(xdt);
    // the partial sums' slices shrink as columns are added: what is reserved never does
    const size_t most = (size_t)((M + 7) / 8) * (size_t)N, cap = (size_t)2048 * 512 + (size_t)N;
    BackwardLayout l;
    l.dz = round_up(transposed_bytes(xdt, M, K, N, count), 256);
    l.split = l.dz + round_up((size_t)M * pitch, 256);
    l.part = l.split + round_up((size_t)gemm_part_floats(M, K) * sizeof(float), 256);
    l.bytes = l.part + (count == 1 ? (most < cap ? most : cap) * sizeof(float) : 0);
    return l;
}

bool whole_steps(int xdt, int64_t n) { return n % gemm_step(xdt) == 0; }

TransposedWeights transposed(int xdt, const Weight4* w, int count, const Weight4Format& f, int64_t K, int64_t N, void* ws)
{
    return TransposedWeights{{w[0], w[count - 1]}, f, ws, N, K, gemm_pitch(xdt, N), count};
}

// dx = [dz_0 dz_1] [W_0; W_1] for dz of rows of `lda` elements and the weights `t`; the bias's gradient
// with it (nullptr: none).
hipError_t input_gradient(int xdt, const void* dz0, const void* dz1, int64_t lda, const TransposedWeights& t, int64_t M,
                          void* dx, float* part, const BiasSum* bias, hipStream_t s)
{
    const int64_t pitch = t.np * t.count;
    Epilogue out{};
    out.y = dx;
    out.N = t.K;
    if (few_rows(xdt, M, t.K, t.N, t.count)) {
        int slices = 0;
        const hipError_t e = launch_few_rows_back(xdt, dz0, dz1, lda, M, t, part, &slices, s);
        return e != hipSuccess ? e : launch_join(xdt, part, slices, M, out, bias, s);
    }
    const GemmArgs g{dz0, dz1, t.out, nullptr, M, t.K, t.np, pitch, lda, pitch};
    return launch_gemm(xdt, false, g, out, part, bias, s);
}

}  // namespace

extern "C" {

size_t qb_dequant_linear_workspace_bytes(qb_dtype xdt, int64_t M, int64_t K, int64_t N)
{
    return valid_sizes(xdt, M, K, N) ? forward_bytes(xdt, M, K, N, 1) : 0;
}

qb_status qb_dequant_linear(const void* x, qb_dtype xdt, int64_t M, int64_t K, const uint8_t* codes,
                            const float* absmax, const qb_dq* dq, qb_code code, int32_t blocksize, int64_t N,
                            const void* bias, qb_dtype bdt, qb_act act, const void* residual, void* z, void* y,
                            void* ws, size_t ws_bytes, void* stream)
{
    if (!valid_sizes(xdt, M, K, N) || !valid_act(act) || (bias && !valid_dtype(bdt))) return QB_EINVAL;
    if (bias && bdt != QB_F32 && bdt != xdt) return QB_EUNSUPPORTED;
    const Weight4 w = weight_of(codes, absmax, dq);
    Weight4Format f{0, 0, 0, dq ? 1 : 0};
    qb_status st = check_format(code, blocksize, dq ? dq->blocksize2 : 0, N, K, &f);
    if (st != QB_OK) return st;
    if (M == 0 || N == 0) return QB_OK;
    if (!x || !y || broken_dq(dq)) return QB_EINVAL;
    int nested = -1;
    st = check_weight(w, &nested);
    if (st != QB_OK) return st;
    if (!aligned16(x) || !aligned16(bias) || !aligned16(residual) || !aligned16(z) || !aligned16(y)) return QB_EALIGN;
    st = check_ws(forward_bytes(xdt, M, K, N, 1), ws, ws_bytes);
    if (st != QB_OK) return st;
    hipStream_t s = static_cast<hipStream_t>(stream);
    const Epilogue e{bias, residual, z, nullptr, y, N, (int32_t)bdt, (int32_t)act};
    if (rows_win(xdt, M, K, N, 1)) return hip_status(launch_linear_rows(xdt, x, M, K, &w, 1, f, e, s));
    return hip_status(unpack_and_multiply(xdt, x, M, K, &w, 1, N, f, e, ws, s));
}

size_t qb_dequant_linear_backward_workspace_bytes(qb_dtype xdt, int64_t M, int64_t K, int64_t N)
{
    return valid_sizes(xdt, M, K, N) && N > 0 ? backward_layout(xdt, M, K, N, 1).bytes : 0;
}

qb_status qb_dequant_linear_backward(const void* dy, const void* z, qb_dtype xdt, int64_t M, int64_t K,
                                     const uint8_t* codes, const float* absmax, const qb_dq* dq, qb_code code,
                                     int32_t blocksize, int64_t N, qb_act act, void* dx, void* dz, void* dbias,
                                     qb_dtype bdt, int32_t accumulate, void* ws, size_t ws_bytes, void* stream)
{
    if (!valid_sizes(xdt, M, K, N) || N == 0 || !valid_act(act) || (dbias && !valid_dtype(bdt)) ||
        (accumulate != 0 && accumulate != 1))
        return QB_EINVAL;
    if (dbias && bdt != QB_F32 && bdt != xdt) return QB_EUNSUPPORTED;
    const Weight4 w = weight_of(codes, absmax, dq);
    Weight4Format f{0, 0, 0, dq ? 1 : 0};
    qb_status st = check_format(code, blocksize, dq ? dq->blocksize2 : 0, N, K, &f);
    if (st != QB_OK) return st;
    if (!dx && !dz && !dbias) return QB_OK;
    if (M == 0 && (!dbias || accumulate)) return QB_OK;
    if (M > 0 && (!dy || (act != QB_ACT_NONE && !z))) return QB_EINVAL;
    if (dx && M > 0) {
        if (broken_dq(dq)) return QB_EINVAL;
        int nested = -1;
        st = check_weight(w, &nested);
        if (st != QB_OK) return st;
    }
    if (!aligned16(dy) || !aligned16(z) || !aligned16(dx) || !aligned16(dz) || !aligned16(dbias)) return QB_EALIGN;
    const BackwardLayout l = backward_layout(xdt, M, K, N, 1);
    st = check_ws(M > 0 && (dx || dbias) ? l.bytes : 0, ws, ws_bytes);
    if (st != QB_OK) return st;
    hipStream_t s = static_cast<hipStream_t>(stream);
    char* const wp = static_cast<char*>(ws);
    const int64_t pitch = gemm_pitch(xdt, N);
    const TransposedWeights t = transposed(xdt, &w, 1, f, K, N, wp);
    const void* a = dy;
    int64_t lda = N;
    hipError_t e = hipSuccess;
    if (M > 0) {
        const bool own = dx && (act != QB_ACT_NONE || !whole_steps(xdt, N));     // dx reads a padded dz
        const bool given = own && dz && whole_steps(xdt, N);                     // ... which the caller's dz is
        e = launch_linear_grad(xdt, own || dz || dbias, dy, act != QB_ACT_NONE ? z : nullptr, act, M, N,
                               own && !given ? wp + l.dz : nullptr, pitch, dz,
                               dbias ? reinterpret_cast<float*>(wp + l.part) : nullptr, linear_dz_slices(M, N),
                               dx && !few_rows(xdt, M, K, N, 1) ? &t : nullptr, s);
        if (own) {
            a = given ? dz : wp + l.dz;
            lda = pitch;
        }
    }
    const BiasSum bias{reinterpret_cast<float*>(wp + l.part), dbias, N, M > 0 ? linear_dz_slices(M, N) : 0, accumulate,
                       (int32_t)bdt};
    if (e == hipSuccess && dx && M > 0)
        e = input_gradient(xdt, a, nullptr, lda, t, M, dx, reinterpret_cast<float*>(wp + l.split), dbias ? &bias : nullptr, s);
    else if (e == hipSuccess && dbias)
        e = launch_bias_sum(bias, s);
    return hip_status(e);
}

size_t qb_dequant_gated_workspace_bytes(qb_dtype xdt, int64_t M, int64_t K, int64_t N)
{
    return valid_sizes(xdt, M, K, N) ? forward_bytes(xdt, M, K, N, 2) : 0;
}

qb_status qb_dequant_gated(const void* x, qb_dtype xdt, int64_t M, int64_t K, const qb_weight* gate,
                           const qb_weight* up, qb_code code, int32_t blocksize, int32_t blocksize2, int64_t N,
                           qb_act act, void* gate_out, void* up_out, void* y, void* ws, size_t ws_bytes, void* stream)
{
    if (!valid_sizes(xdt, M, K, N) || !valid_act(act) || !gate || !up) return QB_EINVAL;
    const Weight4 w[2] = {weight_of(*gate), weight_of(*up)};
    Weight4Format f{0, 0, 0, w[0].c2 ? 1 : 0};
    qb_status st = check_format(code, blocksize, blocksize2, N, K, &f);
    if (st != QB_OK) return st;
    if (M == 0 || N == 0) return QB_OK;
    if (!x || !y) return QB_EINVAL;
    int nested = -1;
    for (const Weight4& v : w) {
        st = check_weight(v, &nested);
        if (st != QB_OK) return st;
    }
    if (!aligned16(x) || !aligned16(gate_out) || !aligned16(up_out) || !aligned16(y)) return QB_EALIGN;
    st = check_ws(forward_bytes(xdt, M, K, N, 2), ws, ws_bytes);
    if (st != QB_OK) return st;
    hipStream_t s = static_cast<hipStream_t>(stream);
    const Epilogue e{nullptr, nullptr, gate_out, up_out, y, N, 0, (int32_t)act};
    if (rows_win(xdt, M, K, N, 2)) return hip_status(launch_linear_rows(xdt, x, M, K, w, 2, f, e, s));
    return hip_status(unpack_and_multiply(xdt, x, M, K, w, 2, N, f, e, ws, s));
}

size_t qb_dequant_gated_backward_workspace_bytes(qb_dtype xdt, int64_t M, int64_t K, int64_t N)
{
    return valid_sizes(xdt, M, K, N) && N > 0 ? backward_layout(xdt, M, K, N, 2).bytes : 0;
}

qb_status qb_dequant_gated_backward(const void* dy, const void* gate_out, const void* up_out, qb_dtype xdt, int64_t M,
                                    int64_t K, const qb_weight* gate, const qb_weight* up, qb_code code,
                                    int32_t blocksize, int32_t blocksize2, int64_t N, qb_act act, void* dx,
                                    void* dgate, void* dup, void* ws, size_t ws_bytes, void* stream)
{
    if (!valid_sizes(xdt, M, K, N) || N == 0 || !valid_act(act) || !gate || !up) return QB_EINVAL;
    const Weight4 w[2] = {weight_of(*gate), weight_of(*up)};
    Weight4Format f{0, 0, 0, w[0].c2 ? 1 : 0};
    qb_status st = check_format(code, blocksize, blocksize2, N, K, &f);
    if (st != QB_OK) return st;
    if (M == 0 || (!dx && !dgate && !dup)) return QB_OK;
    if (!dy || !gate_out || !up_out) return QB_EINVAL;
    int nested = -1;
    for (const Weight4& v : w) {
        st = dx ? check_weight(v, &nested) : QB_OK;
        if (st != QB_OK) return st;
    }
    if (!aligned16(dy) || !aligned16(gate_out) || !aligned16(up_out) || !aligned16(dx) || !aligned16(dgate) ||
        !aligned16(dup))
        return QB_EALIGN;
    const BackwardLayout l = backward_layout(xdt, M, K, N, 2);
    st = check_ws(dx ? l.bytes : 0, ws, ws_bytes);
    if (st != QB_OK) return st;
    hipStream_t s = static_cast<hipStream_t>(stream);
    char* const wp = static_cast<char*>(ws);
    const int64_t pitch = gemm_pitch(xdt, N);
    const bool given = dgate && dup && whole_steps(xdt, N);       // dx reads the caller's arrays
    const TransposedWeights t = transposed(xdt, w, 2, f, K, N, wp);
    hipError_t e = launch_gated_grad(xdt, dy, gate_out, up_out, act, M, N, dx && !given ? wp + l.dz : nullptr, pitch, dgate,
                                     dup, dx && !few_rows(xdt, M, K, N, 2) ? &t : nullptr, s);
    if (e == hipSuccess && dx) {
        const void* const dg = given ? dgate : wp + l.dz;
        const void* const du = given ? dup : wp + l.dz + (size_t)M * pitch * dtype_bytes(xdt);
        e = input_gradient(xdt, dg, du, pitch, t, M, dx, reinterpret_cast<float*>(wp + l.split), nullptr, s);
    }
    return hip_status(e);
}

size_t qb_multi_tensor_grad_norm_workspace_bytes(int32_t count)
{
    if (count <= 0) return 0;
    return (size_t)((count + kNormGrads - 1) / kNormGrads) * kNormGroups * sizeof(double);
}

}  // extern "C"

namespace {

bool aligned_to(const void* p, int bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }

qb_status check_grads(const qb_grad* grads, int32_t count, bool out)
{
    if (count < 0 || (count > 0 && !grads)) return QB_EINVAL;
    for (int32_t i = 0; i < count; ++i) {
        const qb_grad& t = grads[i];
        if (t.n < 0 || !valid_dtype(t.dtype)) return QB_EINVAL;
        if (t.n == 0) continue;
        if (!t.g || (out && !t.out) || t.n >= kGradMax) return QB_EINVAL;
        const int e = dtype_bytes(t.dtype);
        if (!aligned_to(t.g, e) || (out && !aligned_to(t.out, e))) return QB_EALIGN;
    }
    return QB_OK;
}

uint64_t size_of(const qb_grad& g) { return (uint64_t)g.n << 2 | (uint64_t)g.dtype; }

int32_t tiles_of(const qb_grad& g)
{
    const int64_t tile = grad_tile_elems(g.dtype);
    return (int32_t)((g.n + tile - 1) / tile);
}

const char* end_of(const void* p, const qb_grad& g) { return static_cast<const char*>(p) + g.n * dtype_bytes(g.dtype); }

// Whether gradient b, and its output, begin where those of a end, as neighbours of a bucket do.
bool joins(const qb_grad& a, const qb_grad& b, bool out)
{
    return a.dtype == b.dtype && a.n + b.n < kGradMax && end_of(a.g, a) == b.g && (!out || end_of(a.out, a) == b.out);
}

// The next launch's gradients, empty ones left out and neighbours joined into one (448 views of a
// bucket, 65536 binary32 each: 60 us for norm and clipping, 73 in entries of their own): from *at on ...
void next_table(const qb_grad* grads, int32_t count, int32_t* at, NormTable* t)
{
    t->count = t->tiles = 0;
    while (t->count < kNormGrads && *at < count) {
        qb_grad g = grads[(*at)++];
        if (g.n == 0) continue;
        for (; *at < count && (grads[*at].n == 0 || joins(g, grads[*at], false)); ++*at) g.n += grads[*at].n;
        t->g[t->count] = g.g;
        t->size[t->count++] = size_of(g);
        t->tiles += tiles_of(g);
    }
}

// ... or from *at back.
void next_table(const qb_grad* grads, int32_t* at, ScaleTable* t)
{
    t->count = t->tiles = 0;
    while (t->count < kScaleGrads && *at >= 0) {
        qb_grad g = grads[(*at)--];
        if (g.n == 0) continue;
        for (; *at >= 0 && (grads[*at].n == 0 || joins(grads[*at], g, true)); --*at) {
            const qb_grad& before = grads[*at];
            if (before.n == 0) continue;
            g.g = before.g;
            g.out = before.out;
            g.n += before.n;
        }
        t->g[t->count] = g.g;
        t->out[t->count] = g.out;
        t->size[t->count++] = size_of(g);
        t->tiles += tiles_of(g);
    }
}

}  // namespace

extern "C" {

qb_status qb_multi_tensor_grad_norm(const qb_grad* grads, int32_t count, float* norm, void* ws, size_t ws_bytes,
                                    void* stream)
{
    qb_status st = check_grads(grads, count, false);
    if (st != QB_OK) return st;
    if (!norm) return QB_EINVAL;
    if (!aligned16(norm)) return QB_EALIGN;
    st = check_ws(qb_multi_tensor_grad_norm_workspace_bytes(count), ws, ws_bytes);
    if (st != QB_OK) return st;
    hipStream_t s = static_cast<hipStream_t>(stream);
    double* const part = static_cast<double*>(ws);
    int32_t at = 0;
    int parts = 0;
    while (at < count) {
        NormTable t;
        const bool first = at == 0;
        next_table(grads, count, &at, &t);
        if (t.count == 0) continue;
        int groups = 0;
        const bool few = first && at >= count && t.tiles <= kNormFewTiles;
        const hipError_t e = launch_grad_squares(t, part + parts, &groups, few ? norm : nullptr, s);
        if (e != hipSuccess || few) return hip_status(e);
        parts += groups;
    }
    return hip_status(launch_grad_norm(part, parts, norm, s));
}

qb_status qb_multi_tensor_clip_grads(const qb_grad* grads, int32_t count, double max_norm, const float* norm,
                                     void* stream)
{
    qb_status st = check_grads(grads, count, true);
    if (st != QB_OK) return st;
    if (!std::isfinite(max_norm) || max_norm < 0 || !norm) return QB_EINVAL;
    if (!aligned16(norm)) return QB_EALIGN;
    int32_t at = count - 1;
    while (at >= 0) {
        ScaleTable t;
        next_table(grads, &at, &t);
        if (t.count == 0) continue;
        const hipError_t e = launch_grad_scale(t, max_norm, norm, static_cast<hipStream_t>(stream));
        if (e != hipSuccess) return hip_status(e);
    }
    return QB_OK;
}

}  // extern "C"
