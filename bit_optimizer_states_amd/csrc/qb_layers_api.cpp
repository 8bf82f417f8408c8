// qb_layers_api.cpp -- the C ABI of the row-wise layers (embedding lookup, layer
// norm, stable embedding) declared in include/qb.h: argument validation,
// workspace layout and dispatch.  Nothing is enqueued unless every argument
// checks out.
#include <hip/hip_runtime.h>

#include <cmath>

#include "qb.h"
#include "qb_layers.h"

namespace {

using namespace qb;

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool valid_dtype(qb_dtype d) { return d == QB_F32 || d == QB_F16 || d == QB_BF16; }
bool valid_index(qb_index i) { return i == QB_I32 || i == QB_I64; }
bool pow2_block(int32_t b) { return b >= 64 && b <= 4096 && (b & (b - 1)) == 0; }
bool is4(qb_code c) { return c == QB_NF4 || c == QB_FP4; }
size_t round_up(size_t v, size_t a) { return (v + a - 1) / a * a; }

constexpr int64_t kIndexMax = int64_t(1) << 31;      // tokens, rows
constexpr int64_t kDimMax = int64_t(1) << 24;        // elements of a row
constexpr int64_t kGradRowsMax = int64_t(1) << 26;   // rows of a table that takes a gradient
constexpr int64_t kGradTokensMax = int64_t(1) << 30; // tokens of a gradient

qb_status hip_status(hipError_t e)
{
    if (e == hipSuccess) return QB_OK;
    if (e == hipErrorNotInitialized) return QB_EINIT;
    return QB_EHIP;
}

bool valid_lookup(int64_t n, int64_t rows, int64_t dim, qb_index idt, double scale)
{
    return n >= 0 && n < kIndexMax && rows >= 0 && rows < kIndexMax && dim >= 1 && dim < kDimMax && valid_index(idt) &&
           std::isfinite(scale) && std::isfinite((float)scale);
}

IdArgs id_args(const void* ids, qb_index idt, int64_t n, int64_t rows, int64_t dim)
{
    return IdArgs{ids, n, rows, idt == QB_I64 ? 1 : 0, (int32_t)dim};
}

// An eps that is a positive normal binary32: a row of equal values then has a finite rstd.
bool valid_eps(double eps) { return std::isfinite(eps) && (float)eps >= 0x1p-126f && std::isfinite((float)eps); }

// Workspace of a table's gradient: the arrays of OrderArgs, the chunks' sums; then
// (stable) the partial sums of dgamma and dbeta; then the ordering's parts, where it
// takes them.
struct GradLayout {
    size_t order, key, used, list, longs, chunks, parts, split, bytes;
};

size_t longs_bytes(int64_t n, int32_t chunk) { return round_up((size_t)(n / chunk + 1) * sizeof(int32_t), 256); }

// The list of long ids and the chunks' sums.
size_t chunk_bytes(int64_t n, int64_t dim, int32_t chunk)
{
    return longs_bytes(n, chunk) + (size_t)(2 * chunk_count(n, chunk) * padded_dim(dim)) * sizeof(float);
}

// As much for whichever chunks a call takes: the size never shrinks when tokens or
// elements are added, so a workspace for the largest batch serves every smaller one.
// Short chunks are at most kChunkWaves waves of 512 columns.
constexpr size_t kShortBytesMax = (size_t)2 * kChunkWaves * 512 * sizeof(float) +
                                  ((size_t)(kChunkWaves + 1) * sizeof(int32_t) + 255) / 256 * 256;

size_t chunk_bytes_reserved(int64_t n, int64_t dim)
{
    const size_t s = chunk_bytes(n, dim, kChunkShort), l = chunk_bytes(n, dim, kChunkLong);
    const size_t at_most = s < kShortBytesMax ? s : kShortBytesMax;
    return l > at_most ? l : at_most;
}

constexpr size_t split_start_bytes = ((kOrderParts + 1) * sizeof(int32_t) + 255) / 256 * 256;
size_t split_bytes(int64_t n) { return round_up((size_t)n * sizeof(int32_t), 256); }

GradLayout grad_layout(int64_t n, int64_t rows, int64_t dim, int64_t parts)
{
    GradLayout l;
    const int64_t classes = int64_t(1) << order_log2g(rows), entries = classes * order_per(rows) + 1;
    l.order = round_up((size_t)entries * sizeof(int32_t), 256);
    l.key = l.order + round_up((size_t)n * sizeof(int32_t), 256);
    l.used = l.key + round_up((size_t)n * sizeof(int32_t), 256);
    l.list = l.used + round_up((size_t)(2 * classes + 2) * sizeof(int32_t), 256);
    l.longs = l.list + round_up((size_t)(n < rows ? n : rows) * 4 * sizeof(int32_t), 256);
    l.chunks = l.longs + longs_bytes(n, chunk_tokens(n, dim));
    l.parts = l.longs + chunk_bytes_reserved(n, dim);
    l.split = l.parts + (size_t)parts * 2 * (size_t)padded_dim(dim) * sizeof(float);
    l.bytes = l.split + (order_in_parts(n, rows) ? split_start_bytes + 2 * split_bytes(n) : 0);
    return l;
}

// Partial rows that the stable embedding's workspace holds: those of up to
// kDirectTokens tokens, one each, are more than those of more tokens of few ids.
int64_t stable_parts_reserved(int64_t n, int64_t rows)
{
    const int64_t parts = stable_parts(n, rows), direct = n < kDirectTokens ? n : kDirectTokens;
    return rows > 0 && direct > parts ? direct : parts;
}

OrderArgs order_args(void* ws, const GradLayout& l, int64_t n, int64_t rows, int64_t dim)
{
    char* const w = static_cast<char*>(ws);
    auto at = [w](size_t offset) { return reinterpret_cast<int32_t*>(w + offset); };
    const bool parts = order_in_parts(n, rows);
    int32_t* const used = at(l.used);
    return OrderArgs{at(0), at(l.order), at(l.key), used, used + (int64_t(2) << order_log2g(rows)), at(l.list),
                     at(l.longs), order_log2g(rows), (int32_t)order_per(rows), chunk_tokens(n, dim),
                     parts ? at(l.split) : nullptr, parts ? at(l.split + split_start_bytes) : nullptr,
                     parts ? at(l.split + split_start_bytes + split_bytes(n)) : nullptr};
}

bool valid_grad_sizes(int64_t n, int64_t rows, int64_t dim)
{
    return n >= 0 && n <= kGradTokensMax && rows >= 0 && rows <= kGradRowsMax && dim >= 1 && dim < kDimMax;
}

// Checks shared by the two gradients of a table.
qb_status check_table_grad(const void* dy, qb_dtype gdt, const void* ids, qb_index idt, int64_t n, int64_t rows,
                           int64_t dim, double scale, int64_t padding_id, const void* dtable, qb_dtype ddt)
{
    if (!valid_lookup(n, rows, dim, idt, scale) || !valid_grad_sizes(n, rows, dim) || !valid_dtype(gdt) ||
        !valid_dtype(ddt) || padding_id < -1 || padding_id >= kIndexMax)
        return QB_EINVAL;
    if (n > 0 && (!dy || !ids)) return QB_EINVAL;
    if (rows > 0 && !dtable) return QB_EINVAL;
    if (!aligned16(dy) || !aligned16(ids) || !aligned16(dtable)) return QB_EALIGN;
    return QB_OK;
}

}  // namespace

extern "C" {

qb_status qb_embedding(const void* table, qb_dtype tdt, int64_t rows, int64_t dim, const void* ids, qb_index idt,
                       int64_t n, double scale, void* y, qb_dtype ydt, void* stream)
{
    if (!valid_lookup(n, rows, dim, idt, scale) || !valid_dtype(tdt) || !valid_dtype(ydt)) return QB_EINVAL;
    if (n == 0) return QB_OK;
    if ((rows > 0 && !table) || !ids || !y) return QB_EINVAL;
    if (!aligned16(table) || !aligned16(ids) || !aligned16(y)) return QB_EALIGN;
    return hip_status(launch_embedding(id_args(ids, idt, n, rows, dim), table, (int)tdt, (float)scale, y, (int)ydt,
                                       static_cast<hipStream_t>(stream)));
}

qb_status qb_dequant_embedding(const uint8_t* codes, const float* absmax, const qb_dq* dq, qb_code code,
                               int32_t blocksize, int64_t rows, int64_t dim, const void* ids, qb_index idt, int64_t n,
                               double scale, void* y, qb_dtype ydt, void* stream)
{
    if (!valid_lookup(n, rows, dim, idt, scale) || !valid_dtype(ydt) || (code != QB_DYN8 && !is4(code)) ||
        !pow2_block(blocksize))
        return QB_EINVAL;
    if (n == 0) return QB_OK;
    if (!ids || !y) return QB_EINVAL;
    if (!aligned16(ids) || !aligned16(y) || !aligned16(codes) || !aligned16(absmax)) return QB_EALIGN;
    DequantDesc d{};
    if (rows > 0) {
        if (!codes) return QB_EINVAL;
        if ((rows * dim + blocksize - 1) / blocksize >= kIndexMax) return QB_EINVAL;
        if (dq) {
            if (absmax || !dq->codes || !dq->absmax2 || !dq->offset || !pow2_block(dq->blocksize2)) return QB_EINVAL;
            if (!aligned16(dq->codes) || !aligned16(dq->absmax2) || !aligned16(dq->offset)) return QB_EALIGN;
        } else if (!absmax) {
            return QB_EINVAL;
        }
    }
    if (!device_tables()) return QB_EINIT;
    if (rows == 0)                     // every id is outside the table
        return hip_status(launch_embedding(id_args(ids, idt, n, 0, dim), nullptr, QB_F32, 0.0f, y, (int)ydt,
                                           static_cast<hipStream_t>(stream)));
    d.codes = codes;
    d.absmax = absmax;
    d.c2 = dq ? dq->codes : nullptr;
    d.absmax2 = dq ? dq->absmax2 : nullptr;
    d.offset = dq ? dq->offset : nullptr;
    return hip_status(launch_dequant_embedding(id_args(ids, idt, n, rows, dim), d, is4(code) ? 4 : 8,
                                               code == QB_FP4 ? 1 : 0, blocksize, dq ? dq->blocksize2 : 256,
                                               (float)scale, y, (int)ydt, static_cast<hipStream_t>(stream)));
}

size_t qb_embedding_workspace_bytes(int64_t n, int64_t rows, int64_t dim)
{
    return valid_grad_sizes(n, rows, dim) ? grad_layout(n, rows, dim, 0).bytes : 0;
}

qb_status qb_embedding_backward(const void* dy, qb_dtype gdt, const void* ids, qb_index idt, int64_t n, int64_t rows,
                                int64_t dim, double scale, int64_t padding_id, int32_t accumulate, void* dtable,
                                qb_dtype ddt, void* ws, size_t ws_bytes, void* stream)
{
    qb_status st = check_table_grad(dy, gdt, ids, idt, n, rows, dim, scale, padding_id, dtable, ddt);
    if (st != QB_OK) return st;
    if (accumulate != 0 && accumulate != 1) return QB_EINVAL;
    if (rows == 0 || (n == 0 && accumulate)) return QB_OK;
    if (!ws) return QB_EINVAL;
    if (!aligned16(ws)) return QB_EALIGN;
    const GradLayout l = grad_layout(n, rows, dim, 0);
    if (ws_bytes < l.bytes) return QB_EWORKSPACE;
    const IdArgs a = id_args(ids, idt, n, rows, dim);
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (takes_direct(n, rows))
        return hip_status(launch_table_grad_direct(a, dy, (int)gdt, (float)scale, padding_id, accumulate != 0, dtable,
                                                   (int)ddt, s));
    const OrderArgs o = order_args(ws, l, n, rows, dim);
    float* const part = reinterpret_cast<float*>(static_cast<char*>(ws) + l.chunks);
    hipError_t e = launch_order(a, o, s);
    if (e == hipSuccess)
        e = launch_table_grad(a, o, dy, (int)gdt, part, (float)scale, padding_id, accumulate != 0, dtable, (int)ddt, s);
    return hip_status(e);
}

qb_status qb_layer_norm(const void* x, qb_dtype xdt, int64_t n, int64_t dim, const void* gamma, const void* beta,
                        qb_dtype wdt, double eps, void* y, float* mean, float* rstd, void* stream)
{
    if (n < 0 || n >= kIndexMax || dim < 1 || dim >= kDimMax || !valid_dtype(xdt) || !valid_dtype(wdt) ||
        !valid_eps(eps))
        return QB_EINVAL;
    if (wdt != QB_F32 && wdt != xdt) return QB_EUNSUPPORTED;
    if (n == 0) return QB_OK;
    if (!x || !y) return QB_EINVAL;
    if (!aligned16(x) || !aligned16(gamma) || !aligned16(beta) || !aligned16(y) || !aligned16(mean) || !aligned16(rstd))
        return QB_EALIGN;
    return hip_status(launch_layer_norm(x, (int)xdt, n, dim, NormArgs{gamma, beta, (int)wdt, (float)eps}, y, mean, rstd,
                                        static_cast<hipStream_t>(stream)));
}

size_t qb_layer_norm_workspace_bytes(int64_t n, int64_t dim)
{
    if (n < 0 || n >= kIndexMax || dim < 1 || dim >= kDimMax) return 0;
    const int64_t parts = n < kNormPartsMax ? (n > 0 ? n : 1) : kNormPartsMax;
    return (size_t)(parts * 2 * padded_dim(dim)) * sizeof(float);
}

qb_status qb_layer_norm_backward(const void* dy, const void* x, qb_dtype xdt, int64_t n, int64_t dim,
                                 const void* gamma, qb_dtype wdt, const float* mean, const float* rstd, void* dx,
                                 void* dgamma, void* dbeta, int32_t accumulate, void* ws, size_t ws_bytes,
                                 void* stream)
{
    if (n < 0 || n >= kIndexMax || dim < 1 || dim >= kDimMax || !valid_dtype(xdt) || !valid_dtype(wdt) ||
        (accumulate != 0 && accumulate != 1))
        return QB_EINVAL;
    if (wdt != QB_F32 && wdt != xdt) return QB_EUNSUPPORTED;
    const bool weights = dgamma || dbeta;
    if (n == 0 && (!weights || accumulate)) return QB_OK;
    if (!dx && !weights) return QB_OK;
    if (n > 0 && (!dy || !x || !mean || !rstd)) return QB_EINVAL;
    if (!aligned16(dy) || !aligned16(x) || !aligned16(gamma) || !aligned16(mean) || !aligned16(rstd) ||
        !aligned16(dx) || !aligned16(dgamma) || !aligned16(dbeta))
        return QB_EALIGN;
    if (weights) {
        if (!ws) return QB_EINVAL;
        if (!aligned16(ws)) return QB_EALIGN;
        if (ws_bytes < qb_layer_norm_workspace_bytes(n, dim)) return QB_EWORKSPACE;
    }
    float* const part = weights ? static_cast<float*>(ws) : nullptr;
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (n > 0) {
        const hipError_t e = launch_layer_norm_grad(dy, x, (int)xdt, n, dim, gamma, (int)wdt, mean, rstd, dx, part, s);
        if (e != hipSuccess) return hip_status(e);
    }
    return hip_status(launch_join_parts(part, n > 0 ? layer_norm_parts(n, dim) : 0, dim, accumulate != 0, dgamma, dbeta,
                                        (int)wdt, s));
}

qb_status qb_stable_embedding(const void* table, qb_dtype tdt, int64_t rows, int64_t dim, const void* ids,
                              qb_index idt, int64_t n, double scale, const void* gamma, const void* beta, qb_dtype wdt,
                              double eps, void* y, qb_dtype ydt, void* stream)
{
    if (!valid_lookup(n, rows, dim, idt, scale) || !valid_dtype(tdt) || !valid_dtype(ydt) || !valid_dtype(wdt) ||
        !valid_eps(eps))
        return QB_EINVAL;
    if (dim > kRowRegMax || (wdt != QB_F32 && wdt != tdt)) return QB_EUNSUPPORTED;
    if (n == 0) return QB_OK;
    if ((rows > 0 && !table) || !ids || !y) return QB_EINVAL;
    if (!aligned16(table) || !aligned16(ids) || !aligned16(gamma) || !aligned16(beta) || !aligned16(y))
        return QB_EALIGN;
    return hip_status(launch_stable_embedding(id_args(ids, idt, n, rows, dim), table, (int)tdt, (float)scale,
                                              NormArgs{gamma, beta, (int)wdt, (float)eps}, y, (int)ydt,
                                              static_cast<hipStream_t>(stream)));
}

size_t qb_stable_embedding_workspace_bytes(int64_t n, int64_t rows, int64_t dim)
{
    if (!valid_grad_sizes(n, rows, dim) || dim > kRowRegMax) return 0;
    return grad_layout(n, rows, dim, stable_parts_reserved(n, rows)).bytes;
}

qb_status qb_stable_embedding_backward(const void* dy, qb_dtype gdt, const void* table, qb_dtype tdt, int64_t rows,
                                       int64_t dim, const void* ids, qb_index idt, int64_t n, double scale,
                                       const void* gamma, qb_dtype wdt, double eps, int64_t padding_id,
                                       int32_t accumulate, void* dtable, qb_dtype ddt, void* dgamma, void* dbeta,
                                       void* ws, size_t ws_bytes, void* stream)
{
    qb_status st = check_table_grad(dy, gdt, ids, idt, n, rows, dim, scale, padding_id, dtable, ddt);
    if (st != QB_OK) return st;
    if (!valid_dtype(tdt) || !valid_dtype(wdt) || !valid_eps(eps) || (accumulate != 0 && accumulate != 1))
        return QB_EINVAL;
    if (dim > kRowRegMax || (wdt != QB_F32 && wdt != tdt)) return QB_EUNSUPPORTED;
    if (rows > 0 && n > 0 && !table) return QB_EINVAL;
    if (!aligned16(table) || !aligned16(gamma) || !aligned16(dgamma) || !aligned16(dbeta)) return QB_EALIGN;
    if (n == 0 && accumulate) return QB_OK;
    if (!ws) return QB_EINVAL;
    if (!aligned16(ws)) return QB_EALIGN;
    const int parts = stable_parts(n, rows);
    const GradLayout l = grad_layout(n, rows, dim, stable_parts_reserved(n, rows));
    if (ws_bytes < l.bytes) return QB_EWORKSPACE;
    char* const w = static_cast<char*>(ws);
    const IdArgs a = id_args(ids, idt, n, rows, dim);
    const OrderArgs o = order_args(ws, l, n, rows, dim);
    float* const chunks = reinterpret_cast<float*>(w + l.chunks);
    float* const part = reinterpret_cast<float*>(w + l.parts);
    hipStream_t s = static_cast<hipStream_t>(stream);
    const NormArgs norm{gamma, nullptr, (int)wdt, (float)eps};
    hipError_t e = hipSuccess;
    if (rows > 0 && takes_direct(n, rows)) {
        e = launch_stable_grad_direct(a, dy, (int)gdt, table, (int)tdt, (float)scale, norm, padding_id, accumulate != 0,
                                      dtable, (int)ddt, part, s);
    } else if (rows > 0) {
        e = launch_order(a, o, s);
        if (e == hipSuccess)
            e = launch_prepare_grad(a, o, dy, (int)gdt, chunks, padding_id, accumulate != 0, dtable, (int)ddt, s);
        if (e == hipSuccess) e = launch_join_chunks(a, o, chunks, s);
        if (e == hipSuccess)
            e = launch_stable_grad(a, o, dy, (int)gdt, chunks, table, (int)tdt, (float)scale,
                                   norm, padding_id, accumulate != 0, dtable, (int)ddt, part, parts, s);
    }
    if (e == hipSuccess) e = launch_join_parts(part, parts, dim, accumulate != 0, dgamma, dbeta, (int)wdt, s);
    return hip_status(e);
}

}  // extern "C"
