// Sanitizer driver for the host code of libqb's row-wise layers
// (qb_layers_api.cpp; test infrastructure): argument checks, workspace sizes and
// host arithmetic of every entry point over ordinary, extreme and invalid sizes,
// built with -fsanitize=address,undefined.  The launchers below stand in for the
// HIP sources: they enqueue nothing and check that what they are given lies
// inside the workspace.  Exits non-zero on the first unexpected status.
#include <algorithm>
#include <cmath>
#include <cstdio>

#include "qb.h"
#include "qb_layers.h"

static int failures = 0, launches = 0;
static char* ws_begin = nullptr;
static size_t ws_bytes = 0;

#define EXPECT(call, want)                                                                          \
    do {                                                                                            \
        const int got_ = (int)(call);                                                               \
        if (got_ != (int)(want)) {                                                                  \
            std::fprintf(stderr, "line %d: %s returned %d, expected %d\n", __LINE__, #call, got_,   \
                         (int)(want));                                                              \
            ++failures;                                                                             \
        }                                                                                           \
    } while (0)

static void inside(const void* p, double bytes)
{
    const char* c = static_cast<const char*>(p);
    if (c < ws_begin || (double)(c - ws_begin) + bytes > (double)ws_bytes) {
        std::fprintf(stderr, "an array of %.0f bytes leaves the workspace\n", bytes);
        ++failures;
    }
}

namespace qb {

const QbTables* device_tables() { return reinterpret_cast<const QbTables*>(uintptr_t(64)); }

static hipError_t done() { ++launches; return hipSuccess; }

hipError_t launch_embedding(const IdArgs&, const void*, int, float, void*, int, hipStream_t) { return done(); }
hipError_t launch_dequant_embedding(const IdArgs&, const DequantDesc&, int, int, int, int, float, void*, int,
                                    hipStream_t)
{
    return done();
}
hipError_t launch_order(const IdArgs& a, const OrderArgs& o, hipStream_t)
{
    const double classes = (double)(int64_t(1) << o.log2g);
    if (classes * o.per < (double)a.rows || o.per > kOrderPerMax || o.per < 1) ++failures;
    inside(o.start, (classes * o.per + 1) * 4);
    inside(o.order, (double)a.n * 4);
    inside(o.key, (double)a.n * 4);
    if (o.chunk < 1 || o.chunk > 32) ++failures;       // two chunks are one wave's lanes
    return done();
}
hipError_t launch_prepare_grad(const IdArgs& a, const OrderArgs& o, const void*, int, float* part, int64_t,
                               bool, void*, int, hipStream_t)
{
    inside(o.used, (double)(int64_t(2) << o.log2g) * 4);
    inside(o.count, 8);
    inside(o.longs, (double)(a.n / o.chunk + 1) * 4);
    inside(o.list, (double)(a.n < a.rows ? a.n : a.rows) * 16);
    inside(part, 2.0 * (double)chunk_count(a.n) * (double)padded_dim(a.dim) * 4);
    return done();
}
hipError_t launch_table_grad(const IdArgs& a, const OrderArgs& o, const void*, int, float* part, float, int64_t, bool,
                             void*, int, hipStream_t)
{
    inside(o.count, 8);
    inside(o.longs, (double)(a.n / o.chunk + 1) * 4);
    inside(part, 2.0 * (double)chunk_count(a.n) * (double)padded_dim(a.dim) * 4);
    return done();
}
hipError_t launch_join_chunks(const IdArgs&, const OrderArgs&, float*, hipStream_t) { return done(); }
hipError_t launch_table_grad_direct(const IdArgs& a, const void*, int, float, int64_t, bool, void*, int, hipStream_t)
{
    if (a.n < 1 || a.n > kDirectTokens || a.rows < 1) ++failures;
    return done();
}
hipError_t launch_stable_grad_direct(const IdArgs& a, const void*, int, const void*, int, float, const NormArgs&, int64_t,
                                     bool, void*, int, float* part, hipStream_t)
{
    if (a.n < 1 || a.n > kDirectTokens || a.rows < 1) ++failures;
    inside(part, 2.0 * (double)a.n * (double)padded_dim(a.dim) * 4);
    return done();
}
hipError_t launch_layer_norm(const void*, int, int64_t, int64_t, const NormArgs&, void*, float*, float*, hipStream_t)
{
    return done();
}
hipError_t launch_stable_embedding(const IdArgs&, const void*, int, float, const NormArgs&, void*, int, hipStream_t)
{
    return done();
}
// the number of workgroups is the HIP sources' choice, at most one per row and kNormPartsMax
int layer_norm_parts(int64_t n, int64_t) { return (int)(n < kNormPartsMax ? n : kNormPartsMax); }
int stable_parts(int64_t n, int64_t rows)
{
    return rows > 0 && takes_direct(n, rows) ? (int)n : (int)std::min<int64_t>(kNormPartsMax, std::min(n, rows));
}
hipError_t launch_layer_norm_grad(const void*, const void*, int, int64_t n, int64_t dim, const void*, int,
                                  const float*, const float*, void*, float* part, hipStream_t)
{
    if (part) inside(part, 2.0 * layer_norm_parts(n, dim) * (double)padded_dim(dim) * 4);
    return done();
}
hipError_t launch_stable_grad(const IdArgs& a, const OrderArgs&, const void*, int, const float*, const void*, int, float,
                              const NormArgs&, int64_t, bool, void*, int, float* part, int parts, hipStream_t)
{
    inside(part, 2.0 * parts * (double)padded_dim(a.dim) * 4);
    return done();
}
hipError_t launch_join_parts(const float*, int, int64_t, bool, void*, void*, int, hipStream_t) { return done(); }

}  // namespace qb

int main()
{
    char* const D = reinterpret_cast<char*>(uintptr_t(1) << 40);       // fake device addresses, never dereferenced
    void* const A = D;
    void* const B = D + 4096;
    float* const F = reinterpret_cast<float*>(D + 8192);
    uint8_t* const U = reinterpret_cast<uint8_t*>(D + 16384);
    ws_begin = reinterpret_cast<char*>(uintptr_t(1) << 41);
    const int64_t top = (int64_t(1) << 31) - 1;

    for (int64_t n : {int64_t(0), int64_t(1), int64_t(63), int64_t(128), int64_t(129), int64_t(5003), int64_t(1) << 20,
                      int64_t(1) << 30, top})
        for (int64_t rows : {int64_t(0), int64_t(1), int64_t(2), int64_t(255), int64_t(257), int64_t(32000),
                             int64_t(256001), int64_t(1) << 26})
            for (int64_t dim : {int64_t(1), int64_t(8), int64_t(1001), int64_t(16384), (int64_t(1) << 24) - 1}) {
                const bool takes = n <= int64_t(1) << 30;
                ws_bytes = qb_embedding_workspace_bytes(n, rows, dim);
                EXPECT(ws_bytes != 0, takes);
                EXPECT(qb_embedding_backward(A, QB_BF16, B, QB_I64, n, rows, dim, 0.5, -1, 0, A, QB_F32, ws_begin,
                                             ws_bytes, nullptr), takes ? QB_OK : QB_EINVAL);
                EXPECT(qb_embedding(A, QB_F32, rows, dim, B, QB_I32, n, 2.0, A, QB_F16, nullptr), QB_OK);
                const bool fits = dim <= 16384;
                ws_bytes = qb_stable_embedding_workspace_bytes(n, rows, dim);
                EXPECT(ws_bytes != 0, fits && takes);
                EXPECT(qb_stable_embedding_backward(A, QB_F16, B, QB_F32, rows, dim, B, QB_I32, n, 1.0, A, QB_F32, 1e-5,
                                                    3, 0, A, QB_F32, A, A, ws_begin, ws_bytes, nullptr),
                       !takes ? QB_EINVAL : fits ? QB_OK : QB_EUNSUPPORTED);
                EXPECT(qb_stable_embedding(A, QB_F32, rows, dim, B, QB_I32, n, 1.0, A, nullptr, QB_F32, 1e-5, A, QB_F32,
                                           nullptr), fits ? QB_OK : QB_EUNSUPPORTED);
                // at most 2^31 - 1 blocks in a quantized table
                EXPECT(qb_dequant_embedding(U, F, nullptr, QB_NF4, 64, rows, dim, B, QB_I64, n, 1.0, A, QB_BF16,
                                            nullptr), n > 0 && (rows * dim + 63) / 64 > top ? QB_EINVAL : QB_OK);
            }
    for (int64_t n : {int64_t(0), int64_t(1), int64_t(511), int64_t(1) << 20, top})
        for (int64_t dim : {int64_t(1), int64_t(4096), int64_t(16385), (int64_t(1) << 24) - 1, int64_t(1) << 24}) {
            const bool fits = dim < int64_t(1) << 24;
            ws_bytes = qb_layer_norm_workspace_bytes(n, dim);
            EXPECT(qb_layer_norm_backward(A, B, QB_F32, n, dim, A, QB_F32, F, F, A, A, A, 0, ws_begin, ws_bytes, nullptr),
                   fits ? QB_OK : QB_EINVAL);
            EXPECT(qb_layer_norm(A, QB_F16, n, dim, nullptr, nullptr, QB_F16, 1e-5, A, F, F, nullptr),
                   fits ? QB_OK : QB_EINVAL);
        }
    const int before = launches;
    EXPECT(qb_embedding(A, QB_F32, 10, 8, B, QB_I32, 4, std::nan(""), A, QB_F16, nullptr), QB_EINVAL);
    EXPECT(qb_embedding(D + 4, QB_F32, 10, 8, B, QB_I32, 4, 1.0, A, QB_F16, nullptr), QB_EALIGN);
    EXPECT(qb_layer_norm(A, QB_F16, 4, 8, A, A, QB_BF16, 1e-5, A, F, F, nullptr), QB_EUNSUPPORTED);
    EXPECT(qb_embedding_backward(A, QB_F32, B, QB_I32, 4, 10, 8, 1.0, -1, 0, A, QB_F32, ws_begin, 16, nullptr),
           QB_EWORKSPACE);
    EXPECT(launches, before);
    if (failures == 0) std::printf("every call returned the expected status (%d launches)\n", launches);
    return failures == 0 ? 0 : 1;
}
