// Sanitizer driver for the host code of the 4-bit layers and the gradient norm
// (qb_linear_api.cpp; test infrastructure): argument checks, workspace layouts and host
// arithmetic of every entry point over ordinary, extreme and invalid sizes, built with
// -fsanitize=address,undefined.  The launchers below stand in for the HIP sources: they
// enqueue nothing and check that what they are given lies inside the workspace, and that
// every gradient is handed over once.  Exits non-zero on the first unexpected status.
#include <cmath>
#include <cstdio>
#include <vector>

#include "qb.h"
#include "qb_clip.h"
#include "qb_linear.h"

static int failures = 0, launches = 0;
static char* ws_begin = nullptr;
static size_t ws_bytes = 0;
static long long seen_elements = 0;

#define EXPECT(call, want)                                                                          \
    do {                                                                                            \
        const long long got_ = (long long)(call);                                                   \
        if (got_ != (long long)(want)) {                                                            \
            std::fprintf(stderr, "line %d: %s returned %lld, expected %lld\n", __LINE__, #call, got_, \
                         (long long)(want));                                                        \
            ++failures;                                                                             \
        }                                                                                           \
    } while (0)

static double offset_of(const void* p) { return (double)(static_cast<const char*>(p) - ws_begin); }

static void inside(const void* p, double bytes)
{
    if (offset_of(p) < 0 || offset_of(p) + bytes > (double)ws_bytes) {
        std::fprintf(stderr, "an array of %.0f bytes leaves the workspace\n", bytes);
        ++failures;
    }
}

namespace qb {

static hipError_t done() { ++launches; return hipSuccess; }
static int es(int dt) { return dt == 0 ? 4 : 2; }
static double dz_end = 0, weights_end = 0;
static bool rows_cheap = false;           // which of the two forms the estimates favour

static void bias_inside(const BiasSum& b)
{
    if (!b.db) ++failures;
    if (b.slices) inside(b.part, 4.0 * b.slices * (double)b.N);
}

hipError_t launch_linear_rows(int, const void*, int64_t M, int64_t K, const Weight4*, int, const Weight4Format&,
                              const Epilogue& e, hipStream_t)
{
    if ((!takes_rows(M, K) && (M > 1024 || !rows_cheap)) || !e.y) ++failures;
    return done();
}
double rows_us(int, int64_t, int64_t, int64_t, int) { return rows_cheap ? 1.0 : 1e30; }
double gemm_us(int, int64_t, int64_t, int64_t) { return 100.0; }
hipError_t launch_unpack(int xdt, const Weight4* w, int count, int64_t N, int64_t K, const Weight4Format&, void* out,
                         size_t each, hipStream_t)
{
    const double bytes = (double)N * (double)K * es(xdt);
    if (!w[0].codes || !w[count - 1].codes || bytes > (double)each) ++failures;
    inside(out, (count - 1) * (double)each + bytes);
    weights_end = offset_of(out) + (count - 1) * (double)each + bytes;
    return done();
}
static void transposed(int xdt, const TransposedWeights* t)
{
    if (!t) return;
    if (!t->w[0].codes || !t->w[t->count - 1].codes || t->np != gemm_pitch(xdt, t->N)) ++failures;
    const double bytes = (double)t->K * (double)t->np * t->count * es(xdt);
    inside(t->out, bytes);
    weights_end = offset_of(t->out) + bytes;
}
hipError_t launch_gemm(int xdt, bool gated, const GemmArgs& g, const Epilogue& e, float* part, const BiasSum* bias, hipStream_t)
{
    inside(part, 4.0 * (double)gemm_part_floats(g.M, g.R));
    if (offset_of(part) < weights_end || offset_of(part) < dz_end) ++failures;       // behind what it reads
    if (g.len < gemm_step(xdt) || g.lda * es(xdt) % 16 || g.ldb * es(xdt) % 16) ++failures;
    if (g.len0 != g.len && (g.len0 % gemm_step(xdt) || !g.a1)) ++failures;
    if (bias) bias_inside(*bias);
    if (gated && (!g.b1 || g.R != gated_rows(e.N))) ++failures;
    if (!gated && g.R != e.N) ++failures;
    dz_end = 0;
    return done();
}
hipError_t launch_linear_grad(int xdt, bool dz_too, const void*, const void*, int, int64_t M, int64_t N, void* dz,
                              int64_t pitch, void* dz_out, float* part, int slices, const TransposedWeights* t, hipStream_t)
{
    if (!dz_too && (dz || dz_out || part)) ++failures;
    transposed(xdt, t);
    if (dz) inside(dz, (double)M * (double)pitch * es(xdt));
    if (dz && t && offset_of(dz) < weights_end) ++failures;
    if (part) inside(part, 4.0 * slices * (double)N);
    dz_end = dz ? offset_of(dz) + (double)M * (double)pitch * es(xdt) : 0;
    if (part && (offset_of(part) < dz_end || (t && offset_of(part) < weights_end))) ++failures;
    return done();
}
hipError_t launch_few_rows_back(int xdt, const void* dz0, const void*, int64_t ldz, int64_t M, const TransposedWeights& t,
                                float* part, int* slices, hipStream_t)
{
    if (!dz0 || xdt == 0 || M > kRowsMax || ldz * 2 % 16 || !t.w[t.count - 1].codes) ++failures;
    *slices = (int)(gemm_part_floats(M, t.K) / (M * t.K));
    inside(part, 4.0 * *slices * (double)M * (double)t.K);
    if (*slices < 1 || offset_of(part) < dz_end) ++failures;
    return done();
}
hipError_t launch_join(int, const float* part, int pieces, int64_t M, const Epilogue& e, const BiasSum* bias, hipStream_t)
{
    if (bias) bias_inside(*bias);
    inside(part, 4.0 * pieces * (double)M * (double)e.N);
    return done();
}
hipError_t launch_bias_sum(const BiasSum& b, hipStream_t)
{
    bias_inside(b);
    return done();
}
hipError_t launch_gated_grad(int xdt, const void*, const void*, const void*, int, int64_t M, int64_t, void* dz,
                             int64_t pitch, void*, void*, const TransposedWeights* t, hipStream_t)
{
    transposed(xdt, t);
    if (dz) inside(dz, 2.0 * (double)M * (double)pitch * es(xdt));
    if (dz && t && offset_of(dz) < weights_end) ++failures;
    dz_end = dz ? offset_of(dz) + 2.0 * (double)M * (double)pitch * es(xdt) : 0;
    return done();
}
hipError_t launch_grad_squares(const NormTable& t, double* part, int* groups, float* norm, hipStream_t)
{
    if (t.count < 1 || t.count > kNormGrads || t.tiles < 1) ++failures;
    if (!norm) inside(part, 8.0 * kNormGroups);
    for (int i = 0; i < t.count; ++i) seen_elements += (long long)(t.size[i] >> 2);
    *groups = kNormGroups;
    return done();
}
hipError_t launch_grad_norm(const double* part, int count, float*, hipStream_t)
{
    if (count) inside(part, 8.0 * count);
    return done();
}
hipError_t launch_grad_scale(const ScaleTable& t, double, const float*, hipStream_t)
{
    if (t.count < 1 || t.count > kScaleGrads || t.tiles < 1) ++failures;
    for (int i = 0; i < t.count; ++i) seen_elements += (long long)(t.size[i] >> 2);
    return done();
}

}  // namespace qb

int main()
{
    char* const D = reinterpret_cast<char*>(uintptr_t(1) << 50);       // fake device addresses, never dereferenced
    void *const A = D, *const B = D + 4096, *const C = D + 8192, *const E = D + 12288;
    float* const F = reinterpret_cast<float*>(D + 16384);
    uint8_t* const U = reinterpret_cast<uint8_t*>(D + 32768);
    ws_begin = reinterpret_cast<char*>(uintptr_t(1) << 51);
    const qb_weight w{U, F, nullptr, nullptr, nullptr}, nested{U, nullptr, U, F, F};
    const int64_t widest = (int64_t(1) << 21) - 1, tall = (int64_t(1) << 31) - 1;

    for (qb_dtype dt : {QB_F32, QB_F16, QB_BF16, QB_F16, QB_F32})
        for (int64_t M : {int64_t(0), int64_t(1), int64_t(64), int64_t(65), int64_t(301), int64_t(4096), tall})
            for (int64_t K : {int64_t(32), int64_t(96), int64_t(4096), widest / 32 * 32})
                for (int64_t N : {int64_t(1), int64_t(64), int64_t(1001), int64_t(11008), widest}) {
                    qb::rows_cheap = !qb::rows_cheap;
                    const bool blocks = (N * K + 63) / 64 < int64_t(1) << 31;
                    const int ok = blocks ? QB_OK : QB_EINVAL;
                    ws_bytes = qb_dequant_linear_workspace_bytes(dt, M, K, N);
                    EXPECT(qb_dequant_linear(A, dt, M, K, U, F, nullptr, QB_NF4, 64, N, B, QB_F32, QB_ACT_GELU, C, E, C,
                                             ws_begin, ws_bytes, nullptr), ok);
                    ws_bytes = qb_dequant_gated_workspace_bytes(dt, M, K, N);
                    EXPECT(qb_dequant_gated(A, dt, M, K, &w, &w, QB_FP4, 64, 0, N, QB_ACT_SILU, B, C, E, ws_begin, ws_bytes,
                                            nullptr), ok);
                    ws_bytes = qb_dequant_linear_backward_workspace_bytes(dt, M, K, N);
                    for (int with = 0; with < 8; ++with)
                        for (qb_act act : {QB_ACT_NONE, QB_ACT_RELU})
                            EXPECT(qb_dequant_linear_backward(A, B, dt, M, K, U, F, nullptr, QB_NF4, 64, N, act,
                                                              with & 1 ? C : nullptr, with & 2 ? E : nullptr,
                                                              with & 4 ? F : nullptr, QB_F32, 0, ws_begin, ws_bytes,
                                                              nullptr), ok);
                    ws_bytes = qb_dequant_gated_backward_workspace_bytes(dt, M, K, N);
                    for (int with = 0; with < 8; ++with)
                        EXPECT(qb_dequant_gated_backward(A, B, C, dt, M, K, &nested, &nested, QB_NF4, 64, 256, N,
                                                         QB_ACT_SILU, with & 1 ? E : nullptr, with & 2 ? A : nullptr,
                                                         with & 4 ? B : nullptr, ws_begin, ws_bytes, nullptr), ok);
                }

    for (int count : {0, 1, 149, 150, 151, 223, 224, 225, 448, 449, 5000}) {
        std::vector<qb_grad> grads;
        long long total = 0;
        for (int i = 0; i < count; ++i) {
            const int64_t n = i % 7 == 3 ? 0 : i % 11 == 5 ? (int64_t(1) << 33) - 1 : 1 + i * 37;
            grads.push_back(qb_grad{D + 2 * i * 4, D + 4 * i, n, i % 3 == 0 ? QB_F32 : i % 3 == 1 ? QB_F16 : QB_BF16});
            total += n;
        }
        ws_bytes = qb_multi_tensor_grad_norm_workspace_bytes(count);
        seen_elements = 0;
        EXPECT(qb_multi_tensor_grad_norm(grads.data(), count, F, ws_begin, ws_bytes, nullptr), QB_OK);
        EXPECT(seen_elements, total);
        seen_elements = 0;
        EXPECT(qb_multi_tensor_clip_grads(grads.data(), count, 1.0, F, nullptr), QB_OK);
        EXPECT(seen_elements, total);
    }
    {
        // neighbours are one entry, up to the longest gradient there may be
        std::vector<qb_grad> grads;
        const int64_t n = int64_t(1) << 30;
        for (int64_t i = 0; i < 300; ++i) grads.push_back(qb_grad{D + 4 * n * i, D + 4 * n * i, n, QB_F32});
        const int start = launches;
        seen_elements = 0;
        ws_bytes = qb_multi_tensor_grad_norm_workspace_bytes(300);
        EXPECT(qb_multi_tensor_grad_norm(grads.data(), 300, F, ws_begin, ws_bytes, nullptr), QB_OK);
        EXPECT(qb_multi_tensor_clip_grads(grads.data(), 300, 1.0, F, nullptr), QB_OK);
        EXPECT(seen_elements, 600 * n);
        EXPECT(launches - start, 3);
    }
    const int before = launches;
    ws_bytes = qb_dequant_linear_workspace_bytes(QB_BF16, 100, 64, 64);
    EXPECT(qb_dequant_linear(A, QB_BF16, 100, 64, U, F, nullptr, QB_NF4, 64, 64, nullptr, QB_F32, QB_ACT_NONE, nullptr,
                             nullptr, B, ws_begin, ws_bytes - 1, nullptr), QB_EWORKSPACE);
    EXPECT(qb_dequant_linear(A, QB_BF16, 100, 48, U, F, nullptr, QB_NF4, 64, 64, nullptr, QB_F32, QB_ACT_NONE, nullptr,
                             nullptr, B, ws_begin, ws_bytes, nullptr), QB_EINVAL);
    EXPECT(qb_dequant_gated(A, QB_BF16, 10, 64, &w, &nested, QB_NF4, 64, 256, 64, QB_ACT_NONE, nullptr, nullptr, B, nullptr,
                            0, nullptr), QB_EUNSUPPORTED);
    EXPECT(qb_multi_tensor_clip_grads(nullptr, 0, std::nan(""), F, nullptr), QB_EINVAL);
    EXPECT(launches, before);
    if (failures == 0) std::printf("every call returned the expected status (%d launches)\n", launches);
    return failures == 0 ? 0 : 1;
}
