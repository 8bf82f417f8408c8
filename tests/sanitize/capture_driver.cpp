// Driver for the host code of the calls that upload a table (qb_api.cpp; test infrastructure): the HIP runtime
// and the launchers below stand in for the real ones, device memory is host memory.  On an ordinary stream a
// call makes one copy from host memory.  On a stream under capture it makes none, since a graph would replay
// the address: the same bytes are handed over by value.  Exits non-zero on the first difference.
#include <hip/hip_runtime.h>

#include <cstdio>
#include <cstring>
#include <vector>

#include "qb.h"
#include "qb_launch.h"

static int copies = 0, values = 0, failures = 0;
static bool capturing = false;

#define CHECK(x)                                                             \
    do {                                                                     \
        if (!(x)) {                                                          \
            std::fprintf(stderr, "line %d: %s does not hold\n", __LINE__, #x); \
            ++failures;                                                      \
        }                                                                    \
    } while (0)

extern "C" {
hipError_t hipMemcpyAsync(void* to, const void* from, size_t bytes, hipMemcpyKind, hipStream_t)
{
    ++copies;
    std::memcpy(to, from, bytes);
    return hipSuccess;
}
hipError_t hipStreamIsCapturing(hipStream_t s, hipStreamCaptureStatus* status)
{
    if (!s) return hipErrorInvalidValue;
    *status = capturing ? hipStreamCaptureStatusActive : hipStreamCaptureStatusNone;
    return hipSuccess;
}
hipError_t hipGetDevice(int* device) { *device = 0; return hipSuccess; }
hipError_t hipGetLastError(void) { return hipSuccess; }
hipError_t hipEventCreateWithFlags(hipEvent_t*, unsigned) { return hipErrorInvalidValue; }
hipError_t hipEventRecord(hipEvent_t, hipStream_t) { return hipErrorInvalidValue; }
hipError_t hipStreamCreateWithFlags(hipStream_t*, unsigned) { return hipErrorInvalidValue; }
hipError_t hipStreamWaitEvent(hipStream_t, hipEvent_t, unsigned) { return hipErrorInvalidValue; }
hipError_t hipPointerGetAttributes(hipPointerAttribute_t*, const void*) { return hipErrorInvalidValue; }
}

namespace qb {

alignas(256) static unsigned char scratch[kScratchBytes];

const QbTables* device_tables() { return host_tables(); }
void* device_scratch() { return scratch; }
int64_t adamw_tiles(int64_t n, int) { return (n + 1023) / 1024; }

hipError_t launch_clear_bins(unsigned long long*, int, hipStream_t) { return hipSuccess; }
hipError_t launch_quant(const QuantDesc&, const TileMap<QuantDesc>*, int64_t, int, int, int, int, bool,
                        unsigned long long*, hipStream_t) { return hipSuccess; }
hipError_t launch_quant_user(const QuantDesc&, int64_t, int, int, const UserCode*, hipStream_t) { return hipSuccess; }
hipError_t launch_dequant_user(const DequantDesc&, int64_t, int, int, const UserCode*, hipStream_t) { return hipSuccess; }
hipError_t launch_normalize(const void*, int, int64_t, const float*, int64_t, float*, hipStream_t) { return hipSuccess; }
hipError_t launch_chunk_quantiles(const void*, int, int64_t, float*, hipStream_t) { return hipSuccess; }
hipError_t launch_quantile_code(const float*, int64_t, double*, double*, UserCode*, hipStream_t) { return hipSuccess; }
hipError_t launch_dq4_matmul(const void*, int, int64_t, int64_t, const uint8_t*, const float*, const uint8_t*,
                             const float*, const float*, int, int, int, int64_t, void*, hipStream_t) { return hipSuccess; }
hipError_t launch_dq4_matmul_grouped(const void*, int, int64_t, int64_t, const MmWeight*, int, int, int, int,
                                     hipStream_t) { return hipSuccess; }
hipError_t launch_dq_mean(const QuantDesc&, const TileMap<QuantDesc>*, int, const unsigned long long*, hipStream_t)
{
    return hipSuccess;
}
hipError_t launch_dequant(const DequantDesc&, const TileMap<DequantDesc>*, int64_t, int, int, int, int, bool, int,
                          hipStream_t) { return hipSuccess; }
hipError_t launch_optim8(int, const TensorDesc&, const TileMap<TensorDesc>*, int64_t, int, int, int, const OptScalars&,
                         const float*, bool, hipStream_t) { return hipSuccess; }
hipError_t launch_trust_norms(int, const TileMap<TensorDesc>&, int64_t, int, int, int, const OptScalars&, double*, bool,
                              hipStream_t) { return hipSuccess; }
hipError_t launch_trust_scalars(int, const TileMap<TensorDesc>&, const double*, double, double, double, float*,
                                hipStream_t) { return hipSuccess; }

}  // namespace qb

static hipError_t by_value(void* to, const void* from, size_t bytes, hipStream_t)
{
    ++values;
    CHECK(bytes > 0 && bytes % 4 == 0);
    std::memcpy(to, from, bytes);
    return hipSuccess;
}

// `call(stream)` writes its table to `to`: the same bytes on an ordinary stream and on one under capture.
template <class F>
static void both(void* to, size_t bytes, F call)
{
    hipStream_t const s = reinterpret_cast<hipStream_t>(uintptr_t(1) << 40);
    std::vector<unsigned char> want(bytes);
    for (hipStream_t ordinary : {s, hipStream_t(nullptr)}) {
        std::memset(to, 0xAB, bytes);
        copies = values = 0;
        CHECK(call(ordinary) == QB_OK);
        CHECK(copies == 1 && values == 0);
        std::memcpy(want.data(), to, bytes);
    }
    std::memset(to, 0xAB, bytes);
    copies = values = 0;
    capturing = true;
    CHECK(call(s) == QB_OK);
    capturing = false;
    CHECK(copies == 0 && values == 1);
    CHECK(std::memcmp(want.data(), to, bytes) == 0);
}

int main()
{
    qb::store_by_value = &by_value;
    char* const D = reinterpret_cast<char*>(uintptr_t(1) << 50);       // fake device addresses, never dereferenced
    uint8_t* const U = reinterpret_cast<uint8_t*>(D);
    float* const F = reinterpret_cast<float*>(D + 4096);
    for (int count : {1, 3, 500}) {
        std::vector<qb_tensor> t;
        std::vector<qb_quant_tensor> q, nested;
        std::vector<qb_dequant_tensor> d;
        for (int i = 0; i < count; ++i) {
            const int64_t n = 100 + 777 * i;
            t.push_back(qb_tensor{F, D + 8192, U, U, F, F, n});
            q.push_back(qb_quant_tensor{D, U, F, nullptr, nullptr, nullptr, n});
            nested.push_back(qb_quant_tensor{D, U, nullptr, U, F, F, n});
            d.push_back(qb_dequant_tensor{U, F, nullptr, nullptr, nullptr, D, n});
        }
        for (qb_optimizer kind : {QB_ADAMW, QB_LAMB}) {
            qb_optim_hparams hp{};
            hp.kind = kind;
            hp.lr = 1e-3;
            hp.beta1 = 0.9;
            hp.beta2 = 0.99;
            hp.eps = 1e-8;
            hp.step = 1;
            std::vector<double> ws(qb_optimizer_workspace_bytes(&hp, t.data(), count, 256) / 8 + 2);
            void* const w = reinterpret_cast<void*>((reinterpret_cast<uintptr_t>(ws.data()) + 15) / 16 * 16);
            const size_t bytes = qb_optimizer_workspace_bytes(&hp, t.data(), count, 256);
            both(w, bytes, [&](hipStream_t s) {
                return qb_multi_tensor_optimizer_step(&hp, t.data(), count, QB_F32, QB_BF16, 256, w, bytes, s);
            });
        }
        const qb_adamw_hparams a{1e-3, 0.9, 0.99, 1e-8, 0.0, 1};
        both(qb::scratch, sizeof(qb::scratch), [&](hipStream_t s) {
            return qb_multi_tensor_step_noalloc(t.data(), count, QB_F32, 256, &a, s);
        });
        for (auto* table : {&q, &nested}) {
            const size_t bytes = qb_multi_tensor_quantize_workspace_bytes(table->data(), count, 64);
            std::vector<double> ws(bytes / 8 + 2);
            void* const w = reinterpret_cast<void*>((reinterpret_cast<uintptr_t>(ws.data()) + 15) / 16 * 16);
            both(w, bytes, [&](hipStream_t s) {
                return qb_multi_tensor_quantize(table->data(), count, QB_F32, QB_NF4, 64, 256, w, bytes, s);
            });
        }
        const size_t bytes = qb_multi_tensor_workspace_bytes(count);
        std::vector<double> ws(bytes / 8 + 2);
        void* const w = reinterpret_cast<void*>((reinterpret_cast<uintptr_t>(ws.data()) + 15) / 16 * 16);
        both(w, bytes, [&](hipStream_t s) {
            return qb_multi_tensor_dequantize(d.data(), count, QB_NF4, 64, 256, QB_BF16, w, bytes, s);
        });
    }
    float code[256];
    for (int i = 0; i < 256; ++i) code[i] = (float)(i - 128) / 128.0f;
    alignas(16) static unsigned char table[sizeof(qb::UserCode)];
    both(table, sizeof(table), [&](hipStream_t s) { return qb_prepare_code(code, table, s); });
    // without the device code a captured call is an error, not a copy
    qb::store_by_value = nullptr;
    capturing = true;
    copies = 0;
    CHECK(qb_prepare_code(code, table, reinterpret_cast<hipStream_t>(uintptr_t(1) << 40)) == QB_EHIP && copies == 0);
    if (failures == 0) std::printf("captured calls carry their tables\n");
    return failures == 0 ? 0 : 1;
}
