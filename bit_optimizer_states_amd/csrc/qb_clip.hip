// qb_clip.hip -- the global norm of many gradients, and clipping by it.
//
//   norm = sqrt(sum over gradients and elements of g^2),
//   out = g * min(1, max_norm / (norm + 1e-6)).
// Squares and sums are binary64: no square of a binary32 value leaves its range, and the
// order of the sums does not show in the norm's binary32 digits (it is fixed all the same:
// the same bits on every run).  Two passes over the gradients, bound by HBM; the second one
// walks them backwards, so that it begins with what the last-level cache still holds.
#include "qb_clip.h"
#include "qb_device.h"

namespace qb {

namespace {

// Gradients are often views of a bucket: they begin at any element.
typedef u32x4 __attribute__((aligned(2))) u32x4_e2;

constexpr int kAcc = 8;                  // accesses of a lane and tile

__device__ __forceinline__ float word_value(int dt, const u32x4& w, int j)
{
    if (dt == DT_F32) return ffrom(w[j & 3]);
    const uint32_t h = w[(j >> 1) & 3];
    if (dt == DT_BF16) return (j & 1) ? bf16_hi(h) : bf16_lo(h);
    return (j & 1) ? f16_hi(h) : f16_lo(h);
}

template <int DT>
__device__ __forceinline__ double squares(const u32x4 w)
{
    double s = 0.0;
#pragma unroll
    for (int j = 0; j < (DT == DT_F32 ? 4 : 8); ++j) {
        const double v = (double)word_value(DT, w, j);
        s = __builtin_fma(v, v, s);
    }
    return s;
}

// The sum of squares over this lane's share of a tile.
template <int DT>
__device__ __forceinline__ double tile_squares(const void* g, int64_t n, int64_t local)
{
    constexpr int E = DT == DT_F32 ? 4 : 8;
    const int lane = threadIdx.x & 63;
    const int64_t first = local * grad_tile_elems(DT), left = n - first;
    const char* const p = static_cast<const char*>(g) + first * (16 / E);
    double s = 0.0;
    if (left >= grad_tile_elems(DT)) {
        u32x4 w[kAcc];
#pragma unroll
        for (int i = 0; i < kAcc; ++i) w[i] = *(const QB_G u32x4_e2*)(p + (i * 64 + lane) * 16);
#pragma unroll
        for (int i = 0; i < kAcc; ++i) s += squares<DT>(w[i]);
    } else {
#pragma unroll
        for (int i = 0; i < kAcc; ++i) {
            const int64_t e = (i * 64 + lane) * E;
            if (e + E <= left) {
                s += squares<DT>(*(const QB_G u32x4_e2*)(p + (i * 64 + lane) * 16));
            } else {
                for (int j = 0; j < E; ++j)
                    if (e + j < left) {
                        const double v = (double)load1<DT>(p, e + j);
                        s = __builtin_fma(v, v, s);
                    }
            }
        }
    }
    return s;
}

template <int DT>
__device__ __forceinline__ u32x4 scaled(const u32x4 w, float scale)
{
    if constexpr (DT == DT_F32) {
        return u32x4{fbits(ffrom(w.x) * scale), fbits(ffrom(w.y) * scale), fbits(ffrom(w.z) * scale),
                     fbits(ffrom(w.w) * scale)};
    } else {
        u32x4 o;
#pragma unroll
        for (int j = 0; j < 4; ++j) o[j] = pack2<DT>(half_lo<DT>(w[j]) * scale, half_hi<DT>(w[j]) * scale);
        return o;
    }
}

template <int DT>
__device__ __forceinline__ void tile_scale(const void* g, void* out, int64_t n, int64_t local, float scale)
{
    constexpr int E = DT == DT_F32 ? 4 : 8;
    const int lane = threadIdx.x & 63;
    const int64_t first = local * grad_tile_elems(DT), left = n - first;
    const char* const p = static_cast<const char*>(g) + first * (16 / E);
    char* const q = static_cast<char*>(out) + first * (16 / E);
    if (left >= grad_tile_elems(DT)) {
        u32x4 w[kAcc];
#pragma unroll
        for (int i = 0; i < kAcc; ++i) w[i] = *(const QB_G u32x4_e2*)(p + (i * 64 + lane) * 16);
#pragma unroll
        for (int i = 0; i < kAcc; ++i) {
            const u32x4 o = scaled<DT>(w[i], scale);
            __builtin_nontemporal_store(o, (QB_G u32x4_e2*)(q + (i * 64 + lane) * 16));
        }
    } else {
#pragma unroll
        for (int i = 0; i < kAcc; ++i) {
            const int64_t e = (i * 64 + lane) * E;
            if (e + E <= left) {
                *(QB_G u32x4_e2*)(q + (i * 64 + lane) * 16) =
                    scaled<DT>(*(const QB_G u32x4_e2*)(p + (i * 64 + lane) * 16), scale);
            } else {
                for (int j = 0; j < E; ++j)
                    if (e + j < left) store1<DT>(q, e + j, load1<DT>(p, e + j) * scale);
            }
        }
    }
}

// Sum over a workgroup, in lane and wave order (valid in thread 0).
template <int NT>
__device__ __forceinline__ double group_sum64(double v)
{
    __shared__ double s_wave[NT / 64];
#pragma unroll
    for (int d = 1; d < 64; d *= 2) v += __shfl_xor(v, d);
    if ((threadIdx.x & 63) == 0) s_wave[threadIdx.x >> 6] = v;
    __syncthreads();
    double sum = 0.0;
    if (threadIdx.x == 0) {
#pragma unroll
        for (int w = 0; w < NT / 64; ++w) sum += s_wave[w];
    }
    return sum;
}

constexpr int kNormThreads = 512;

__global__ __launch_bounds__(kNormThreads) void k_grad_squares(const GradTable t, double* __restrict__ part,
                                                               float* __restrict__ norm)
{
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int total = t.tile_begin[t.count];
    double sum = 0.0;
    int i = 0;
    for (int tile = blockIdx.x * (kNormThreads / 64) + wave; tile < total; tile += gridDim.x * (kNormThreads / 64)) {
        while (tile >= t.tile_begin[i + 1]) ++i;         // (uniform; tiles ascend)
        const int64_t local = tile - t.tile_begin[i];
        const int dt = t.dt[i];
        sum += dt == DT_F32   ? tile_squares<DT_F32>(t.g[i], t.n[i], local)
               : dt == DT_F16 ? tile_squares<DT_F16>(t.g[i], t.n[i], local)
                              : tile_squares<DT_BF16>(t.g[i], t.n[i], local);
    }
    sum = group_sum64<kNormThreads>(sum);
    if (threadIdx.x == 0) {
        if (norm) norm[0] = (float)sqrt(sum);
        else part[blockIdx.x] = sum;
    }
}

__global__ __launch_bounds__(1024) void k_grad_norm(const double* __restrict__ part, int count, float* __restrict__ norm)
{
    double sum = 0.0;
    for (int i = threadIdx.x; i < count; i += 1024) sum += part[i];
    sum = group_sum64<1024>(sum);
    if (threadIdx.x == 0) norm[0] = (float)sqrt(sum);
}

__global__ __launch_bounds__(256) void k_grad_scale(const GradTable t, double max_norm, const float* __restrict__ norm)
{
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const double s = max_norm / ((double)norm[0] + 1e-6);
    const float scale = s >= 1.0 ? 1.0f : (float)s;      // (a NaN stays one)
    const int total = t.tile_begin[t.count];
    int i = 0;
    for (int tile = blockIdx.x * 4 + wave; tile < total; tile += gridDim.x * 4) {
        while (tile >= t.tile_begin[i + 1]) ++i;
        const void* const g = t.g[i];
        void* const out = t.out[i];
        if (scale == 1.0f && g == out) continue;         // nothing to change
        const int64_t local = t.tile_begin[i + 1] - 1 - tile;      // the gradient's tiles from its end
        const int dt = t.dt[i];
        if (dt == DT_F32) tile_scale<DT_F32>(g, out, t.n[i], local, scale);
        else if (dt == DT_F16) tile_scale<DT_F16>(g, out, t.n[i], local, scale);
        else tile_scale<DT_BF16>(g, out, t.n[i], local, scale);
    }
}

}  // namespace

hipError_t launch_grad_squares(const GradTable& t, double* part, int* groups, float* norm, hipStream_t s)
{
    const int total = t.tile_begin[t.count], per = kNormThreads / 64;
    const int grid = norm ? 1 : (total + per - 1) / per < kNormGroups ? (total + per - 1) / per : kNormGroups;
    if (groups) *groups = grid;
    return launch_kernel_nt(k_grad_squares, grid, kNormThreads, s, t, part, norm);
}

hipError_t launch_grad_norm(const double* part, int count, float* norm, hipStream_t s)
{
    return launch_kernel_nt(k_grad_norm, 1, 1024, s, part, count, norm);
}

hipError_t launch_grad_scale(const GradTable& t, double max_norm, const float* norm, hipStream_t s)
{
    const int total = t.tile_begin[t.count];
    const int grid = (total + 3) / 4 < 2048 ? (total + 3) / 4 : 2048;
    return launch_kernel(k_grad_scale, grid, s, t, max_norm, norm);
}

}  // namespace qb
