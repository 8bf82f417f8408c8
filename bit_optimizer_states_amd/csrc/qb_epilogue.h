// qb_epilogue.h -- what becomes of a 4-bit layer's sums (struct Epilogue): bias,
// activation and residual, or activation and product, in binary32, each output
// rounded once.
#pragma once
#include "qb_act.h"
#include "qb_linear.h"
#include "qb_mm_device.h"

namespace qb {

// Rows of C begin at any element (N may be odd): accesses of four elements through types
// of element alignment, which the GLOBAL instructions take as they are.
typedef u32x2 __attribute__((aligned(2))) u32x2_e2;
typedef u32x4 __attribute__((aligned(2))) u32x4_e2;
typedef f32x4 __attribute__((aligned(4))) f32x4_e4;

// Up to four elements from element i on (cnt of them).
template <int DT>
__device__ __forceinline__ f32x4 load_up_to4(const void* p, int64_t i, int cnt)
{
    f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
    if (cnt >= 4) {
        if constexpr (DT == DT_F32) {
            v = *(const QB_G f32x4_e4*)(static_cast<const float*>(p) + i);
        } else {
            const u32x2 w = *(const QB_G u32x2_e2*)(static_cast<const uint16_t*>(p) + i);
            v = f32x4{half_lo<DT>(w.x), half_hi<DT>(w.x), half_lo<DT>(w.y), half_hi<DT>(w.y)};
        }
    } else {
#pragma unroll
        for (int j = 0; j < 3; ++j)
            if (j < cnt) v[j] = load1<DT>(p, i + j);
    }
    return v;
}

template <int DT>
__device__ __forceinline__ void store_up_to4(void* p, int64_t i, int cnt, const f32x4& v)
{
    if (cnt >= 4) {
        if constexpr (DT == DT_F32) *(QB_G f32x4_e4*)(static_cast<float*>(p) + i) = v;
        else *(QB_G u32x2_e2*)(static_cast<uint16_t*>(p) + i) = u32x2{pack_two<DT>(v.x, v.y), pack_two<DT>(v.z, v.w)};
    } else {
#pragma unroll
        for (int j = 0; j < 3; ++j)
            if (j < cnt) store1<DT>(p, i + j, v[j]);
    }
}

__device__ __forceinline__ f32x4 load_bias4(const Epilogue& e, int64_t n, int cnt)
{
    return e.bias_dt == DT_F32   ? load_up_to4<DT_F32>(e.bias, n, cnt)
           : e.bias_dt == DT_F16 ? load_up_to4<DT_F16>(e.bias, n, cnt)
                                 : load_up_to4<DT_BF16>(e.bias, n, cnt);
}

__device__ __forceinline__ int columns_left(int64_t n, int64_t N)
{
    return N - n >= 4 ? 4 : N > n ? (int)(N - n) : 0;
}

// Four neighbouring columns n .. n + 3 of row m (those below N).
template <int XDT>
__device__ __forceinline__ void finish_linear4(const Epilogue& e, int64_t m, int64_t n, f32x4 z)
{
    const int cnt = columns_left(n, e.N);
    if (cnt == 0) return;
    const int64_t at = m * e.N + n;
    if (e.bias) z += load_bias4(e, n, cnt);
    if (e.z) store_up_to4<XDT>(e.z, at, cnt, z);
    float a[4] = {z.x, z.y, z.z, z.w};
    act_values<4>(e.act, a);
    f32x4 y = {a[0], a[1], a[2], a[3]};
    if (e.residual) y += load_up_to4<XDT>(e.residual, at, cnt);
    store_up_to4<XDT>(e.y, at, cnt, y);
}

// Eight neighbouring columns (cnt of them below N), the bias and the residual read before.
template <int DT>
__device__ __forceinline__ void load_up_to8(const void* p, int64_t i, int cnt, float* v)
{
    if (cnt >= 8) {
        if constexpr (DT == DT_F32) {
            *reinterpret_cast<f32x4*>(v) = load_up_to4<DT>(p, i, 4);
            *reinterpret_cast<f32x4*>(v + 4) = load_up_to4<DT>(p, i + 4, 4);
        } else {
            const u32x4 w = *(const QB_G u32x4_e2*)(static_cast<const uint16_t*>(p) + i);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v[2 * j] = half_lo<DT>(w[j]);
                v[2 * j + 1] = half_hi<DT>(w[j]);
            }
        }
    } else {
#pragma unroll
        for (int j = 0; j < 7; ++j)
            if (j < cnt) v[j] = load1<DT>(p, i + j);
    }
}

template <int DT>
__device__ __forceinline__ void store_up_to8(void* p, int64_t i, int cnt, const float* v)
{
    if (cnt >= 8) {
        if constexpr (DT == DT_F32) {
            store_up_to4<DT>(p, i, 4, f32x4{v[0], v[1], v[2], v[3]});
            store_up_to4<DT>(p, i + 4, 4, f32x4{v[4], v[5], v[6], v[7]});
        } else {
            *(QB_G u32x4_e2*)(static_cast<uint16_t*>(p) + i) =
                u32x4{pack_two<DT>(v[0], v[1]), pack_two<DT>(v[2], v[3]), pack_two<DT>(v[4], v[5]),
                      pack_two<DT>(v[6], v[7])};
        }
    } else {
#pragma unroll
        for (int j = 0; j < 7; ++j)
            if (j < cnt) store1<DT>(p, i + j, v[j]);
    }
}

__device__ __forceinline__ int columns_left8(int64_t n, int64_t N) { return N - n >= 8 ? 8 : N > n ? (int)(N - n) : 0; }

__device__ __forceinline__ void load_bias8(const Epilogue& e, int64_t n, int cnt, float* v)
{
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = 0.0f;
    if (!e.bias) return;
    if (e.bias_dt == DT_F32) load_up_to8<DT_F32>(e.bias, n, cnt, v);
    else if (e.bias_dt == DT_F16) load_up_to8<DT_F16>(e.bias, n, cnt, v);
    else load_up_to8<DT_BF16>(e.bias, n, cnt, v);
}

template <int XDT>
__device__ __forceinline__ void finish_linear8(const Epilogue& e, int64_t m, int64_t n, int cnt, float* z,
                                               const float* bias, const float* residual)
{
    const int64_t at = m * e.N + n;
    if (e.bias) {
#pragma unroll
        for (int j = 0; j < 8; ++j) z[j] += bias[j];
    }
    if (e.z) store_up_to8<XDT>(e.z, at, cnt, z);
    act_values<8>(e.act, z);
    if (e.residual) {
#pragma unroll
        for (int j = 0; j < 8; ++j) z[j] += residual[j];
    }
    store_up_to8<XDT>(e.y, at, cnt, z);
}

template <int XDT>
__device__ __forceinline__ void finish_gated8(const Epilogue& e, int64_t m, int64_t n, int cnt, float* g,
                                              const float* u)
{
    const int64_t at = m * e.N + n;
    if (e.z) store_up_to8<XDT>(e.z, at, cnt, g);
    if (e.u) store_up_to8<XDT>(e.u, at, cnt, u);
    act_values<8>(e.act, g);
#pragma unroll
    for (int j = 0; j < 8; ++j) g[j] *= u[j];
    store_up_to8<XDT>(e.y, at, cnt, g);
}

template <int XDT>
__device__ __forceinline__ void finish_gated4(const Epilogue& e, int64_t m, int64_t n, const f32x4& g, const f32x4& u)
{
    const int cnt = columns_left(n, e.N);
    if (cnt == 0) return;
    const int64_t at = m * e.N + n;
    if (e.z) store_up_to4<XDT>(e.z, at, cnt, g);
    if (e.u) store_up_to4<XDT>(e.u, at, cnt, u);
    float a[4] = {g.x, g.y, g.z, g.w};
    act_values<4>(e.act, a);
    store_up_to4<XDT>(e.y, at, cnt, f32x4{a[0] * u.x, a[1] * u.y, a[2] * u.z, a[3] * u.w});
}

}  // namespace qb
