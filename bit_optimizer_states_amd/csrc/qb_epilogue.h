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
        else *(QB_G u32x2_e2*)(static_cast<uint16_t*>(p) + i) = u32x2{pack_pair<DT>(v.x, v.y), pack_pair<DT>(v.z, v.w)};
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
    f32x4 y = z;
    if (e.act != ACT_NONE) {
#pragma unroll
        for (int j = 0; j < 4; ++j) y[j] = act_value(e.act, z[j]);
    }
    if (e.residual) y += load_up_to4<XDT>(e.residual, at, cnt);
    store_up_to4<XDT>(e.y, at, cnt, y);
}

template <int XDT>
__device__ __forceinline__ void finish_gated4(const Epilogue& e, int64_t m, int64_t n, const f32x4& g, const f32x4& u)
{
    const int cnt = columns_left(n, e.N);
    if (cnt == 0) return;
    const int64_t at = m * e.N + n;
    if (e.z) store_up_to4<XDT>(e.z, at, cnt, g);
    if (e.u) store_up_to4<XDT>(e.u, at, cnt, u);
    f32x4 y;
#pragma unroll
    for (int j = 0; j < 4; ++j) y[j] = act_value(e.act, g[j]) * u[j];
    store_up_to4<XDT>(e.y, at, cnt, y);
}

}  // namespace qb
