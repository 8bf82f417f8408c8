// qb_act.h -- activations of the 4-bit layers and their derivatives, in binary32.
//
//   none x;  relu max(x, 0);  silu x s(x), s(x) = 1 / (1 + e^-x);
//   gelu x P(x), P(x) = erfc(-x / sqrt 2) / 2 (the normal distribution);
//   gelu_tanh x (1 + tanh(sqrt(2 / pi) (x + 0.044715 x^3))) / 2 = x s(q(x)), q twice the
//   argument of tanh.
// Their derivatives, with s' = s(x) s(-x) and p the normal density:
//   silu s + x s',  gelu P + x p,  gelu_tanh s(q) + x s'(q) q'.
// 1 - s(x) is taken as s(-x), which keeps its digits where s(x) is near 1.
// At the infinities both are their limits (a 16-bit pre-activation may have become one): the factor
// of a probability is held above -infinity, whose product with a probability of 0 would be NaN.
// At NaN both are NaN.
#pragma once
#include "qb_device.h"

namespace qb {

enum Act { ACT_NONE = 0, ACT_RELU = 1, ACT_GELU = 2, ACT_GELU_TANH = 3, ACT_SILU = 4 };

// e^x as 2^(x log2 e) by the hardware's exponential, the product's rounding and log2 e's
// carried along: a rounded product alone is off by up to |x| 2^-24 in the result's
// relative error.  Beyond binary32's range 0 and infinity.
__device__ __forceinline__ float exp_f32(float x)
{
    constexpr float kL = 1.44269502f, kLow = 1.92596299e-8f, kLn2 = 0.693147182f;    // log2 e in two parts, ln 2
    const float c = x < -150.0f ? -150.0f : x > 150.0f ? 150.0f : x;                 // (a NaN stays one)
    const float t = c * kL;
    const float e = __builtin_fmaf(c, kLow, __builtin_fmaf(c, kL, -t));
    const float p = __builtin_amdgcn_exp2f(t);
    return p == __builtin_inff() ? p : __builtin_fmaf(p, e * kLn2, p);
}

__device__ __forceinline__ float sigmoid_f32(float x) { return __builtin_amdgcn_rcpf(1.0f + exp_f32(-x)); }

// x, -infinity as the lowest number.
__device__ __forceinline__ float above_minus_infinity(float x) { return __builtin_fmaxf(x, -__FLT_MAX__); }

constexpr float kGeluA = 1.59576917f, kGeluB = 0.044715f;      // 2 sqrt(2 / pi)

__device__ __forceinline__ float act_value(int act, float x)
{
    switch (act) {
    case ACT_RELU: return x < 0.0f ? 0.0f : x;
    case ACT_GELU: return 0.5f * above_minus_infinity(x) * erfcf(x * -0.707106769f);
    case ACT_GELU_TANH:
        return above_minus_infinity(x) * sigmoid_f32(kGeluA * __builtin_fmaf(kGeluB * x * x, x, x));
    case ACT_SILU: return above_minus_infinity(x) * sigmoid_f32(x);
    default: return x;
    }
}

// act of each of N values, the kind told apart once.
template <int N>
__device__ __forceinline__ void act_values(int act, float* v)
{
    switch (act) {
    case ACT_RELU:
#pragma unroll
        for (int j = 0; j < N; ++j) v[j] = act_value(ACT_RELU, v[j]);
        return;
    case ACT_GELU:
#pragma unroll
        for (int j = 0; j < N; ++j) v[j] = act_value(ACT_GELU, v[j]);
        return;
    case ACT_GELU_TANH:
#pragma unroll
        for (int j = 0; j < N; ++j) v[j] = act_value(ACT_GELU_TANH, v[j]);
        return;
    case ACT_SILU:
#pragma unroll
        for (int j = 0; j < N; ++j) v[j] = act_value(ACT_SILU, v[j]);
        return;
    default: return;
    }
}

// a s(q) s(-q), zero where that product is (a may be infinite there).
__device__ __forceinline__ float times_slope(float a, float s, float s_neg)
{
    const float d = s * s_neg;
    return d == 0.0f ? 0.0f : a * d;
}

// act(x) and act'(x).
__device__ __forceinline__ void act_both(int act, float x, float& value, float& slope)
{
    switch (act) {
    case ACT_RELU:
        value = x < 0.0f ? 0.0f : x;
        slope = x > 0.0f ? 1.0f : x == x ? 0.0f : x;
        return;
    case ACT_GELU: {
        const float cdf = 0.5f * erfcf(x * -0.707106769f), p = 0.398942292f * exp_f32(-0.5f * x * x);
        value = above_minus_infinity(x) * cdf;
        slope = p == 0.0f ? cdf : __builtin_fmaf(x, p, cdf);
        return;
    }
    case ACT_GELU_TANH: {
        const float q = kGeluA * __builtin_fmaf(kGeluB * x * x, x, x);
        const float s = sigmoid_f32(q), dq = kGeluA * __builtin_fmaf(3.0f * kGeluB * x, x, 1.0f);
        value = above_minus_infinity(x) * s;
        slope = s + times_slope(x * dq, s, sigmoid_f32(-q));
        return;
    }
    case ACT_SILU: {
        const float s = sigmoid_f32(x);
        value = above_minus_infinity(x) * s;
        slope = s + times_slope(x, s, sigmoid_f32(-x));
        return;
    }
    default:
        value = x;
        slope = 1.0f;
        return;
    }
}

// a[j] *= act'(z[j]), b[j] *= act(z[j]) (act known at compile time).
template <int ACT, int N>
__device__ __forceinline__ void times_act_of(const float* z, float* a, float* b)
{
#pragma unroll
    for (int j = 0; j < N; ++j) {
        float value, slope;
        act_both(ACT, z[j], value, slope);
        a[j] *= slope;
        if (b) b[j] *= value;
    }
}

template <int N>
__device__ __forceinline__ void times_act_both(int act, const float* z, float* a, float* b)
{
    switch (act) {
    case ACT_RELU: return times_act_of<ACT_RELU, N>(z, a, b);
    case ACT_GELU: return times_act_of<ACT_GELU, N>(z, a, b);
    case ACT_GELU_TANH: return times_act_of<ACT_GELU_TANH, N>(z, a, b);
    case ACT_SILU: return times_act_of<ACT_SILU, N>(z, a, b);
    default: return times_act_of<ACT_NONE, N>(z, a, b);
    }
}

template <int N>
__device__ __forceinline__ void times_act_slopes(int act, const float* z, float* d)
{
    times_act_both<N>(act, z, d, nullptr);
}

}  // namespace qb
