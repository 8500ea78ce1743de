// activation.cuh -- the activations of the feed-forward operators and their
// derivatives, in FP32.
//
//   none      a(z) = z
//   relu      a(z) = max(z, 0)                       a'(z) = [z > 0]
//   gelu      a(z) = z Phi(z)                        a'(z) = Phi(z) + z phi(z)
//   gelu_tanh a(z) = z s(2v), v = c (z + k z^3)      a'(z) = s + z s (1 - s) 2c (1 + 3k z^2)
//   silu      a(z) = z s(z)                          a'(z) = s + z s (1 - s)
// with Phi and phi the standard normal's distribution and density, s the
// logistic function, c = sqrt(2/pi), k = 0.044715 (0.5 (1 + tanh v) = s(2v)).
//
// e = exp(-x) = 2^(-x log2 e) is cut at 2^127, so that s = 1 / (1 + e) and
// 1 - s = e s need no case for the sign, do not cancel and stay finite (at
// 2^127 the reciprocal is flushed to s = 0, and every use of 1 - s there is
// times z s): a finite z of any size gives a finite value and derivative.
// The exponential and the reciprocal are the special-function unit's own (2
// units in the last place each), one instruction apiece; their error is below
// the products'.  Largest errors over 2 million z in each of seven ranges up to
// |z| = 30, as multiples of 2^-24 |z| for the value and of 2^-24 for the
// derivative: gelu 5.6 and 5.6 (near z = 0; beyond 2 at most 2.7 and 3.0),
// gelu_tanh 2.8 and 3.8, silu 2.8 and 3.6.  gelu's mean error is -0.9e-7 for 2 <
// |z| < 4 (largest 2.1e-7 below zero, where a form with erff has 1.2e-7 and mean
// 0.01e-7).  What an activation costs a product's epilogue, whose eight
// warps have little else to overlap with (M = 6144, K = 256, N = 1024, plain
// product 27.6 us): relu 27.1, gelu 29.0, gelu_tanh 28.9, silu 28.9 us; with
// expf, erff and a division behind them gelu took 42.6 and silu 34.0.
//
// The kernels choose among three forms of code (Family) once per tile, not per
// value: gelu_tanh and silu are both z s(w) with w = z (c0 + c1 z^2).
#pragma once

#include <cuda_runtime.h>

namespace emu {

enum Act : int { ACT_NONE = 0, ACT_RELU = 1, ACT_GELU = 2, ACT_GELU_TANH = 3, ACT_SILU = 4 };
enum Family : int { FAMILY_LINEAR = 0, FAMILY_ERF = 1, FAMILY_LOGISTIC = 2 };

// An activation as the kernels take it.
struct ActParams {
    int family;
    int relu;      // FAMILY_LINEAR: negative values to zero
    float c0, c1;  // FAMILY_LOGISTIC
};
inline ActParams act_params(int act) {
    constexpr float kTwoSqrt2OverPi = 1.5957691216057308f, kCubic = 0.044715f;
    switch (act) {
        case ACT_RELU: return {FAMILY_LINEAR, 1, 0.f, 0.f};
        case ACT_GELU: return {FAMILY_ERF, 0, 0.f, 0.f};
        case ACT_GELU_TANH: return {FAMILY_LOGISTIC, 0, kTwoSqrt2OverPi, kTwoSqrt2OverPi * kCubic};
        case ACT_SILU: return {FAMILY_LOGISTIC, 0, 1.f, 0.f};
        default: return {FAMILY_LINEAR, 0, 0.f, 0.f};
    }
}

constexpr float kLog2e = 1.4426950408889634f;
__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcp_approx(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// s(x) and 1 - s(x)
__device__ __forceinline__ void logistic(float x, float& s, float& c) {
    const float e = exp2_approx(fminf(-kLog2e * x, 127.0f));
    s = rcp_approx(1.0f + e);
    c = e * s;
}

// Phi(z) and exp(-z^2 / 2).  The upper tail 1 - Phi(|z|) = erfc(|z| / sqrt 2) / 2
// by the rational approximation 7.1.26 of Abramowitz and Stegun, Handbook of
// Mathematical Functions (erf to 1.5e-7 everywhere, so Phi to 0.75e-7, just
// above half a unit in the last place of 1), whose exponential is the one the
// derivative needs.
__device__ __forceinline__ void normal_cdf(float z, float& cdf, float& e) {
    e = exp2_approx(-0.5f * kLog2e * z * z);
    const float t = rcp_approx(fmaf(0.3275911f * 0.7071067811865476f, fabsf(z), 1.0f));
    float q = fmaf(t, 0.5f * 1.061405429f, 0.5f * -1.453152027f);
    q = fmaf(t, q, 0.5f * 1.421413741f);
    q = fmaf(t, q, 0.5f * -0.284496736f);
    q = fmaf(t, q, 0.5f * 0.254829592f);
    q *= t * e;
    cdf = z >= 0.0f ? 1.0f - q : q;
}

// a = a(z), d = a'(z) (whichever is not used is not computed)
template <int FAMILY>
__device__ __forceinline__ void act_value_grad(const ActParams& p, float z, float& a, float& d) {
    if constexpr (FAMILY == FAMILY_LINEAR) {
        a = p.relu && z < 0.0f ? 0.0f : z;  // (a NaN stays one)
        d = p.relu && !(z > 0.0f) ? 0.0f : 1.0f;
    } else if constexpr (FAMILY == FAMILY_ERF) {
        float s, e;
        normal_cdf(z, s, e);
        a = z * s;
        d = fmaf(z * 0.3989422804014327f, e, s);
    } else {
        // beyond |z| = 16 one of s and 1 - s is zero in either function, so
        // z^2 is cut there: w and its derivative stay finite
        const float z2 = fminf(z * z, 256.0f);
        float s, c;
        logistic(z * fmaf(p.c1, z2, p.c0), s, c);
        a = z * s;
        d = fmaf(a * c, fmaf(3.0f * p.c1, z2, p.c0), s);
    }
}
template <int FAMILY>
__device__ __forceinline__ void act_value_grad4(const ActParams& p, const float4& z, float4& a, float4& d) {
    act_value_grad<FAMILY>(p, z.x, a.x, d.x);
    act_value_grad<FAMILY>(p, z.y, a.y, d.y);
    act_value_grad<FAMILY>(p, z.z, a.z, d.z);
    act_value_grad<FAMILY>(p, z.w, a.w, d.w);
}

// f(integral constant of the family)
template <int V> struct ValueIs { static constexpr int value = V; };
template <class F> __host__ __device__ __forceinline__ void for_family(int family, F f) {
    if (family == FAMILY_LOGISTIC) f(ValueIs<FAMILY_LOGISTIC>{});
    else if (family == FAMILY_ERF) f(ValueIs<FAMILY_ERF>{});
    else f(ValueIs<FAMILY_LINEAR>{});
}

}  // namespace emu
