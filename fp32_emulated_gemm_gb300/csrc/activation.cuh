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
// s(x) and 1 - s(x) both come from e = exp(-|x|) and 1 / (1 + e): no
// cancellation for either sign and no overflow, so a finite z of any size
// gives a finite value and derivative.  __expf and __fdividef keep the cost
// at two special-function instructions per value; their error (a few units
// in the last place of e, which is at most 1) is below the products' own.
#pragma once

#include <cuda_runtime.h>

namespace emu {

enum Act : int { ACT_NONE = 0, ACT_RELU = 1, ACT_GELU = 2, ACT_GELU_TANH = 3, ACT_SILU = 4 };

constexpr float kSqrt2OverPi = 0.7978845608028654f;
constexpr float kGeluCubic = 0.044715f;
constexpr float kSqrtHalf = 0.7071067811865476f;
constexpr float kInvSqrt2Pi = 0.3989422804014327f;

// s(x) and 1 - s(x)
__device__ __forceinline__ void logistic(float x, float& s, float& c) {
    const float e = __expf(-fabsf(x));
    const float big = __fdividef(1.0f, 1.0f + e), small = e * big;
    s = x >= 0.0f ? big : small;
    c = x >= 0.0f ? small : big;
}

__device__ __forceinline__ float act_value(int act, float z) {
    float s, c;
    switch (act) {
        case ACT_RELU: return z < 0.0f ? 0.0f : z;  // (a NaN stays one)
        case ACT_GELU: return 0.5f * z * (1.0f + erff(z * kSqrtHalf));
        case ACT_GELU_TANH:
            logistic(2.0f * kSqrt2OverPi * fmaf(kGeluCubic * z * z, z, z), s, c);
            return z * s;
        case ACT_SILU:
            logistic(z, s, c);
            return z * s;
        default: return z;
    }
}

// a = a(z), d = a'(z)
__device__ __forceinline__ void act_value_grad(int act, float z, float& a, float& d) {
    float s, c;
    switch (act) {
        case ACT_RELU:
            a = z < 0.0f ? 0.0f : z;
            d = z > 0.0f ? 1.0f : 0.0f;
            break;
        case ACT_GELU:
            s = 0.5f * (1.0f + erff(z * kSqrtHalf));
            a = z * s;
            d = fmaf(z * kInvSqrt2Pi, __expf(-0.5f * z * z), s);
            break;
        case ACT_GELU_TANH: {
            logistic(2.0f * kSqrt2OverPi * fmaf(kGeluCubic * z * z, z, z), s, c);
            a = z * s;
            // beyond |z| = 16 one of s and 1 - s is zero: the clamp keeps the
            // polynomial finite there
            const float zc = fminf(fmaxf(z, -16.0f), 16.0f);
            d = fmaf(a * c, 2.0f * kSqrt2OverPi * fmaf(3.0f * kGeluCubic * zc, zc, 1.0f), s);
            break;
        }
        case ACT_SILU:
            logistic(z, s, c);
            a = z * s;
            d = fmaf(a, c, s);
            break;
        default:
            a = z;
            d = 1.0f;
    }
}

}  // namespace emu
