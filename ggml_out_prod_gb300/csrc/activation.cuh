// activation.cuh -- the activations of the gated feed-forward block.
#pragma once

#include "oop_internal.cuh"

namespace oop {

// 1 / (1 + exp(-v)), and with REST its difference from 1 without cancellation.  Of the two
// the one below 1/2 is taken from exp(-|v|), so it falls to 0 as it should, whatever is
// multiplied with it (a limit on the argument would leave 2e-35, which a gate of -1e35 or
// its square shows), and the divisor stays between 1 and 2, in the fast division's range
// (2 ulp).
__device__ __forceinline__ float logistic(float v) {
    const float e = expf(-fabsf(v)), s = __fdividef(1.f, 1.f + e);
    return v < 0.f ? e * s : s;
}
__device__ __forceinline__ float logistic(float v, float &rest) {
    const float e = expf(-fabsf(v)), s = __fdividef(1.f, 1.f + e);
    rest = v < 0.f ? s : e * s;
    return v < 0.f ? e * s : s;
}

constexpr float kGeluTwice = 1.5957691216057308f;          // 2 sqrt(2 / pi)

// (1 + tanh z) / 2 is the logistic function of 2 z: no cancellation for negative v.
__device__ __forceinline__ float gelu_argument(float v) { return kGeluTwice * (v + 0.044715f * v * v * v); }

__device__ __forceinline__ float activation_of(int act, float v) {
    if (act == OOP_ACT_SILU) return v * logistic(v);
    if (act == OOP_ACT_GELU_TANH) return v * logistic(gelu_argument(v));
    if (act == OOP_ACT_GELU_ERF) return v * (0.5f * erfcf(-v * 0.7071067811865476f));
    return v < 0.f ? 0.f : v;
}

// Four at a time as a call, where the code would be repeated for every register of a row.
static __device__ __noinline__ float4 activation_call(int act, float4 v) {
    return make_float4(activation_of(act, v.x), activation_of(act, v.y), activation_of(act, v.z), activation_of(act, v.w));
}

// The activation and its derivative.
__device__ __forceinline__ float activation_and_slope(int act, float v, float &slope) {
    if (act == OOP_ACT_SILU) {
        float rest;
        const float s = logistic(v, rest);
        slope = s + v * s * rest;
        return v * s;
    }
    if (act == OOP_ACT_GELU_TANH) {
        float rest;
        const float s = logistic(gelu_argument(v), rest);
        const float both = s * rest;                       // 0 long before v * v overflows
        slope = both == 0.f ? s : s + v * both * (kGeluTwice * (1.f + 0.134145f * v * v));
        return v * s;
    }
    if (act == OOP_ACT_GELU_ERF) {
        const float e = 0.5f * erfcf(-v * 0.7071067811865476f);
        slope = e + v * (expf(-0.5f * v * v) * 0.3989422804014327f);
        return v * e;
    }
    slope = v > 0.f ? 1.f : v == v ? 0.f : v;
    return v < 0.f ? 0.f : v;
}

}  // namespace oop
