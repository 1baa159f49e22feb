// activation.h - the activations that the layer's kernels apply in fp32 before a result is rounded.
//
//     silu(v)      = v sigmoid(v)
//     gelu_tanh(v) = v (1 + tanh(u)) / 2 = v sigmoid(2 u),   u = sqrt(2 / pi) (v + 0.044715 v^3)
#pragma once

#include "scan_update.h"

namespace jscan {

enum class Act : int { None, Silu, GeluTanh };

// 1 / (1 + e^-v) with the hardware exponential and reciprocal.  Its relative error is a few units of 2^-24 for v > 0 and
// grows to about 2 |v| 2^-24 below, where the rounding of the exponent counts (1e-5 at v = -87); from v = -88.8 on e^-v is
// infinite and the result 0, so silu and gelu_tanh are zero where they would be below 3e-37 in size.
__device__ __forceinline__ float sigmoid_f32(float v) {
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-v * kLog2e));
}

template <Act A> __device__ __forceinline__ float activate(float v) {
    if constexpr (A == Act::Silu) return v * sigmoid_f32(v);
    if constexpr (A == Act::GeluTanh) {
        constexpr float kTwoRoot = 1.59576912160573071176f;   // 2 sqrt(2 / pi)
        return v * sigmoid_f32(kTwoRoot * __builtin_fmaf(0.044715f * v * v, v, v));
    }
    return v;
}

// The same with the activation as a value that is the same in every lane.
__device__ __forceinline__ float activate(float v, Act a) {
    return a == Act::Silu ? activate<Act::Silu>(v) : a == Act::GeluTanh ? activate<Act::GeluTanh>(v) : v;
}

// d silu(v) / dv = g (1 + v (1 - g)), g = sigmoid(v)
__device__ __forceinline__ float silu_slope(float v) {
    const float g = sigmoid_f32(v);
    return g * __builtin_fmaf(v, 1.0f - g, 1.0f);
}

// What follows the scan in its layer: out = (y + skip x) silu(z), skip one value per channel.
// Without a skip or without a gate their part is left out.  z rows start every ld_z elements, in the order of x's.
struct OutGate {
    const float *skip;
    const void *z;
    int64_t ld_z;
};
__device__ __forceinline__ float gated_output(float y, bool skipped, float skip, float x, bool gated, float z) {
    if (skipped) y = __builtin_fmaf(skip, x, y);
    return gated ? y * activate<Act::Silu>(z) : y;
}

}  // namespace jscan
