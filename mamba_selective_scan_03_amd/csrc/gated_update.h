// gated_update.h - how the gated recurrence advances by one token, and how its gradient walks back.
//
// One fp32 state per channel (no expansion over d_state), its gate g an input like u:
//     decay form     a = exp(g)       h <- a h + u
//     sigmoid form   a = sigmoid(g)   h <- a h + b u,   b = 1 - a = sigmoid(-g)
// Every kernel of the recurrence takes a and b from gate() and walks along tokens, be it with a state or with a run's
// map, by gated_advance().
//
// Backward.  With G_t = dL/dh_t and c_t = a_t G_t, the gradient that token t hands to token t-1,
//     G_t = dy_t + c_{t+1},   c_t = a_t G_t       (a reverse scan of the same affine kind)
//     decay form     du_t = G_t        dg_t = c_t h_{t-1}
//     sigmoid form   du_t = b_t G_t    dg_t = c_t b_t (h_{t-1} - u_t)
// from da/dg = a (decay) and a b (sigmoid), db/dg = -a b.
#pragma once

#include "scan_update.h"

namespace jscan {

enum class GateForm : int { Decay, Sigmoid };

struct Gate {
    float a, b;   // decay of the state; weight of the input (1 in the decay form)
};

// exp(g) is the hardware base-2 exponential of g log2(e).  The sigmoid is formed from
// t = exp(-|g|) in (0, 1], so that both a and 1 - a keep their relative precision at either
// end and no infinity arises from a finite gate: the larger of the two is 1 / (1 + t), the
// smaller t / (1 + t).  g = -inf gives a = 0 in both forms (a finite state is dropped; an infinite one becomes
// NaN), +inf in the sigmoid form a = 1, b = 0; a NaN stays one.
template <GateForm F> __device__ __forceinline__ Gate gate(float g) {
    if constexpr (F == GateForm::Decay) {
        return Gate{__builtin_amdgcn_exp2f(g * kLog2e), 1.0f};
    } else {
        const float t = __builtin_amdgcn_exp2f(-fabsf(g) * kLog2e);
        const float big = __builtin_amdgcn_rcpf(1.0f + t), small = t * big;
        return g < 0.0f ? Gate{small, big} : Gate{big, small};
    }
}

// The input term of a token: u, or b u.
template <GateForm F> __device__ __forceinline__ float gated_input(Gate k, float u) {
    return F == GateForm::Decay ? u : k.b * u;
}

__device__ __forceinline__ float gated_advance(float h, float a, float input) { return __builtin_fmaf(a, h, input); }

}  // namespace jscan
