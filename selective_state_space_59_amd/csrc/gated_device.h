// gated_device.h -- the gates of the gated linear recurrence (gfx950): decay and
// input weight of one step, and their derivatives, in fp32.
//
//   h_t = a_t h_{t-1} + b_t,  with for each mode (ssm.h, ssm_gate_mode_t)
//   DECAY    a = g,                  b = x
//   SIGMOID  s = sig(g),  a = 1 - s, b = s x
//   RATE     r = sig(g),  a = e^{A r},  b = sqrt(1 - a^2) i x,  i = sig(ig) or 1
//
// Both halves s and 1 - s of a logistic come from one exponential of -|v|, so
// neither cancels.  1 - a^2 = -(e^{2 A r} - 1) is a series near a = 1, where the
// subtraction would lose the channels that remember longest.
#pragma once

#include <type_traits>

#include "../../include/ssm.h"
#include "ssm_device.h"

namespace ssm {

// Host side: call f(io type, mode constant, has-in_gate constant) for a call's options.
template <typename F>
void gate_dispatch(int32_t io_dtype, int32_t mode, bool in_gate, F &&f) {
    auto with_io = [&](auto io) {
        if (mode == SSM_GATE_DECAY)
            f(io, std::integral_constant<int, SSM_GATE_DECAY>{}, std::false_type{});
        else if (mode == SSM_GATE_SIGMOID)
            f(io, std::integral_constant<int, SSM_GATE_SIGMOID>{}, std::false_type{});
        else if (in_gate)
            f(io, std::integral_constant<int, SSM_GATE_RATE>{}, std::true_type{});
        else
            f(io, std::integral_constant<int, SSM_GATE_RATE>{}, std::false_type{});
    };
    if (io_dtype == SSM_BF16)
        with_io(io_bf16{});
    else
        with_io(io_f32{});
}

struct Sig {
    float s, c;  // sig(v) and 1 - sig(v)
};

__device__ __forceinline__ Sig sigmoid_pair(float v) {
    const float t = hw_exp2(-fabsf(v) * kLog2e);  // in (0, 1]; NaN stays NaN
    const float hi = hw_rcp(1.0f + t), lo = t * hi;
    Sig r;
    r.s = v < 0.0f ? lo : hi;
    r.c = v < 0.0f ? hi : lo;
    return r;
}

// 1 - a^2 for a = e^{la}, w = 2 la <= 0 (0 where la > 0).
__device__ __forceinline__ float one_minus_sq(float w, float a) {
    float p = __builtin_fmaf(w, 1.0f / 720.0f, 1.0f / 120.0f);
    p = __builtin_fmaf(w, p, 1.0f / 24.0f);
    p = __builtin_fmaf(w, p, 1.0f / 6.0f);
    p = __builtin_fmaf(w, p, 0.5f);
    p = __builtin_fmaf(w, p, 1.0f);
    // |w| < 1/4: the series' next term is below 2^-24 of it
    const float q = w > -0.25f ? -w * p : __builtin_fmaf(-a, a, 1.0f);
    return q < 0.0f ? 0.0f : q;
}

// Per-channel constants of a lane.
struct GateChannel {
    float A, gb, ib;
};

// a and b of one step.  `g`, `ig` without their biases; IG: an input gate is given.
template <int MODE, bool IG>
__device__ __forceinline__ void gate_step(float x, float g, float ig, const GateChannel &c, float &a, float &b) {
    if constexpr (MODE == SSM_GATE_DECAY) {
        a = g;
        b = x;
    } else if constexpr (MODE == SSM_GATE_SIGMOID) {
        const Sig s = sigmoid_pair(g + c.gb);
        a = s.c;
        b = s.s * x;
    } else {
        const float la = c.A * sigmoid_pair(g + c.gb).s;
        a = hw_exp2(la * kLog2e);
        b = __builtin_amdgcn_sqrtf(one_minus_sq(2.0f * la, a)) * x;
        if constexpr (IG) b *= sigmoid_pair(ig + c.ib).s;
    }
}

// Gradients of one step: da = dL/da (lambda h_{t-1}, 0 at a reset), db = dL/db (lambda).
// dg, di are also the contributions to the biases' gradients, dA to A's.
struct GateGrad {
    float dx, dg, di, dA;
};

template <int MODE, bool IG>
__device__ __forceinline__ GateGrad gate_grad(float x, float g, float ig, const GateChannel &c, float da, float db) {
    GateGrad o = {};
    if constexpr (MODE == SSM_GATE_DECAY) {
        o.dx = db;
        o.dg = da;
    } else if constexpr (MODE == SSM_GATE_SIGMOID) {
        const Sig s = sigmoid_pair(g + c.gb);
        o.dx = db * s.s;
        o.dg = __builtin_fmaf(db, x, -da) * (s.s * s.c);
    } else {
        const Sig r = sigmoid_pair(g + c.gb);
        const float la = c.A * r.s, a = hw_exp2(la * kLog2e), q = one_minus_sq(2.0f * la, a);
        const float rs = q > 0.0f ? __builtin_amdgcn_rsqf(q) : 0.0f;  // 1 / sqrt(1 - a^2), 0 where that is 0
        Sig i = {1.0f, 0.0f};
        if constexpr (IG) i = sigmoid_pair(ig + c.ib);
        const float dbb = db * (q * rs);  // dL/d(i x)
        o.dx = dbb * i.s;
        if constexpr (IG) o.di = dbb * x * (i.s * i.c);
        // dL/d(log a): da a from the state, and d sqrt(1 - a^2) / d(log a) = -a^2 / sqrt(1 - a^2)
        const float dla = a * __builtin_fmaf(-(db * i.s * x) * a, rs, da);
        o.dA = dla * r.s;
        o.dg = dla * c.A * (r.s * r.c);
    }
    return o;
}

}  // namespace ssm
