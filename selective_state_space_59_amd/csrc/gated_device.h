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

// Logistics of v = v2 / log2(e).
__device__ __forceinline__ Sig sigmoid_pair(float v2) {
    const float t = hw_exp2(-fabsf(v2));  // in (0, 1]; NaN stays NaN
    const float hi = hw_rcp(1.0f + t), lo = t * hi;
    Sig r;
    r.s = v2 < 0.0f ? lo : hi;
    r.c = v2 < 0.0f ? hi : lo;
    return r;
}
// sig(v) alone: 1 / (1 + e^-v) does not cancel either.
__device__ __forceinline__ float sigmoid(float v2) { return hw_rcp(1.0f + hw_exp2(-v2)); }

// 1 - a^2 for a = 2^{y}, y <= 0 (not above 0 where y > 0).
__device__ __forceinline__ float one_minus_sq(float y, float a) {
    // -(e^w - 1) with w = 2 ln2 y, as w (1 + w/2 + w^2/6 + ...) in powers of y
    constexpr float k = 1.38629436111989062f;
    float p = __builtin_fmaf(y, k * k * k * k * k / 120.0f, k * k * k * k / 24.0f);
    p = __builtin_fmaf(y, p, k * k * k / 6.0f);
    p = __builtin_fmaf(y, p, k * k / 2.0f);
    p = __builtin_fmaf(y, p, k);
    // |w| < 1/8: the series' next term is below 2^-24 of it; beyond, 1 - a^2 > 0.117 loses at
    // most 3 bits to the subtraction
    const float series = -y * p, direct = __builtin_fmaf(-a, a, 1.0f);
    return y > -0.09f ? series : direct;
}

// Per-channel constants of a lane, A and the biases in units of the exponential's argument
// (times log2(e)).
struct GateChannel {
    float A2, gb2, ib2;
};

__device__ __forceinline__ float gate_arg(float g, float b2) { return __builtin_fmaf(g, kLog2e, b2); }

// a and b of one step.  `g`, `ig` without their biases; IG: an input gate is given.
template <int MODE, bool IG>
__device__ __forceinline__ void gate_step(float x, float g, float ig, const GateChannel &c, float &a, float &b) {
    if constexpr (MODE == SSM_GATE_DECAY) {
        a = g;
        b = x;
    } else if constexpr (MODE == SSM_GATE_SIGMOID) {
        const Sig s = sigmoid_pair(gate_arg(g, c.gb2));
        a = s.c;
        b = s.s * x;
    } else {
        const float y = c.A2 * sigmoid(gate_arg(g, c.gb2));
        a = hw_exp2(y);
        const float q = one_minus_sq(y, a);
        b = __builtin_amdgcn_sqrtf(q < 0.0f ? 0.0f : q) * x;
        if constexpr (IG) b *= sigmoid(gate_arg(ig, c.ib2));
    }
}

// One step with all that its gradients need.
template <int MODE, bool IG>
struct Gate {
    float a, w;  // h_t = a h_{t-1} + w x
    float s, sc; // the gate's logistic and its derivative
    float i, ic; // the input gate's
    float beta, inv_beta;
};

struct Logistic {
    float s, sc;  // sig(v), sig(v) (1 - sig(v))
};
__device__ __forceinline__ Logistic logistic(float v2) {
    const float t = hw_exp2(-fabsf(v2)), hi = hw_rcp(1.0f + t), lo = t * hi;
    return {v2 < 0.0f ? lo : hi, lo * hi};
}

template <int MODE, bool IG>
__device__ __forceinline__ Gate<MODE, IG> gate_of(float g, float ig, const GateChannel &c) {
    Gate<MODE, IG> o = {};
    if constexpr (MODE == SSM_GATE_DECAY) {
        o.a = g;
        o.w = 1.0f;
    } else if constexpr (MODE == SSM_GATE_SIGMOID) {
        const Sig s = sigmoid_pair(gate_arg(g, c.gb2));
        o.a = s.c;
        o.w = o.s = s.s;
        o.sc = s.s * s.c;
    } else {
        const Logistic r = logistic(gate_arg(g, c.gb2));
        o.s = r.s;
        o.sc = r.sc;
        const float y = c.A2 * r.s;
        o.a = hw_exp2(y);
        const float q = one_minus_sq(y, o.a);
        // 0 where sqrt(1 - a^2) is 0, and below the normal range, whose inverse root the hardware
        // makes an infinity
        o.inv_beta = q >= 0x1p-126f ? __builtin_amdgcn_rsqf(q) : 0.0f;
        o.w = o.beta = q * o.inv_beta;
        if constexpr (IG) {
            const Logistic i = logistic(gate_arg(ig, c.ib2));
            o.i = i.s;
            o.ic = i.sc;
            o.w *= i.s;
        }
    }
    return o;
}

// Gradients of one step: da = dL/da (lambda h_{t-1}, 0 at a reset), db = dL/db (lambda).
// dg, di are also the contributions to the biases' gradients, dA to A's.
struct GateGrad {
    float dx, dg, di, dA;
};

template <int MODE, bool IG>
__device__ __forceinline__ GateGrad gate_grad(const Gate<MODE, IG> &t, float x, float A, float da, float db) {
    GateGrad o = {};
    if constexpr (MODE == SSM_GATE_DECAY) {
        o.dx = db;
        o.dg = da;
    } else if constexpr (MODE == SSM_GATE_SIGMOID) {
        o.dx = db * t.s;
        o.dg = __builtin_fmaf(db, x, -da) * t.sc;
    } else {
        const float di = db * x;
        if constexpr (IG) o.di = di * t.beta * t.ic;
        o.dx = db * t.w;
        // dL/d(log a): da a from the state, and d sqrt(1 - a^2) / d(log a) = -a^2 / sqrt(1 - a^2)
        const float dbeta = IG ? di * t.i : di;
        const float dla = t.a * __builtin_fmaf(-dbeta * t.a, t.inv_beta, da);
        o.dA = dla * t.s;
        o.dg = dla * A * t.sc;
    }
    return o;
}

}  // namespace ssm
