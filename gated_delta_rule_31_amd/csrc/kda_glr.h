// Shared parts of the gated linear recurrence's kernels (kda_glr_fwd.hip, kda_glr_bwd.hip): for
// every channel of a row
//   g_t = lower sigmoid(e^A (z_t + bias))  (the library's bounded decay), or as given, <= 0
//   a_t = e^{g_t},   b_t = f_t i_t x_t,    f = sqrt(1 - e^{2g}) or 1,   i = sigmoid(i_t) or 1
//   h_t = a_t h_{t-1} + b_t
// A stretch of rows maps the state in front of it to the one behind it as h -> A h + H; a
// sequence that begins inside it makes A zero.  Two stretches joined: (A2 A1, A2 H1 + H2).
// Where A is zero the state in front is not looked at, so nothing of one sequence reaches another,
// infinities and NaN among it.
#pragma once

#include "kda_rows.h"

namespace kda {

// What a channel's gate is made of: t = scale2 z + bias2 is log2(e) e^A (z + bias).
template <int VEC, bool LOGITS>
struct GateConst {
    float scale2[VEC], bias2[VEC];
    __device__ __forceinline__ void load(const GlrGates &g, int c) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            if constexpr (LOGITS) {
                scale2[i] = expf(g.log_scale[(c + i) / g.K]) * LOG2E;
                bias2[i] = g.bias ? scale2[i] * g.bias[c + i] : 0.f;
            } else {
                scale2[i] = bias2[i] = 0.f;
            }
        }
    }
};

// One row's gates.
struct Gate {
    float a, f, i;    // decay; what the input is multiplied by; the input gate
    float p, q, j;    // logits: sigmoid(u) and 1 - that; 1 - i
};

// sqrt(1 - e^{2g}) from a = e^g and x = 2g: 1 - a^2 loses digits for a near 1, where the series of
// -expm1(x) takes over (six terms: 5e-8 at |x| = 1/4, where 1 - a^2 is off by 5e-7 at most).
__device__ __forceinline__ float keep_norm(float a, float x) {
    const float s = fmaf(x, fmaf(x, fmaf(x, fmaf(x, fmaf(x, 1.f / 720, 1.f / 120), 1.f / 24), 1.f / 6), 0.5f), 1.f);
    return __builtin_amdgcn_sqrtf(x > -0.25f ? -x * s : fmaf(-a, a, 1.f));
}

template <bool LOGITS, bool NORM, bool GATED>
__device__ __forceinline__ Gate make_gate(float z, float in, float scale2, float bias2, float lower) {
    Gate g;
    float x;  // the log decay
    if constexpr (LOGITS) {
        const float e = __builtin_amdgcn_exp2f(-fmaf(scale2, z, bias2));
        g.p = __builtin_amdgcn_rcpf(1.f + e);
        g.q = fminf(e, 3e38f) * g.p;
        x = lower * g.p;
    } else {
        g.p = g.q = 0.f;
        x = z;
    }
    g.a = __builtin_amdgcn_exp2f(LOG2E * x);
    g.f = NORM ? keep_norm(g.a, 2.f * x) : 1.f;
    g.j = 0.f;
    g.i = GATED ? sigmoid_f32(in, g.j) : 1.f;
    return g;
}

__device__ __forceinline__ float join(float a, float h, float before) { return a == 0.f ? h : fmaf(a, before, h); }

// The types of a call: x and the logits are T, log decays float32.
template <typename T, bool LOGITS>
using gate_t = std::conditional_t<LOGITS, T, float>;

// What a forward launch does with a tile of GLR_TILE rows: its A and H, or its rows.
enum { GLR_AGGREGATE, GLR_APPLY };
// kept[tile] = the state in front of every tile from the tiles' A and H
hipError_t launch_glr_carry(const float *agg, float *kept, int tiles, int C, bool reverse, hipStream_t stream);
hipError_t launch_glr_tiles(const GlrArgs &a, bool fp32, bool wide, int mode, hipStream_t stream);

}  // namespace kda
