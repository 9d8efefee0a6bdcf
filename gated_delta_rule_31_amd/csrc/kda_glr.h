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

// ------------------------------------------------------------------ one pass over a long row
//
// A workgroup holds a tile of rows in registers, publishes the tile's A and H, and waits for what the
// tiles in front do to the state; so a row is read once, however long the sequence.  Tiles come in
// groups: a group's last tile publishes the A and H of the whole group as soon as the tiles of its
// group are there.  The state in front of a tile is that of the groups before its own, joined in
// their order, and then the tiles before it in its group: about the root of the number of tiles to
// look at, two publications deep however many tiles there are, and always the same sums in the
// same order.  (With a state carried from group to group every group would wait for the one before.)
//
// Workgroups take their tile by a ticket, the first tile first: one only waits for tiles whose
// workgroups have taken theirs, are running, and wait for smaller tickets alone.  So the smallest
// ticket that has not finished always can, and every wait ends.
//
// What is published is written, and read, by relaxed atomics of device scope, which do not stay in an XCD's
// cache.  The flag is stored when the wave's earlier stores have been acknowledged (vmcnt 0), so
// whoever sees the flag reads what is behind it.  (A release of device scope would write back the
// XCD's whole cache, outputs and all, for every tile.)

__device__ __forceinline__ void publish_word(uint64_t *p, float a, float h) {
    __hip_atomic_store(p, (uint64_t)__builtin_bit_cast(uint32_t, h) << 32 | __builtin_bit_cast(uint32_t, a), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ void publish_flag(uint32_t *flag, int lane) {
    __builtin_amdgcn_s_waitcnt(0);
    asm volatile("" ::: "memory");
    if (lane == 0) __hip_atomic_store(flag, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// One wave: A and H of the entries lo <= i < hi joined in their order, for VEC channels a lane.  Waits for all of them.
template <int VEC>
__device__ __forceinline__ void look(float (&A)[VEC], float (&H)[VEC], const uint64_t *entry, const uint32_t *there, int columns, int C, int lo, int hi,
                                     int lane, bool on) {
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
        A[i] = 1.f;
        H[i] = 0.f;
    }
    for (int at = lo; at < hi; at += 64) {
        const int e = at + lane;
        while (!__all(e >= hi || __hip_atomic_load(there + (int64_t)e * columns, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT))) __builtin_amdgcn_s_sleep(2);
    }
    asm volatile("" ::: "memory");
    if (!on) return;
    constexpr int U = 8;
    for (int at = lo; at < hi; at += U) {
        uint64_t w[U][VEC];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < VEC; ++i)
                w[u][i] = __hip_atomic_load(entry + (int64_t)(at + u < hi ? at + u : hi - 1) * C + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (at + u < hi)
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    const float a = __builtin_bit_cast(float, (uint32_t)w[u][i]), h = __builtin_bit_cast(float, (uint32_t)(w[u][i] >> 32));
                    H[i] = join(a, h, H[i]);
                    A[i] *= a;
                }
    }
}

// The whole of it, for a workgroup of WAVES waves whose parts of the tile have left their A and H in
// sA, sH (a barrier behind them), in the order in which the state goes through them.  On return, behind a
// barrier, `state` (...) gives the state in front of the part of any wave.
template <int VEC, int WAVES>
struct LookBack {
    float A[WAVES][64][VEC], H[WAVES][64][VEC];    // of the tile's parts, first part first
    float LA[WAVES][64][VEC], LH[WAVES][64][VEC];  // of what is in front: groups by waves 1.., the own group's tiles by wave 0
    int ticket;

    // the tile that this workgroup takes
    __device__ __forceinline__ int take(uint32_t *counter) {
        if (threadIdx.x == 0) ticket = (int)__hip_atomic_fetch_add(counter, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        __syncthreads();
        return __builtin_amdgcn_readfirstlane(ticket);
    }

    __device__ __forceinline__ void front(const GlrLook &g, int C, int tile, int column, int c, bool on, int wave, int lane) {
        const int group = tile / g.group, begin = group * g.group, groups = g.groups();
        float a[VEC], h[VEC];
        if (wave == 0) {
            float ta[VEC], th[VEC];
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                ta[i] = 1.f;
                th[i] = 0.f;
                for (int w = 0; w < WAVES; ++w) {
                    th[i] = join(A[w][lane][i], H[w][lane][i], th[i]);
                    ta[i] *= A[w][lane][i];
                }
                if (on) publish_word(g.tile + (int64_t)tile * C + c + i, ta[i], th[i]);
            }
            publish_flag(g.tile_there + (int64_t)tile * g.columns + column, lane);
            look<VEC>(a, h, g.tile + c, g.tile_there + column, g.columns, C, begin, tile, lane, on);
            if (tile + 1 == begin + g.group && group + 1 < groups) {
#pragma unroll
                for (int i = 0; i < VEC; ++i)
                    if (on) publish_word(g.whole + (int64_t)group * C + c + i, a[i] * ta[i], join(ta[i], th[i], h[i]));
                publish_flag(g.group_there + (int64_t)group * g.columns + column, lane);
            }
        } else {
            const int each = (group + WAVES - 2) / (WAVES - 1), lo = (wave - 1) * each, hi = lo + each < group ? lo + each : group;
            look<VEC>(a, h, g.whole + c, g.group_there + column, g.columns, C, lo, hi, lane, on);
        }
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            LA[wave][lane][i] = a[i];
            LH[wave][lane][i] = h[i];
        }
        __syncthreads();
    }

    // the state in front of part `part`
    __device__ __forceinline__ void state(float (&x)[VEC], int part, int lane, bool alone) const {
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            float s = 0.f;
            if (!alone) {
                for (int w = 1; w < WAVES; ++w) s = join(LA[w][lane][i], LH[w][lane][i], s);
                s = join(LA[0][lane][i], LH[0][lane][i], s);
            }
            for (int w = 0; w < part; ++w) s = join(A[w][lane][i], H[w][lane][i], s);
            x[i] = s;
        }
    }
};

// the columns of channels of a launch, and zeros where its flags and the ticket are
hipError_t launch_glr_begin(GlrLook &g, int columns, hipStream_t stream);
// tiles of a call and their groups
void glr_plan(GlrLook &g, int64_t rows, int tile_rows);
void carve_glr_look(GlrLook &g, Pieces &w, int C);

}  // namespace kda
