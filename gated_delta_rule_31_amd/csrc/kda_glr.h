// Shared parts of the gated linear recurrence's kernels (kda_glr_fwd.hip, kda_glr_bwd.hip): for
// every channel of a row
//   g_t = lower sigmoid(e^A (z_t + bias))  (the library's bounded decay), or as given, <= 0
//   a_t = e^{g_t},   b_t = f_t i_t x_t,    f = sqrt(1 - e^{2g}) or 1,   i = sigmoid(i_t) or 1
//   h_t = a_t h_{t-1} + b_t
// A stretch of rows maps the state in front of it to the one behind it as h -> A h + H; a
// sequence that begins inside it makes A minus zero.  Two stretches joined: (A2 A1, A2 H1 + H2), or, where a sequence
// begins in either, A minus zero: as a product the mark would be lost to a second one (-0 x -0 = +0) and to a NaN.
// Where A is minus zero the state in front is not looked at, so nothing of one sequence reaches another,
// infinities and NaN among it; where decays alone made it zero (plus zero: they are not negative) it
// is, so that an infinity or a NaN of a sequence is not forgotten by it.
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

constexpr float CUT = -0.f;  // the A of a stretch in which a sequence begins
__host__ __device__ __forceinline__ bool is_cut(float a) { return __builtin_bit_cast(uint32_t, a) == 0x80000000u; }
// The state behind a stretch from the one in front of it, and the A of two stretches one behind the other.
__host__ __device__ __forceinline__ float join(float a, float h, float before) { return is_cut(a) ? h : fmaf(a, before, h); }
__host__ __device__ __forceinline__ float both(float a, float b) { return is_cut(a) || is_cut(b) ? CUT : a * b; }

// The types of a call: x and the logits are T, log decays float32.
template <typename T, bool LOGITS>
using gate_t = std::conditional_t<LOGITS, T, float>;

// Launches.  Rows are cut into tiles, and a wave goes through a tile's rows for 64 VEC channels:
//   1. A and H of every tile (with one tile: not needed)
//   2. the state in front of every tile (with few tiles their readers join the words themselves)
//   3. the rows themselves, from the state in front of their tile
// so the rows are read twice, the second time partly from the last-level cache.  Reading them once was measured for 7957
// x 4096: tiles that wait for what the tiles in front publish, 97-102 us (63 without the waiting) against 108 for these
// launches, which wait for nothing; and workgroups that take 16 channels through all rows, 109 us at best.

constexpr int GLR_FEW = 16;  // tiles that readers join themselves: a launch less where launches are what a call takes
constexpr int U = 8;         // rows that a wave has on their way

// A wave's tile: its column of channels, rows and marks.
struct GlrPlace {
    int tile, c, count, own;     // count: rows of the tile; own: those of them that belong to a sequence
    int64_t t0;
    uint64_t first, last;
    bool there;
};
template <int VEC>
__device__ __forceinline__ GlrPlace glr_place(const GlrArgs &a, int wave) {
    GlrPlace p;
    p.tile = wave / a.tiles.columns;
    p.c = (wave % a.tiles.columns * 64 + (threadIdx.x & 63)) * VEC;
    p.there = p.c < a.C;
    p.t0 = (int64_t)p.tile * a.tiles.rows;
    const int64_t left = a.seqs.rows - p.t0, used = (int64_t)__builtin_amdgcn_readfirstlane((int)a.seqs.limit()) - p.t0;
    p.count = (int)(left < a.tiles.rows ? left : a.tiles.rows);
    p.own = (int)(used < 0 ? 0 : used < p.count ? used : p.count);
    uniform_marks(a.seqs, p.t0, p.count, p.first, p.last);
    return p;
}

// The state in front of a tile (reverse: behind it).
template <int VEC>
__device__ __forceinline__ void glr_front(float (&h)[VEC], const GlrArgs &a, const float *front, int tile, int c, bool reverse) {
#pragma unroll
    for (int i = 0; i < VEC; ++i) h[i] = 0.f;
    if (a.tiles.n == 1) return;
    if (front) return load_f32<VEC>(h, front + (int64_t)tile * a.C + c);
    const int n = reverse ? a.tiles.n - 1 - tile : tile;
#pragma unroll 4
    for (int j = 0; j < n; ++j) {
        float w[2 * VEC];
        load_f32<2 * VEC>(w, a.tiles.words + ((int64_t)(reverse ? a.tiles.n - 1 - j : j) * a.C + c) * 2);
#pragma unroll
        for (int i = 0; i < VEC; ++i) h[i] = join(w[2 * i], w[2 * i + 1], h[i]);
    }
}
template <int VEC>
__device__ __forceinline__ void glr_word(const GlrArgs &a, int tile, int c, const float (&A)[VEC], const float (&H)[VEC]) {
    Raw<float, 2 * VEC> w;
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
        w.set(2 * i, A[i]);
        w.set(2 * i + 1, H[i]);
    }
    w.store(a.tiles.words + ((int64_t)tile * a.C + c) * 2);
}

// the tiles of a call, and of a launch whose lanes take `vec` channels each
void glr_plan(GlrArgs &a);
void carve_glr_tiles(GlrArgs &a, Pieces &w);
inline int64_t glr_waves(GlrArgs &a, int vec) {
    a.tiles.columns = (a.C + 64 * vec - 1) / (64 * vec);
    return (int64_t)a.tiles.n * a.tiles.columns;
}
// a.tiles.front from the words, if there are enough tiles for it to be wanted
hipError_t launch_glr_carry(const GlrArgs &a, bool reverse, hipStream_t stream);

}  // namespace kda
