// kda_conv.hip -- the short causal convolution of a layer's rows (gfx950), channel by channel:
//   pre_t = bias + sum_w weight[w] x_{t-W+1+w},   out_t = silu(pre_t) or pre_t,
// over packed sequences, the W - 1 rows before a sequence being kept ones or zeros; its
// gradients; and decoding over a pool of kept rows.
//
// Bound by memory: a row is read and a row written.  A lane owns VEC neighbouring channels (one
// load of a row: two of them forward and in decode, four for gradients, where rows allow it) and goes through a run of rows with the last W - 1 of them in registers, so a
// row is read once, but for the W - 1 in front of a run.  Where sequences begin and end is the
// same for all lanes of a wave: two bit masks for a run, looked up once.  W = 4, bf16, a large copy having 5.0 TB/s:
// 7957 packed rows of 12288 channels 81 us (4.85 TB/s); gradients of 8192 rows of 4096 channels 52 us (0.2 GB and
// 0.02 of partial sums) and 5 for the sums; decoding 64 requests of 1 to 4 tokens, 12288 channels, 7.8 us
// (0.024 GB: a chain of table, state and output).  Channels of a lane, more waves against fewer instructions a row:
// forward 2, 4, 8 channels 82, 85, 89 us; gradients 59, 57, 65; decoding 7.8, 8.1, 9.9.
#include "kda_rows.h"

namespace kda {
namespace {

constexpr int WAVES = 4;

// the kept rows in front of row t (the first of sequence n where `whole`), newest last
template <typename T, int VEC, int W>
__device__ __forceinline__ void window(float (&f)[W - 1][VEC], const ConvArgs &a, int64_t t, int c) {
    const int n = a.seqs.of(t);
    const int64_t b = a.seqs.begin(n, t);
#pragma unroll
    for (int j = 1; j < W; ++j) {
        Raw<T, VEC> r;
        r.zero();
        if (t - j >= b) r.load(static_cast<const T *>(a.x) + (t - j) * a.x_stride + c);
        else if (a.s0) r.load(static_cast<const T *>(a.s0) + ((int64_t)n * (W - 1) + W - 1 + (t - j - b)) * a.D + c);
#pragma unroll
        for (int i = 0; i < VEC; ++i) f[W - 1 - j][i] = r.get(i);
    }
}

template <int VEC, int W>
__device__ __forceinline__ void taps(float (&w)[W][VEC], float (&b)[VEC], const float *weight, const float *bias, int c) {
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
#pragma unroll
        for (int j = 0; j < W; ++j) w[j][i] = weight[(int64_t)(c + i) * W + j];
        b[i] = bias ? bias[c + i] : 0.f;
    }
}

template <int VEC, int W>
__device__ __forceinline__ float convolve(const float (&w)[W][VEC], const float (&b)[VEC], const float (&f)[W - 1][VEC], float x, int i) {
    float pre = b[i];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) pre = fmaf(w[j][i], f[j][i], pre);
    return fmaf(w[W - 1][i], x, pre);
}

template <int VEC, int W>
__device__ __forceinline__ void shift(float (&f)[W - 1][VEC], float x, int i) {
#pragma unroll
    for (int j = 0; j + 1 < W - 1; ++j) f[j][i] = f[j + 1][i];
    f[W - 2][i] = x;
}

// what an empty sequence hands on: `to` = `from` or zeros, for the sequences that have no row
template <typename T>
__device__ __forceinline__ void empty_states(const Seqs &s, int64_t block, int64_t each, const T *from, T *to) {
    const int64_t i = block * (64 * WAVES) + threadIdx.x;
    if (i >= s.N * each) return;
    const int n = (int)(i / each);
    if (s.cu[n + 1] <= s.cu[n]) to[i] = from ? from[i] : T{};
}

template <typename T, int VEC, int W>
__global__ __launch_bounds__(64 * WAVES) void conv_fwd_kernel(const ConvArgs a, int blocks) {
    if ((int)blockIdx.x >= blocks)
        return empty_states(a.seqs, blockIdx.x - blocks, (int64_t)(W - 1) * a.D, static_cast<const T *>(a.s0), static_cast<T *>(a.sf));
    const int wave = blockIdx.x * WAVES + __builtin_amdgcn_readfirstlane(threadIdx.x / 64), lane = threadIdx.x & 63;
    const int tiles = (a.vecs + 63) / 64, run = wave / tiles, v = wave % tiles * 64 + lane, c = v * VEC;
    const int64_t t0 = (int64_t)run * a.run, limit = __builtin_amdgcn_readfirstlane((int)a.seqs.limit());
    if (run >= a.runs || v >= a.vecs || t0 >= limit) return;
    const int count = (int)(limit - t0 < a.run ? limit - t0 : a.run);
    uint64_t first, last;
    uniform_marks(a.seqs, t0, count, first, last);
    float w[W][VEC], b[VEC], f[W - 1][VEC];
    taps<VEC, W>(w, b, a.weight, a.bias, c);
    window<T, VEC, W>(f, a, t0, c);
    const int64_t sx = a.x_stride * sizeof(T), sd = a.D * sizeof(T);
    const char *x = static_cast<const char *>(a.x) + t0 * sx;
    char *out = static_cast<char *>(a.out) + t0 * sd;
    const uint32_t ct = c * (uint32_t)sizeof(T);
    constexpr int U = 16;
    for (int t = 0; t < count; t += U) {
        Raw<T, VEC> r[U];
        load_run(r, x + t * sx, sx, ct, count - t);
        const uint32_t ot = here(ct);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (t + u >= count) continue;
            if (t + u > 0 && first >> (t + u) & 1) window<T, VEC, W>(f, a, t0 + t + u, c);
            Raw<T, VEC> y;
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const float xi = r[u].get(i), pre = convolve<VEC, W>(w, b, f, xi, i);
                y.set(i, a.silu ? pre * sigmoid_f32(pre) : pre);
                shift<VEC, W>(f, xi, i);
            }
            y.store(out + (t + u) * sd, ot);
            if (a.sf && last >> (t + u) & 1) {
                T *to = static_cast<T *>(a.sf) + (int64_t)a.seqs.of(t0 + t + u) * (W - 1) * a.D + c;
#pragma unroll
                for (int j = 0; j < W - 1; ++j) {
                    Raw<T, VEC> k;
#pragma unroll
                    for (int i = 0; i < VEC; ++i) k.set(i, f[j][i]);
                    k.store(to + (int64_t)j * a.D);
                }
            }
        }
    }
}

// Gradients.  d pre_t = d out_t silu'(pre_t) with pre_t made again; row s receives weight[W-1-j] d pre_{s+j}
// from the W rows s..s+W-1 of its sequence, so a lane keeps the W sums that are open and closes one a row;
// a run goes on for W - 1 rows behind its end.  What a kept row receives, and what the rows handed on
// bring back, goes through the same sums (row -1 of a sequence is its newest kept row).  The weight's
// sums of a run are written as they are; launch_column_sums adds the runs in their order.
template <typename T, int VEC, int W>
__global__ __launch_bounds__(64 * WAVES) void conv_bwd_kernel(const ConvArgs a, int blocks) {
    if ((int)blockIdx.x >= blocks)
        return empty_states(a.seqs, blockIdx.x - blocks, (int64_t)(W - 1) * a.D, static_cast<const T *>(a.d_sf), static_cast<T *>(a.ds0));
    const int wave = blockIdx.x * WAVES + __builtin_amdgcn_readfirstlane(threadIdx.x / 64), lane = threadIdx.x & 63;
    const int tiles = (a.vecs + 63) / 64, run = wave / tiles, v = wave % tiles * 64 + lane, c = v * VEC;
    if (run >= a.runs || v >= a.vecs) return;
    const int64_t t0 = (int64_t)run * a.run, limit = __builtin_amdgcn_readfirstlane((int)a.seqs.limit());
    const int rows = (int)(a.seqs.rows - t0 < a.run ? a.seqs.rows - t0 : a.run);          // of this run
    const int own = (int)(limit - t0 < 0 ? 0 : limit - t0 < rows ? limit - t0 : rows);     // of them in a sequence
    const int count = (int)(limit - t0 < 0 ? 0 : limit - t0 < own + W - 1 ? limit - t0 : own + W - 1);
    T *dx = static_cast<T *>(a.dx) + t0 * a.D + c;
    float dw[W][VEC] = {}, db[VEC] = {};
    if (own > 0) {
        uint64_t first, last;
        uniform_marks(a.seqs, t0, count, first, last);
        float w[W][VEC], b[VEC], f[W - 1][VEC], acc[W][VEC] = {};
        taps<VEC, W>(w, b, a.weight, a.bias, c);
        window<T, VEC, W>(f, a, t0, c);
        int n = a.seqs.of(t0);
        int64_t begin = a.seqs.begin(n, t0) - t0;  // of the sequence, counted from t0 as t below
        const int64_t sx = a.x_stride * sizeof(T), sd = a.D * sizeof(T);
        const char *x = static_cast<const char *>(a.x) + t0 * sx, *d_out = static_cast<const char *>(a.d_out) + t0 * sd;
        const uint32_t ct = c * (uint32_t)sizeof(T);
        auto close = [&](int64_t s, const float(&g)[VEC]) {  // the sum of row s is whole
            Raw<T, VEC> r;
#pragma unroll
            for (int i = 0; i < VEC; ++i) r.set(i, g[i]);
            if (s >= begin) {
                if (s >= 0 && s < own) r.store(dx + s * a.D);
            } else if (a.ds0 && begin >= 0 && begin < own && s >= begin - (W - 1)) {
                r.store(static_cast<T *>(a.ds0) + ((int64_t)n * (W - 1) + W - 1 + (s - begin)) * a.D + c);
            }
        };
        constexpr int U = 4;
        for (int t = 0; t < count; t += U) {
            Raw<T, VEC> rx[U], rd[U];
            load_run(rx, x + t * sx, sx, ct, count - t);
            load_run(rd, d_out + t * sd, sd, ct, count - t);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (t + u >= count) continue;
                if (t + u > 0 && first >> (t + u) & 1) {
                    window<T, VEC, W>(f, a, t0 + t + u, c);
                    n = a.seqs.of(t0 + t + u);
                    begin = t + u;
                }
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    const float xi = rx[u].get(i);
                    float d = rd[u].get(i);
                    if (a.silu) {
                        const float pre = convolve<VEC, W>(w, b, f, xi, i), g = sigmoid_f32(pre);
                        d *= g * fmaf(pre, 1.f - g, 1.f);
                    }
#pragma unroll
                    for (int j = 0; j < W; ++j) acc[j][i] = fmaf(w[W - 1 - j][i], d, acc[j][i]);
                    if (t + u < own) {
#pragma unroll
                        for (int j = 0; j < W - 1; ++j) dw[j][i] = fmaf(d, f[j][i], dw[j][i]);
                        dw[W - 1][i] = fmaf(d, xi, dw[W - 1][i]);
                        db[i] += d;
                    }
                    shift<VEC, W>(f, xi, i);
                }
                if (last >> (t + u) & 1) {  // nothing behind it: what was handed on comes back, and all sums are whole
                    if (a.d_sf) {
#pragma unroll
                        for (int j = 0; j < W - 1; ++j) {
                            Raw<T, VEC> g;
                            g.load(static_cast<const T *>(a.d_sf) + ((int64_t)n * (W - 1) + W - 2 - j) * a.D + c);
#pragma unroll
                            for (int i = 0; i < VEC; ++i) acc[j][i] += g.get(i);
                        }
                    }
#pragma unroll
                    for (int j = 0; j < W; ++j) {
                        close(t + u - j, acc[j]);
#pragma unroll
                        for (int i = 0; i < VEC; ++i) acc[j][i] = 0.f;
                    }
                } else {
                    close(t + u - (W - 1), acc[W - 1]);
#pragma unroll
                    for (int i = 0; i < VEC; ++i) {
#pragma unroll
                        for (int j = W - 1; j > 0; --j) acc[j][i] = acc[j - 1][i];
                        acc[0][i] = 0.f;
                    }
                }
            }
        }
    }
    Raw<T, VEC> zero;
    zero.zero();
    for (int t = own; t < rows; ++t) zero.store(dx + (int64_t)t * a.D);
    if (!a.part) return;
#pragma unroll
    for (int j = 0; j <= W; ++j) {
        Raw<float, VEC> s;
#pragma unroll
        for (int i = 0; i < VEC; ++i) s.set(i, j < W ? dw[j < W ? j : 0][i] : db[i]);
        s.store(a.part + ((int64_t)run * (W + 1) + j) * a.D + c);
    }
}

template <typename T, int VEC, int W>
__global__ __launch_bounds__(64) void conv_step_kernel(const ConvStepArgs a) {
    const int tiles = (a.vecs + 63) / 64, b = blockIdx.x / tiles, v = blockIdx.x % tiles * 64 + threadIdx.x, c = v * VEC;
    const int len = a.slots.tokens(b);
    if (v >= a.vecs || len == 0) return;
    const T *x = static_cast<const T *>(a.x) + (int64_t)b * a.S * a.D + c;
    T *states = static_cast<T *>(a.states) + c, *out = static_cast<T *>(a.out) + (int64_t)b * a.S * a.D + c;
    float w[W][VEC], bias[VEC];
    taps<VEC, W>(w, bias, a.weight, a.bias, c);
    Raw<T, VEC> f[W - 1];
    const int64_t from = a.slots.from(b);
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
        f[j].zero();
        if (from >= 0) f[j].load(states + (from * (W - 1) + j) * a.D);
    }
    Raw<T, VEC> next;
    next.load(x);
    for (int t = 0; t < len; ++t) {
        const Raw<T, VEC> r = next;
        Raw<T, VEC> y;
        if (t + 1 < len) next.load(x + (int64_t)(t + 1) * a.D);
        const int64_t to = a.slots.to(b, t, len);
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            float pre = bias[i];
#pragma unroll
            for (int j = 0; j < W - 1; ++j) pre = fmaf(w[j][i], f[j].get(i), pre);
            pre = fmaf(w[W - 1][i], r.get(i), pre);
            y.set(i, a.silu ? pre * sigmoid_f32(pre) : pre);
        }
        y.store(out + (int64_t)t * a.D);
#pragma unroll
        for (int j = 0; j + 1 < W - 1; ++j) f[j] = f[j + 1];
        f[W - 2] = r;
        if (to >= 0)
#pragma unroll
            for (int j = 0; j < W - 1; ++j) f[j].store(states + (to * (W - 1) + j) * a.D);
    }
}

enum { FWD, BWD };
template <int KIND, typename T, int VEC>
hipError_t by_taps(const ConvArgs &a, hipStream_t stream) {
    const int blocks = (int)(((int64_t)((a.vecs + 63) / 64) * a.runs + WAVES - 1) / WAVES);
    const bool states = a.seqs.cu && (KIND == FWD ? a.sf : a.ds0);
    const int64_t more = states ? ((int64_t)a.seqs.N * (a.W - 1) * a.D + 64 * WAVES - 1) / (64 * WAVES) : 0;
    const dim3 grid((unsigned)(blocks + more)), block(64 * WAVES);
#define KDA_CONV(W_)                                                                                                   \
    case W_:                                                                                                           \
        if constexpr (KIND == FWD) hipLaunchKernelGGL((conv_fwd_kernel<T, VEC, W_>), grid, block, 0, stream, a, blocks); \
        else hipLaunchKernelGGL((conv_bwd_kernel<T, VEC, W_>), grid, block, 0, stream, a, blocks);                      \
        return hipGetLastError();
    switch (a.W) { KDA_CONV(2) KDA_CONV(3) KDA_CONV(4) }
#undef KDA_CONV
    return hipErrorNotSupported;
}
template <int KIND>
hipError_t by_type(ConvArgs &a, bool fp32, bool wide, hipStream_t stream) {
    constexpr int VEC = KIND == FWD ? CONV_FWD_VEC : CONV_BWD_VEC;
    a.vecs = wide ? a.D / VEC : a.D;
    conv_runs(a.seqs.rows, a.vecs, a.run, a.runs);
    if (wide) return fp32 ? by_taps<KIND, float, VEC>(a, stream) : by_taps<KIND, __bf16, VEC>(a, stream);
    return fp32 ? by_taps<KIND, float, 1>(a, stream) : by_taps<KIND, __bf16, 1>(a, stream);
}

template <typename T, int VEC>
hipError_t step_by_taps(const ConvStepArgs &a, hipStream_t stream) {
    const dim3 grid((unsigned)(a.B * ((a.vecs + 63) / 64))), block(64);
    switch (a.W) {
        case 2: hipLaunchKernelGGL((conv_step_kernel<T, VEC, 2>), grid, block, 0, stream, a); return hipGetLastError();
        case 3: hipLaunchKernelGGL((conv_step_kernel<T, VEC, 3>), grid, block, 0, stream, a); return hipGetLastError();
        case 4: hipLaunchKernelGGL((conv_step_kernel<T, VEC, 4>), grid, block, 0, stream, a); return hipGetLastError();
    }
    return hipErrorNotSupported;
}

}  // namespace

// Rows that a wave goes through: 32, in front of (and, for gradients, behind) which W - 1 are read twice; 48 and 60 took 85 and
// 84 us against 82 forward, 60 and 67 against 57 for gradients.  Fewer where that leaves compute units idle.
void conv_runs(int64_t rows, int vecs, int &run, int &runs) {
    const int64_t tiles = (vecs + 63) / 64;
    run = 32;
    while (run > 8 && tiles * ((rows + run - 1) / run) < 2048) run /= 2;
    runs = (int)((rows + run - 1) / run);
}

hipError_t launch_conv_fwd(ConvArgs a, bool fp32, bool wide, hipStream_t stream) { return by_type<FWD>(a, fp32, wide, stream); }

hipError_t launch_conv_bwd(ConvArgs a, bool fp32, bool wide, float *d_weight, float *d_bias, hipStream_t stream) {
    const hipError_t e = by_type<BWD>(a, fp32, wide, stream);
    if (e != hipSuccess || !a.part) return e;
    return launch_column_sums(ColumnSums{a.part, a.runs, (a.W + 1) * a.D, a.D, a.W, d_weight, d_bias}, stream);
}

hipError_t launch_conv_step(ConvStepArgs a, bool fp32, bool wide, hipStream_t stream) {
    a.vecs = wide ? a.D / CONV_STEP_VEC : a.D;
    if (wide) return fp32 ? step_by_taps<float, CONV_STEP_VEC>(a, stream) : step_by_taps<__bf16, CONV_STEP_VEC>(a, stream);
    return fp32 ? step_by_taps<float, 1>(a, stream) : step_by_taps<__bf16, 1>(a, stream);
}

}  // namespace kda
