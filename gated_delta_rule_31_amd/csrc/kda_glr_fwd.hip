// kda_glr_fwd.hip -- the gated linear recurrence over long rows (gfx950), and its decode step.
//
// Three launches: every tile of 64 rows gives its A and H, one pass over the tiles carries the
// state through them, and every tile goes through its rows from the state in front of it.  A
// workgroup is four waves of 16 rows each for 64 VEC channels.
#include "kda_glr.h"

namespace kda {
namespace {

constexpr int WAVES = 4, L = GLR_TILE / WAVES;

template <typename T, int VEC, bool LOGITS, bool NORM, bool GATED, int MODE>
__global__ __launch_bounds__(64 * WAVES) void glr_fwd_kernel(const GlrArgs a, int blocks) {
    constexpr int U = VEC == 1 ? 1 : VEC;
    if ((int)blockIdx.x >= blocks) {  // sequences without a row hand on what they got
        const int64_t i = (int64_t)(blockIdx.x - blocks) * blockDim.x + threadIdx.x;
        if (i < (int64_t)a.seqs.N * a.C) {
            const int n = (int)(i / a.C);
            if (a.seqs.cu[n + 1] <= a.seqs.cu[n]) a.sf[i] = a.s0 ? a.s0[i] : 0.f;
        }
        return;
    }
    __shared__ float sA[WAVES][64][U], sH[WAVES][64][U];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), lane = threadIdx.x & 63;
    const int ctiles = (a.C + 64 * VEC - 1) / (64 * VEC), tile = blockIdx.x / ctiles, c = (blockIdx.x % ctiles * 64 + lane) * VEC;
    const bool there = c < a.C;
    const int64_t t0 = (int64_t)tile * GLR_TILE + wave * L, limit = a.seqs.limit();
    const int count = (int)(a.seqs.rows - t0 < 0 ? 0 : a.seqs.rows - t0 < L ? a.seqs.rows - t0 : L);
    uint64_t first, last;
    a.seqs.marks(t0, count, first, last);
    float av[L][VEC], bv[L][VEC], A[VEC], H[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
        A[i] = 1.f;
        H[i] = 0.f;
    }
    if (there && count > 0) {
        GateConst<VEC, LOGITS> k;
        k.load(a.gates, c);
        const T *x = static_cast<const T *>(a.x) + t0 * a.x_stride + c, *in = static_cast<const T *>(a.gates.in_gate) + t0 * a.gates.in_stride + c;
        const gate_t<T, LOGITS> *z = static_cast<const gate_t<T, LOGITS> *>(a.gates.gate) + t0 * a.gates.gate_stride + c;
#pragma unroll
        for (int u = 0; u < L; ++u) {
            const int64_t at = u < count ? u : count - 1;
            Raw<T, VEC> rx, ri;
            Raw<gate_t<T, LOGITS>, VEC> rz;
            rx.load(x + at * a.x_stride);
            rz.load(z + at * a.gates.gate_stride);
            if constexpr (GATED) ri.load(in + at * a.gates.in_stride);
            else ri.zero();
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const Gate g = make_gate<LOGITS, NORM, GATED>(rz.get(i), ri.get(i), k.scale2[i], k.bias2[i], a.gates.lower);
                av[u][i] = g.a;
                bv[u][i] = g.f * g.i * rx.get(i);
            }
        }
#pragma unroll
        for (int u = 0; u < L; ++u) {
            if (u >= count) break;
            if (first >> u & 1) {
                float s0[VEC] = {};
                if (a.s0) load_f32<VEC>(s0, a.s0 + (int64_t)a.seqs.of(t0 + u) * a.C + c);
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    bv[u][i] = fmaf(av[u][i], s0[i], bv[u][i]);
                    av[u][i] = A[i] = H[i] = 0.f;
                }
            }
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                A[i] *= av[u][i];
                H[i] = fmaf(av[u][i], H[i], bv[u][i]);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
        sA[wave][lane][i] = A[i];
        sH[wave][lane][i] = H[i];
    }
    __syncthreads();
    if (!there) return;
    if constexpr (MODE == GLR_AGGREGATE) {
        if (wave) return;
        float *agg = a.agg + (int64_t)tile * 2 * a.C + c;
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            for (int w = 1; w < WAVES; ++w) {
                H[i] = join(sA[w][lane][i], sH[w][lane][i], H[i]);
                A[i] *= sA[w][lane][i];
            }
            agg[i] = A[i];
            agg[a.C + i] = H[i];
        }
    } else {
        float h[VEC];
        load_f32<VEC>(h, a.kept + (int64_t)tile * a.C + c);
        for (int w = 0; w < wave; ++w)
#pragma unroll
            for (int i = 0; i < VEC; ++i) h[i] = join(sA[w][lane][i], sH[w][lane][i], h[i]);
        T *out = static_cast<T *>(a.out) + t0 * a.C + c;
#pragma unroll
        for (int u = 0; u < L; ++u) {
            if (u >= count) break;
            if (first >> u & 1)
#pragma unroll
                for (int i = 0; i < VEC; ++i) h[i] = 0.f;
            Raw<T, VEC> y;
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                h[i] = fmaf(av[u][i], h[i], bv[u][i]);
                y.set(i, h[i]);
            }
            if (t0 + u < limit) y.store(out + (int64_t)u * a.C);
            if (a.sf && last >> u & 1) {
                float *sf = a.sf + (int64_t)a.seqs.of(t0 + u) * a.C + c;
#pragma unroll
                for (int i = 0; i < VEC; ++i) sf[i] = h[i];
            }
        }
    }
}

__global__ __launch_bounds__(64) void glr_carry_kernel(const float *agg, float *kept, int tiles, int C, int reverse) {
    const int c = blockIdx.x * 64 + threadIdx.x;
    if (c >= C) return;
    float h = 0.f;
    for (int j = 0; j < tiles; ++j) {
        const int64_t t = reverse ? tiles - 1 - j : j;
        kept[t * C + c] = h;
        h = join(agg[t * 2 * C + c], agg[t * 2 * C + C + c], h);
    }
}

template <typename T, int VEC, bool LOGITS>
__global__ __launch_bounds__(64) void glr_step_kernel(const GlrStepArgs a) {
    const int tiles = (a.vecs + 63) / 64, b = blockIdx.x / tiles, v = blockIdx.x % tiles * 64 + threadIdx.x, c = v * VEC;
    const int len = a.slots.tokens(b);
    if (v >= a.vecs || len == 0) return;
    GateConst<VEC, LOGITS> k;
    k.load(a.gates, c);
    const int64_t at = (int64_t)b * a.S * a.C + c;
    const T *x = static_cast<const T *>(a.x) + at, *in = static_cast<const T *>(a.gates.in_gate) + at;
    const gate_t<T, LOGITS> *z = static_cast<const gate_t<T, LOGITS> *>(a.gates.gate) + at;
    T *out = static_cast<T *>(a.out) + at;
    float h[VEC] = {};
    const int64_t from = a.slots.from(b);
    if (from >= 0) load_f32<VEC>(h, a.states + from * a.C + c);
    for (int t = 0; t < len; ++t) {
        const int64_t to = a.slots.to(b, t, len);
        Raw<T, VEC> rx, ri, y;
        Raw<gate_t<T, LOGITS>, VEC> rz;
        rx.load(x + (int64_t)t * a.C);
        rz.load(z + (int64_t)t * a.C);
        ri.zero();
        if (a.gates.in_gate) ri.load(in + (int64_t)t * a.C);
        Raw<float, VEC> s;
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            const Gate g = make_gate<LOGITS, true, true>(rz.get(i), ri.get(i), k.scale2[i], k.bias2[i], a.gates.lower);
            const float f = a.gates.normalize ? g.f : 1.f, in = a.gates.in_gate ? g.i : 1.f;
            h[i] = fmaf(g.a, h[i], f * in * rx.get(i));
            y.set(i, h[i]);
            s.set(i, h[i]);
        }
        y.store(out + (int64_t)t * a.C);
        if (to >= 0) s.store(a.states + to * a.C + c);
    }
}

template <typename T, int VEC, int MODE, bool LOGITS, bool NORM>
hipError_t by_input(const GlrArgs &a, hipStream_t stream) {
    const int64_t blocks = (int64_t)((a.C + 64 * VEC - 1) / (64 * VEC)) * a.tiles;
    const int64_t more = MODE == GLR_APPLY && a.seqs.cu && a.sf ? ((int64_t)a.seqs.N * a.C + 64 * WAVES - 1) / (64 * WAVES) : 0;
    const dim3 grid((unsigned)(blocks + more)), block(64 * WAVES);
    if (a.gates.in_gate) hipLaunchKernelGGL((glr_fwd_kernel<T, VEC, LOGITS, NORM, true, MODE>), grid, block, 0, stream, a, (int)blocks);
    else hipLaunchKernelGGL((glr_fwd_kernel<T, VEC, LOGITS, NORM, false, MODE>), grid, block, 0, stream, a, (int)blocks);
    return hipGetLastError();
}
template <typename T, int VEC, int MODE>
hipError_t by_gate(const GlrArgs &a, hipStream_t stream) {
    if (a.gates.log_scale) return a.gates.normalize ? by_input<T, VEC, MODE, true, true>(a, stream) : by_input<T, VEC, MODE, true, false>(a, stream);
    return a.gates.normalize ? by_input<T, VEC, MODE, false, true>(a, stream) : by_input<T, VEC, MODE, false, false>(a, stream);
}
template <int MODE>
hipError_t by_type(const GlrArgs &a, bool fp32, bool wide, hipStream_t stream) {
    if (wide) return fp32 ? by_gate<float, 4, MODE>(a, stream) : by_gate<__bf16, 4, MODE>(a, stream);
    return fp32 ? by_gate<float, 1, MODE>(a, stream) : by_gate<__bf16, 1, MODE>(a, stream);
}

template <typename T, int VEC>
hipError_t step_by_gate(const GlrStepArgs &a, hipStream_t stream) {
    const dim3 grid((unsigned)(a.B * ((a.vecs + 63) / 64))), block(64);
    if (a.gates.log_scale) hipLaunchKernelGGL((glr_step_kernel<T, VEC, true>), grid, block, 0, stream, a);
    else hipLaunchKernelGGL((glr_step_kernel<T, VEC, false>), grid, block, 0, stream, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_glr_carry(const float *agg, float *kept, int tiles, int C, bool reverse, hipStream_t stream) {
    hipLaunchKernelGGL(glr_carry_kernel, dim3((unsigned)((C + 63) / 64)), dim3(64), 0, stream, agg, kept, tiles, C, reverse ? 1 : 0);
    return hipGetLastError();
}

hipError_t launch_glr_tiles(const GlrArgs &a, bool fp32, bool wide, int mode, hipStream_t stream) {
    return mode == GLR_AGGREGATE ? by_type<GLR_AGGREGATE>(a, fp32, wide, stream) : by_type<GLR_APPLY>(a, fp32, wide, stream);
}

size_t carve_glr_fwd(GlrArgs &a, void *base) {
    Pieces w{static_cast<char *>(base)};
    w.take(a.agg, (int64_t)a.tiles * 2 * a.C);
    float *kept;
    w.take(kept, (int64_t)a.tiles * a.C);
    if (!a.kept) a.kept = kept;
    return w.used;
}

hipError_t launch_glr_states(const GlrArgs &a, bool fp32, bool wide, hipStream_t stream) {
    const hipError_t e = launch_glr_tiles(a, fp32, wide, GLR_AGGREGATE, stream);
    return e == hipSuccess ? launch_glr_carry(a.agg, a.kept, a.tiles, a.C, false, stream) : e;
}

hipError_t launch_glr_fwd(const GlrArgs &a, bool fp32, bool wide, hipStream_t stream) {
    const hipError_t e = launch_glr_states(a, fp32, wide, stream);
    return e == hipSuccess ? launch_glr_tiles(a, fp32, wide, GLR_APPLY, stream) : e;
}

hipError_t launch_glr_step(GlrStepArgs a, bool fp32, bool wide, hipStream_t stream) {
    a.vecs = wide ? a.C / 4 : a.C;
    if (wide) return fp32 ? step_by_gate<float, 4>(a, stream) : step_by_gate<__bf16, 4>(a, stream);
    return fp32 ? step_by_gate<float, 1>(a, stream) : step_by_gate<__bf16, 1>(a, stream);
}

}  // namespace kda
