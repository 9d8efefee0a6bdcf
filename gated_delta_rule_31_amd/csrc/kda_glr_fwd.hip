// kda_glr_fwd.hip -- the gated linear recurrence over long rows (gfx950), and its decode step.
//
// One pass (kda_glr.h): a workgroup of eight waves, 16 rows each, for 64 VEC channels holds its rows' decays
// and inputs in registers while the state in front of them is found.
#include "kda_glr.h"

namespace kda {
namespace {

constexpr int WAVES = 8, L = 16, ROWS = WAVES * L;

template <typename T, int VEC, bool LOGITS, bool NORM, bool GATED>
__global__ __launch_bounds__(64 * WAVES, 4) void glr_fwd_kernel(const GlrArgs a, int blocks) {
    if ((int)blockIdx.x >= blocks) {  // sequences without a row hand on what they got
        const int64_t i = (int64_t)(blockIdx.x - blocks) * blockDim.x + threadIdx.x;
        if (i < (int64_t)a.seqs.N * a.C) {
            const int n = (int)(i / a.C);
            if (a.seqs.cu[n + 1] <= a.seqs.cu[n]) a.sf[i] = a.s0 ? a.s0[i] : 0.f;
        }
        return;
    }
    __shared__ LookBack<VEC, WAVES> lds;
    typedef gate_t<T, LOGITS> Z;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), lane = threadIdx.x & 63;
    const bool alone = a.look.n == 1;
    const int ticket = alone ? (int)blockIdx.x : lds.take(a.look.ticket);
    const int tile = ticket / a.look.columns, column = ticket % a.look.columns;
    const int c = (column * 64 + lane) * VEC, cc = c < a.C ? c : 0;
    const bool there = c < a.C;
    const int64_t t0 = (int64_t)tile * ROWS + wave * L, limit = a.seqs.limit();
    const int count = (int)(a.seqs.rows - t0 < 0 ? 0 : a.seqs.rows - t0 < L ? a.seqs.rows - t0 : L);
    uint64_t first = 0, last = 0;
    float av[L][VEC], bv[L][VEC], A[VEC], H[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
        A[i] = 1.f;
        H[i] = 0.f;
    }
    if (count > 0) {
        a.seqs.marks(t0, count, first, last);
        const T *x = static_cast<const T *>(a.x) + t0 * a.x_stride, *in = static_cast<const T *>(a.gates.in_gate) + t0 * a.gates.in_stride;
        const Z *z = static_cast<const Z *>(a.gates.gate) + t0 * a.gates.gate_stride;
        Raw<T, VEC> rx[L], ri[L];
        Raw<Z, VEC> rz[L];
#pragma unroll
        for (int u = 0; u < L; ++u) {
            const int64_t at = u < count ? u : count - 1;
            rz[u].load(z + at * a.gates.gate_stride + cc);
            rx[u].load(x + at * a.x_stride + cc);
            if constexpr (GATED) ri[u].load(in + at * a.gates.in_stride + cc);
            else ri[u].zero();
        }
        GateConst<VEC, LOGITS> k;
        k.load(a.gates, cc);
#pragma unroll
        for (int u = 0; u < L; ++u) {
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const Gate g = make_gate<LOGITS, NORM, GATED>(rz[u].get(i), ri[u].get(i), k.scale2[i], k.bias2[i], a.gates.lower);
                av[u][i] = u < count ? g.a : 1.f;  // rows behind the end leave the state as it is
                bv[u][i] = u < count ? g.f * g.i * rx[u].get(i) : 0.f;
            }
            if (first >> u & 1) {  // the state in front of it is the sequence's own
                float s0[VEC] = {};
                if (a.s0) load_f32<VEC>(s0, a.s0 + (int64_t)a.seqs.of(t0 + u) * a.C + cc);
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
        lds.A[wave][lane][i] = A[i];
        lds.H[wave][lane][i] = H[i];
    }
    __syncthreads();
    if (!alone) lds.front(a.look, a.C, tile, column, cc, there, wave, lane);
    if (!there || count <= 0) return;
    float h[VEC];
    lds.state(h, wave, lane, alone);
    if (a.kept && t0 % GLR_KEPT == 0) {
        Raw<float, VEC> s;
#pragma unroll
        for (int i = 0; i < VEC; ++i) s.set(i, h[i]);
        s.store(a.kept + t0 / GLR_KEPT * a.C + c);
    }
    if (!a.out) return;
    T *out = static_cast<T *>(a.out) + t0 * a.C;
#pragma unroll
    for (int u = 0; u < L; ++u) {
        if (first >> u & 1)
#pragma unroll
            for (int i = 0; i < VEC; ++i) h[i] = 0.f;
        Raw<T, VEC> y;
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            h[i] = fmaf(av[u][i], h[i], bv[u][i]);
            y.set(i, h[i]);
        }
        if (t0 + u < limit) y.store(out + (int64_t)u * a.C + c);
        if (a.sf && last >> u & 1) {
            Raw<float, VEC> s;
#pragma unroll
            for (int i = 0; i < VEC; ++i) s.set(i, h[i]);
            s.store(a.sf + (int64_t)a.seqs.of(t0 + u) * a.C + c);
        }
    }
}

__global__ __launch_bounds__(256) void glr_clear_kernel(uint32_t *p, int64_t n) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i < n) p[i] = 0;
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

template <typename T, int VEC, bool LOGITS, bool NORM>
hipError_t by_input(const GlrArgs &a, hipStream_t stream) {
    const int64_t blocks = (int64_t)a.look.n * a.look.columns;
    const int64_t more = a.seqs.cu && a.sf ? ((int64_t)a.seqs.N * a.C + 64 * WAVES - 1) / (64 * WAVES) : 0;
    const dim3 grid((unsigned)(blocks + more)), block(64 * WAVES);
    if (a.gates.in_gate) hipLaunchKernelGGL((glr_fwd_kernel<T, VEC, LOGITS, NORM, true>), grid, block, 0, stream, a, (int)blocks);
    else hipLaunchKernelGGL((glr_fwd_kernel<T, VEC, LOGITS, NORM, false>), grid, block, 0, stream, a, (int)blocks);
    return hipGetLastError();
}
template <typename T, int VEC>
hipError_t by_gate(GlrArgs a, hipStream_t stream) {
    const hipError_t e = launch_glr_begin(a.look, (a.C + 64 * VEC - 1) / (64 * VEC), stream);
    if (e != hipSuccess) return e;
    if (a.gates.log_scale) return a.gates.normalize ? by_input<T, VEC, true, true>(a, stream) : by_input<T, VEC, true, false>(a, stream);
    return a.gates.normalize ? by_input<T, VEC, false, true>(a, stream) : by_input<T, VEC, false, false>(a, stream);
}

template <typename T, int VEC>
hipError_t step_by_gate(const GlrStepArgs &a, hipStream_t stream) {
    const dim3 grid((unsigned)(a.B * ((a.vecs + 63) / 64))), block(64);
    if (a.gates.log_scale) hipLaunchKernelGGL((glr_step_kernel<T, VEC, true>), grid, block, 0, stream, a);
    else hipLaunchKernelGGL((glr_step_kernel<T, VEC, false>), grid, block, 0, stream, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_glr_begin(GlrLook &g, int columns, hipStream_t stream) {
    g.columns = columns;
    g.group_there = g.tile_there + (int64_t)g.n * columns;
    if (g.n == 1) return hipSuccess;
    const int64_t n = g.words();
    hipLaunchKernelGGL(glr_clear_kernel, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, stream, g.ticket, n);
    return hipGetLastError();
}

// Groups of about the root of half the tiles: a tile looks at up to `group` tiles with one wave, and at the groups in
// front with seven.
void glr_plan(GlrLook &g, int64_t rows, int tile_rows) {
    g.n = (int)((rows + tile_rows - 1) / tile_rows);
    g.group = 4;
    while ((int64_t)g.group * g.group * 2 < g.n) g.group *= 2;
}

void carve_glr_look(GlrLook &g, Pieces &w, int C) {
    g.columns = (C + 63) / 64;  // the most there are
    w.take(g.ticket, g.words());
    g.tile_there = g.ticket ? g.ticket + 1 : nullptr;
    w.take(g.tile, (int64_t)g.n * C);
    w.take(g.whole, (int64_t)g.groups() * C);
}

size_t carve_glr_fwd(GlrArgs &a, void *base) {
    Pieces w{static_cast<char *>(base)};
    glr_plan(a.look, a.seqs.rows, ROWS);
    carve_glr_look(a.look, w, a.C);
    return w.used;
}

hipError_t launch_glr_fwd(const GlrArgs &a, bool fp32, bool wide, hipStream_t stream) {
    if (wide) return fp32 ? by_gate<float, 2>(a, stream) : by_gate<__bf16, 2>(a, stream);
    return fp32 ? by_gate<float, 1>(a, stream) : by_gate<__bf16, 1>(a, stream);
}

hipError_t launch_glr_step(GlrStepArgs a, bool fp32, bool wide, hipStream_t stream) {
    a.vecs = wide ? a.C / 2 : a.C;
    if (wide) return fp32 ? step_by_gate<float, 2>(a, stream) : step_by_gate<__bf16, 2>(a, stream);
    return fp32 ? step_by_gate<float, 1>(a, stream) : step_by_gate<__bf16, 1>(a, stream);
}

}  // namespace kda
