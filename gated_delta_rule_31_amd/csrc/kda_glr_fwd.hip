// kda_glr_fwd.hip -- the gated linear recurrence over long rows (gfx950), and its decode step.
//
// Bound by memory and the vector units: a number takes 33 instructions, six of them transcendental, in each of the two
// launches that read the rows, and the first has them from memory, the second partly from the last-level cache.  7957 packed
// rows of 4096 channels, bf16, logits and input gate: A and H 52 us (0.2 GB), the pass over the tiles 5, the rows 52 (0.26 GB);
// a large copy takes 52 us for 0.26 GB.  131072 rows of 256 channels, log decays as given: 45, 14 and 42 us.
#include "kda_glr.h"

namespace kda {
namespace {

constexpr int WAVES = 4;

// The rows of a wave's tile, U at a time with the next U on their way.  OUT: out, final and kept states, from the state in
// front of the tile; otherwise the tile's A and H.
template <typename T, int VEC, bool LOGITS, bool NORM, bool GATED, bool OUT>
__global__ __launch_bounds__(64 * WAVES) void glr_fwd_kernel(const GlrArgs a, int blocks) {
    if ((int)blockIdx.x >= blocks) {  // sequences without a row hand on what they got
        const int64_t i = (int64_t)(blockIdx.x - blocks) * blockDim.x + threadIdx.x;
        if (i < (int64_t)a.seqs.N * a.C) {
            const int n = (int)(i / a.C);
            if (a.seqs.cu[n + 1] <= a.seqs.cu[n]) a.sf[i] = a.s0 ? a.s0[i] : 0.f;
        }
        return;
    }
    typedef gate_t<T, LOGITS> Z;
    const int wave = blockIdx.x * WAVES + __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    if (wave >= a.tiles.n * a.tiles.columns) return;
    const GlrPlace p = glr_place<VEC>(a, wave);
    if (!p.there) return;
    const int64_t sx = a.x_stride * sizeof(T), sz = a.gates.gate_stride * sizeof(Z), si = a.gates.in_stride * sizeof(T);
    const char *x = static_cast<const char *>(a.x) + p.t0 * sx, *z = static_cast<const char *>(a.gates.gate) + p.t0 * sz;
    const char *in = static_cast<const char *>(a.gates.in_gate) + p.t0 * si;
    Raw<T, VEC> nx[U], ni[U];
    Raw<Z, VEC> nz[U];
    auto fetch = [&](int r) {
        load_run(nz, z + r * sz, sz, p.c * (uint32_t)sizeof(Z), p.count - r);
        load_run(nx, x + r * sx, sx, p.c * (uint32_t)sizeof(T), p.count - r);
        if constexpr (GATED) load_run(ni, in + r * si, si, p.c * (uint32_t)sizeof(T), p.count - r);
    };
    fetch(0);
    GateConst<VEC, LOGITS> k;
    k.load(a.gates, p.c);
    float A[VEC], h[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) A[i] = 1.f;
    if constexpr (OUT) {
        glr_front<VEC>(h, a, a.tiles.front, p.tile, p.c, false);
    } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i) h[i] = 0.f;
    }
    char *out = static_cast<char *>(a.out) + p.t0 * a.C * sizeof(T);
    float *kept = a.kept + (p.t0 / GLR_KEPT) * a.C + p.c;
    for (int r = 0; r < p.count; r += U) {
        float av[U][VEC], bv[U][VEC];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const Gate g = make_gate<LOGITS, NORM, GATED>(nz[u].get(i), GATED ? ni[u].get(i) : 0.f, k.scale2[i], k.bias2[i], a.gates.lower);
                av[u][i] = g.a;
                bv[u][i] = g.f * g.i * nx[u].get(i);
            }
        if (r + U < p.count) fetch(r + U);
        if (OUT && a.kept) {
            Raw<float, VEC> s;
#pragma unroll
            for (int i = 0; i < VEC; ++i) s.set(i, h[i]);
            s.store(kept + (int64_t)(r / GLR_KEPT) * a.C);
        }
        const uint32_t first = (uint32_t)(p.first >> r) & ((1u << U) - 1), last = (uint32_t)(p.last >> r) & ((1u << U) - 1);
        // HERE: a sequence begins or ends among these rows, or the rows end
        auto rows = [&](auto marked) {
            constexpr bool HERE = decltype(marked)::value;
            const uint32_t ot = here(p.c * (uint32_t)sizeof(T));
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (HERE && r + u >= p.count) continue;
                if (HERE && first >> u & 1) {
#pragma unroll
                    for (int i = 0; i < VEC; ++i) {
                        A[i] = CUT;
                        h[i] = 0.f;
                    }
                    if (a.s0) load_f32<VEC>(h, a.s0 + (int64_t)a.seqs.of(p.t0 + r + u) * a.C + p.c);
                }
                Raw<T, VEC> y;
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    h[i] = fmaf(av[u][i], h[i], bv[u][i]);
                    if constexpr (OUT) y.set(i, h[i]);
                    else A[i] *= av[u][i];
                }
                if constexpr (OUT) {
                    if (a.out && (!HERE || r + u < p.own)) y.store(out + (int64_t)(r + u) * a.C * sizeof(T), ot);
                    if (HERE && a.sf && last >> u & 1) {
                        Raw<float, VEC> s;
#pragma unroll
                        for (int i = 0; i < VEC; ++i) s.set(i, h[i]);
                        s.store(a.sf + (int64_t)a.seqs.of(p.t0 + r + u) * a.C + p.c);
                    }
                }
            }
        };
        if (first | last || r + U > p.own) rows(std::true_type{});
        else rows(std::false_type{});
    }
    if constexpr (!OUT) glr_word<VEC>(a, p.tile, p.c, A, h);
}

// The state in front of every tile: a workgroup takes a few channels, and its groups of lanes a stretch of tiles each: the
// stretch's A and H, joined over the groups of a wave by shuffles and over the waves through LDS, then its tiles from
// the state in front of it.  What it takes is the words' way, so 16 of them are on it at a time (four at a time:
// 22 us for 4096 tiles of 256 channels).  16 channels a workgroup read whole cache lines; where that leaves few
// workgroups, four.
constexpr int CARRY_T = 1024, CARRY_U = 16;
template <int CARRY_C>
__global__ __launch_bounds__(CARRY_T) void glr_carry_kernel(const float *words, float *front, int n, int C, int reverse) {
    __shared__ float sA[CARRY_T / 64][CARRY_C], sH[CARRY_T / 64][CARRY_C];
    const int ch = threadIdx.x % CARRY_C, group = threadIdx.x / CARRY_C, c = blockIdx.x * CARRY_C + ch, lane = threadIdx.x & 63, wave = threadIdx.x / 64;
    const int groups = CARRY_T / CARRY_C, each = (n + groups - 1) / groups, lo = group * each, end = lo + each < n ? lo + each : n, hi = c < C ? end : lo;
    float A = 1.f, H = 0.f, a[CARRY_U], h[CARRY_U];
    auto words_from = [&](int at) {
#pragma unroll
        for (int u = 0; u < CARRY_U; ++u) {
            a[u] = 1.f;
            h[u] = 0.f;
            if (at + u < hi) {
                const float *w = words + ((int64_t)(reverse ? n - 1 - at - u : at + u) * C + c) * 2;
                a[u] = w[0];
                h[u] = w[1];
            }
        }
    };
    for (int at = lo; at < hi; at += CARRY_U) {
        words_from(at);
#pragma unroll
        for (int u = 0; u < CARRY_U; ++u) {
            H = join(a[u], h[u], H);
            A = both(A, a[u]);
        }
    }
#pragma unroll
    for (int d = CARRY_C; d < 64; d *= 2) {
        const float pa = __shfl_up(A, d), ph = __shfl_up(H, d);
        if (lane >= d) {
            H = join(A, H, ph);
            A = both(A, pa);
        }
    }
    if (lane >= 64 - CARRY_C) {
        sA[wave][ch] = A;
        sH[wave][ch] = H;
    }
    float ea = __shfl_up(A, CARRY_C), eh = __shfl_up(H, CARRY_C);
    __syncthreads();
    float x = 0.f;
    for (int w = 0; w < wave; ++w) x = join(sA[w][ch], sH[w][ch], x);
    if (lane >= CARRY_C) x = join(ea, eh, x);
    for (int at = lo; at < hi; at += CARRY_U) {
        if (each > CARRY_U) words_from(at);  // otherwise they are still there
#pragma unroll
        for (int u = 0; u < CARRY_U; ++u)
            if (at + u < hi) {
                front[(int64_t)(reverse ? n - 1 - at - u : at + u) * C + c] = x;
                x = join(a[u], h[u], x);
            }
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

template <bool OUT, typename T, int VEC, bool LOGITS, bool NORM>
hipError_t by_input(GlrArgs &a, hipStream_t stream) {
    const int64_t blocks = (glr_waves(a, VEC) + WAVES - 1) / WAVES;
    const int64_t more = OUT && a.seqs.cu && a.sf ? ((int64_t)a.seqs.N * a.C + 64 * WAVES - 1) / (64 * WAVES) : 0;
    const dim3 grid((unsigned)(blocks + more)), block(64 * WAVES);
    if (a.gates.in_gate) hipLaunchKernelGGL((glr_fwd_kernel<T, VEC, LOGITS, NORM, true, OUT>), grid, block, 0, stream, a, (int)blocks);
    else hipLaunchKernelGGL((glr_fwd_kernel<T, VEC, LOGITS, NORM, false, OUT>), grid, block, 0, stream, a, (int)blocks);
    return hipGetLastError();
}
template <bool OUT, typename T, int VEC>
hipError_t by_gate(GlrArgs &a, hipStream_t stream) {
    if (a.gates.log_scale) return a.gates.normalize ? by_input<OUT, T, VEC, true, true>(a, stream) : by_input<OUT, T, VEC, true, false>(a, stream);
    return a.gates.normalize ? by_input<OUT, T, VEC, false, true>(a, stream) : by_input<OUT, T, VEC, false, false>(a, stream);
}
template <bool OUT>
hipError_t by_type(GlrArgs a, bool fp32, bool wide, hipStream_t stream) {
    if (wide) return fp32 ? by_gate<OUT, float, 2>(a, stream) : by_gate<OUT, __bf16, 2>(a, stream);
    return fp32 ? by_gate<OUT, float, 1>(a, stream) : by_gate<OUT, __bf16, 1>(a, stream);
}

template <typename T, int VEC>
hipError_t step_by_gate(const GlrStepArgs &a, hipStream_t stream) {
    const dim3 grid((unsigned)(a.B * ((a.vecs + 63) / 64))), block(64);
    if (a.gates.log_scale) hipLaunchKernelGGL((glr_step_kernel<T, VEC, true>), grid, block, 0, stream, a);
    else hipLaunchKernelGGL((glr_step_kernel<T, VEC, false>), grid, block, 0, stream, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_glr_carry(const GlrArgs &a, bool reverse, hipStream_t stream) {
    if (!a.tiles.front) return hipSuccess;
    if (a.C <= 1024) hipLaunchKernelGGL(glr_carry_kernel<4>, dim3((unsigned)((a.C + 3) / 4)), dim3(CARRY_T), 0, stream, a.tiles.words, a.tiles.front, a.tiles.n, a.C, reverse ? 1 : 0);
    else hipLaunchKernelGGL(glr_carry_kernel<16>, dim3((unsigned)((a.C + 15) / 16)), dim3(CARRY_T), 0, stream, a.tiles.words, a.tiles.front, a.tiles.n, a.C, reverse ? 1 : 0);
    return hipGetLastError();
}

// Tiles of 64 rows, or shorter ones where those are too few waves to cover their loads: 7957 x 4096 in 108 us with 32 rows
// (8000 waves), 117 with 64, 125 with 16.  Few rows take what a tile's rows take one after another, in each launch: 64 rows of
// 32 channels 10.6 us with tiles of 8, 12.8 with 16, 16.9 in one tile (and one launch); 16 rows 9.9 and, in one tile, 7.2.
void glr_plan(GlrArgs &a) {
    const int64_t columns = (a.C + 127) / 128;
    const int least = a.seqs.rows > 16 ? 8 : 16;
    a.tiles.rows = 64;
    while (a.tiles.rows > least && (a.seqs.rows + a.tiles.rows - 1) / a.tiles.rows * columns < 6000) a.tiles.rows /= 2;
    a.tiles.n = (int)((a.seqs.rows + a.tiles.rows - 1) / a.tiles.rows);
}

void carve_glr_tiles(GlrArgs &a, Pieces &w) {
    const int64_t n = (int64_t)a.tiles.n * a.C;
    w.take(a.tiles.words, a.tiles.n > 1 ? 2 * n : 0);
    w.take(a.tiles.front, a.tiles.n > GLR_FEW ? n : 0);
    if (a.tiles.n <= GLR_FEW) a.tiles.front = nullptr;
}

size_t carve_glr_fwd(GlrArgs &a, void *base) {
    Pieces w{static_cast<char *>(base)};
    glr_plan(a);
    carve_glr_tiles(a, w);
    return w.used;
}

hipError_t launch_glr_fwd(const GlrArgs &a, bool fp32, bool wide, hipStream_t stream) {
    hipError_t e = hipSuccess;
    if (a.tiles.n > 1) e = by_type<false>(a, fp32, wide, stream);
    if (e == hipSuccess) e = launch_glr_carry(a, false, stream);
    return e == hipSuccess ? by_type<true>(a, fp32, wide, stream) : e;
}

hipError_t launch_glr_step(GlrStepArgs a, bool fp32, bool wide, hipStream_t stream) {
    a.vecs = wide ? a.C / 2 : a.C;
    if (wide) return fp32 ? step_by_gate<float, 2>(a, stream) : step_by_gate<__bf16, 2>(a, stream);
    return fp32 ? step_by_gate<float, 1>(a, stream) : step_by_gate<__bf16, 1>(a, stream);
}

}  // namespace kda
