// kda_glr_bwd.hip -- gradients of the gated linear recurrence (gfx950).
//
// With lambda_t the gradient of h_t and m_t = a_t lambda_t that of h_{t-1}:
//   lambda_t = d out_t + m_{t+1}   (behind a sequence's last row: the gradient of its final state)
//   dx = lambda f i,   di_t = lambda f x i (1 - i),   dg = a lambda h_{t-1} - lambda i x a^2 / f
// (the second term where f = sqrt(1 - a^2), 0 where f is), and through the bounded gate
// du = dg lower p (1 - p), dz = e^A du, d bias = sum dz, d log_scale = sum u du.
// m is a recurrence from the right with the same decays: a stretch of rows maps the m behind it to the
// one in front as m -> A m + Q, and one pass takes the tiles from the last to the first (kda_glr.h). A
// tile's own states come from the one that the forward kept in front of it.
#include "kda_glr.h"

namespace kda {
namespace {

constexpr int WAVES = 8, L = 8, ROWS = WAVES * L;
static_assert(ROWS == GLR_KEPT, "a tile begins where a state is kept");

template <typename T, int VEC, bool LOGITS, bool NORM, bool GATED>
__global__ __launch_bounds__(64 * WAVES, 2) void glr_bwd_kernel(const GlrArgs a, int blocks) {
    if ((int)blockIdx.x >= blocks) {  // the gradient of a sequence without a row is that of what it handed on
        const int64_t i = (int64_t)(blockIdx.x - blocks) * blockDim.x + threadIdx.x;
        if (i < (int64_t)a.seqs.N * a.C) {
            const int n = (int)(i / a.C);
            if (a.seqs.cu[n + 1] <= a.seqs.cu[n]) a.ds0[i] = a.d_sf ? a.d_sf[i] : 0.f;
        }
        return;
    }
    __shared__ LookBack<VEC, WAVES> lds;
    __shared__ float sA[WAVES][64][VEC], sH[WAVES][64][VEC];
    typedef gate_t<T, LOGITS> Z;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), lane = threadIdx.x & 63;
    const bool alone = a.look.n == 1;
    const int ticket = alone ? (int)blockIdx.x : lds.take(a.look.ticket);
    const int turn = ticket / a.look.columns, tile = a.look.n - 1 - turn, column = ticket % a.look.columns;
    const int c = (column * 64 + lane) * VEC, cc = c < a.C ? c : 0;
    const bool there = c < a.C;
    const int64_t t0 = (int64_t)tile * ROWS + wave * L, limit = a.seqs.limit();
    const int rows = (int)(a.seqs.rows - t0 < 0 ? 0 : a.seqs.rows - t0 < L ? a.seqs.rows - t0 : L);
    const int count = (int)(limit - t0 < 0 ? 0 : limit - t0 < L ? limit - t0 : L);
    uint64_t first = 0, last = 0;
    GateConst<VEC, LOGITS> k;
    Raw<T, VEC> rx[L], ri[L], rd[L];
    Raw<Z, VEC> rz[L];
    // decay; input, then the state in front; f i; i; a^2 / f^2; p (1 - p)
    float av[L][VEC], bv[L][VEC], fi[L][VEC], iv[L][VEC], wv[L][VEC], pq[L][VEC];
    float A[VEC], H[VEC], B[VEC], Q[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
        A[i] = B[i] = 1.f;
        H[i] = Q[i] = 0.f;
    }
    // the state in front of a sequence's first row, what comes back behind its last
    auto front = [&](float(&h)[VEC], int u) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) h[i] = 0.f;
        if (a.s0) load_f32<VEC>(h, a.s0 + (int64_t)a.seqs.of(t0 + u) * a.C + cc);
    };
    auto back = [&](float(&m)[VEC], int u) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) m[i] = 0.f;
        if (a.d_sf) load_f32<VEC>(m, a.d_sf + (int64_t)a.seqs.of(t0 + u) * a.C + cc);
    };
    if (count > 0) {
        a.seqs.marks(t0, count, first, last);
        const T *x = static_cast<const T *>(a.x) + t0 * a.x_stride, *in = static_cast<const T *>(a.gates.in_gate) + t0 * a.gates.in_stride;
        const T *d = static_cast<const T *>(a.d_out) + t0 * a.C;
        const Z *z = static_cast<const Z *>(a.gates.gate) + t0 * a.gates.gate_stride;
#pragma unroll
        for (int u = 0; u < L; ++u) {
            const int64_t at = u < count ? u : count - 1;
            rz[u].load(z + at * a.gates.gate_stride + cc);
            rx[u].load(x + at * a.x_stride + cc);
            if constexpr (GATED) ri[u].load(in + at * a.gates.in_stride + cc);
            else ri[u].zero();
            rd[u].load(d + at * a.C + cc);
        }
        k.load(a.gates, cc);
#pragma unroll
        for (int u = 0; u < L; ++u) {
            if (first >> u & 1) {
                front(H, u);
#pragma unroll
                for (int i = 0; i < VEC; ++i) A[i] = 0.f;
            }
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const Gate g = make_gate<LOGITS, NORM, GATED>(rz[u].get(i), ri[u].get(i), k.scale2[i], k.bias2[i], a.gates.lower);
                const bool is = u < count;  // rows behind the end leave everything as it is
                av[u][i] = is ? g.a : 1.f;
                fi[u][i] = g.f * g.i;
                iv[u][i] = g.i;
                pq[u][i] = g.p * g.q;
                if constexpr (NORM) wv[u][i] = g.f > 0.f ? g.a * g.a * __builtin_amdgcn_rcpf(g.f * g.f) : 0.f;
                bv[u][i] = is ? fi[u][i] * rx[u].get(i) : 0.f;
                A[i] *= av[u][i];
                H[i] = fmaf(av[u][i], H[i], bv[u][i]);
            }
        }
#pragma unroll
        for (int u = L - 1; u >= 0; --u) {
            if (last >> u & 1) {
                back(Q, u);
#pragma unroll
                for (int i = 0; i < VEC; ++i) B[i] = 0.f;
            }
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                B[i] *= av[u][i];
                Q[i] = u < count ? av[u][i] * (rd[u].get(i) + Q[i]) : Q[i];
            }
        }
    }
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
        sA[wave][lane][i] = A[i];
        sH[wave][lane][i] = H[i];
        lds.A[WAVES - 1 - wave][lane][i] = B[i];
        lds.H[WAVES - 1 - wave][lane][i] = Q[i];
    }
    __syncthreads();
    if (!alone) lds.front(a.look, a.C, turn, column, cc, there, wave, lane);
    float dz_sum[VEC] = {}, u_sum[VEC] = {};
    T *dx = static_cast<T *>(a.dx) + t0 * a.C, *di = static_cast<T *>(a.d_in) + t0 * a.C;
    Z *dz = static_cast<Z *>(a.d_gate) + t0 * a.C;
    if (there && count > 0) {
        float h[VEC], m[VEC];
        load_f32<VEC>(h, a.kept + (int64_t)tile * a.C + c);
        for (int w = 0; w < wave; ++w)
#pragma unroll
            for (int i = 0; i < VEC; ++i) h[i] = join(sA[w][lane][i], sH[w][lane][i], h[i]);
        lds.state(m, WAVES - 1 - wave, lane, alone);
#pragma unroll
        for (int u = 0; u < L; ++u) {
            if (first >> u & 1) front(h, u);
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const float next = fmaf(av[u][i], h[i], bv[u][i]);
                bv[u][i] = h[i];
                h[i] = next;
            }
        }
#pragma unroll
        for (int u = L - 1; u >= 0; --u) {
            if (u < count) {
                if (last >> u & 1) back(m, u);
                Raw<T, VEC> ox, oi;
                Raw<Z, VEC> oz;
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    const float lam = rd[u].get(i) + m[i];
                    m[i] = av[u][i] * lam;
                    const float v = lam * fi[u][i], b = v * rx[u].get(i);
                    ox.set(i, v);
                    if constexpr (GATED) oi.set(i, fmaf(-b, iv[u][i], b));
                    float dg = m[i] * bv[u][i];
                    if constexpr (NORM) dg = fmaf(-b, wv[u][i], dg);
                    if constexpr (LOGITS) {
                        const float du = dg * a.gates.lower * pq[u][i], t = (k.scale2[i] * (1.f / LOG2E)) * du;
                        u_sum[i] = fmaf(fmaf(k.scale2[i], rz[u].get(i), k.bias2[i]), du, u_sum[i]);
                        dz_sum[i] += t;
                        oz.set(i, t);
                    } else {
                        oz.set(i, dg);
                    }
                }
                ox.store(dx + (int64_t)u * a.C + c);
                oz.store(dz + (int64_t)u * a.C + c);
                if constexpr (GATED) oi.store(di + (int64_t)u * a.C + c);
                if (a.ds0 && first >> u & 1) {
                    Raw<float, VEC> s;
#pragma unroll
                    for (int i = 0; i < VEC; ++i) s.set(i, m[i]);
                    s.store(a.ds0 + (int64_t)a.seqs.of(t0 + u) * a.C + c);
                }
            }
        }
    }
    if (there) {  // rows behind the last sequence
        Raw<T, VEC> ox;
        Raw<Z, VEC> oz;
        ox.zero();
        oz.zero();
        for (int u = count; u < rows; ++u) {
            ox.store(dx + (int64_t)u * a.C + c);
            oz.store(dz + (int64_t)u * a.C + c);
            if constexpr (GATED) ox.store(di + (int64_t)u * a.C + c);
        }
    }
    if constexpr (LOGITS) {
        if (!a.part) return;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            sA[wave][lane][i] = dz_sum[i];
            sH[wave][lane][i] = u_sum[i] * (1.f / LOG2E);
        }
        __syncthreads();
        if (wave || !there) return;
        float *part = a.part + (int64_t)tile * 2 * a.C + c;
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            float x = 0.f, y = 0.f;
            for (int w = 0; w < WAVES; ++w) {
                x += sA[w][lane][i];
                y += sH[w][lane][i];
            }
            part[i] = x;
            part[a.C + i] = y;
        }
    }
}

// d log_scale[h] = the sum over the head's channels
__global__ __launch_bounds__(64) void head_sums_kernel(const float *x, int K, float *out) {
    float s = 0.f;
    for (int i = threadIdx.x; i < K; i += 64) s += x[(int64_t)blockIdx.x * K + i];
    for (int d = 32; d > 0; d /= 2) s += __shfl_xor(s, d);
    if (threadIdx.x == 0) out[blockIdx.x] = s;
}

template <typename T, int VEC, bool LOGITS, bool NORM>
hipError_t by_input(const GlrArgs &a, hipStream_t stream) {
    const int64_t blocks = (int64_t)a.look.n * a.look.columns;
    const int64_t more = a.seqs.cu && a.ds0 ? ((int64_t)a.seqs.N * a.C + 64 * WAVES - 1) / (64 * WAVES) : 0;
    const dim3 grid((unsigned)(blocks + more)), block(64 * WAVES);
    if (a.gates.in_gate) hipLaunchKernelGGL((glr_bwd_kernel<T, VEC, LOGITS, NORM, true>), grid, block, 0, stream, a, (int)blocks);
    else hipLaunchKernelGGL((glr_bwd_kernel<T, VEC, LOGITS, NORM, false>), grid, block, 0, stream, a, (int)blocks);
    return hipGetLastError();
}
template <typename T, int VEC>
hipError_t by_gate(GlrArgs a, hipStream_t stream) {
    const hipError_t e = launch_glr_begin(a.look, (a.C + 64 * VEC - 1) / (64 * VEC), stream);
    if (e != hipSuccess) return e;
    if (a.gates.log_scale) return a.gates.normalize ? by_input<T, VEC, true, true>(a, stream) : by_input<T, VEC, true, false>(a, stream);
    return a.gates.normalize ? by_input<T, VEC, false, true>(a, stream) : by_input<T, VEC, false, false>(a, stream);
}

}  // namespace

// The workspace: the tiles' words, partial sums and their sums, and the states in front of the tiles, with the forward's
// own workspace, where the caller has not kept them.
size_t carve_glr_bwd(GlrArgs &a, void *base, bool kept, float *&sums, void *&more) {
    Pieces w{static_cast<char *>(base)};
    glr_plan(a.look, a.seqs.rows, ROWS);
    carve_glr_look(a.look, w, a.C);
    const int64_t n = (int64_t)a.look.n * a.C;
    w.take(a.part, a.gates.log_scale ? 2 * n : 0);
    w.take(sums, a.gates.log_scale ? a.C : 0);
    more = nullptr;
    if (!kept) {
        w.take(a.kept, n);
        GlrArgs f{};
        f.seqs = a.seqs;
        f.C = a.C;
        char *at;
        w.take(at, (int64_t)carve_glr_fwd(f, nullptr));
        more = at;
    }
    return w.used;
}

hipError_t launch_glr_bwd(const GlrArgs &a, bool fp32, bool wide, float *sums, void *more, float *d_log_scale, float *d_bias, hipStream_t stream) {
    hipError_t e = hipSuccess;
    if (more) {  // the states that were not kept
        GlrArgs f = a;
        f.out = nullptr;
        f.sf = nullptr;
        carve_glr_fwd(f, more);
        e = launch_glr_fwd(f, fp32, wide, stream);
        if (e != hipSuccess) return e;
    }
    if (wide) e = fp32 ? by_gate<float, 2>(a, stream) : by_gate<__bf16, 2>(a, stream);
    else e = fp32 ? by_gate<float, 1>(a, stream) : by_gate<__bf16, 1>(a, stream);
    if (e != hipSuccess || !a.part) return e;
    e = launch_column_sums(ColumnSums{a.part, a.look.n, 2 * a.C, a.C, 1, d_bias, sums}, stream);
    if (e != hipSuccess || !d_log_scale) return e;
    hipLaunchKernelGGL(head_sums_kernel, dim3((unsigned)(a.C / a.gates.K)), dim3(64), 0, stream, sums, a.gates.K, d_log_scale);
    return hipGetLastError();
}

}  // namespace kda
