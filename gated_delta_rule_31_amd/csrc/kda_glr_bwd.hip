// kda_glr_bwd.hip -- gradients of the gated linear recurrence (gfx950).
//
// With lambda_t the gradient of h_t and m_t = a_t lambda_t that of h_{t-1}:
//   lambda_t = d out_t + m_{t+1}   (behind a sequence's last row: the gradient of its final state)
//   dx = lambda f i,   di_t = lambda f x i (1 - i),   dg = a lambda h_{t-1} - lambda i x a^2 / f
// (the second term where f = sqrt(1 - a^2), 0 where f is), and through the bounded gate
// du = dg lower p (1 - p), dz = e^A du, d bias = sum dz, d log_scale = sum u du.
// m is a recurrence from the right with the same decays, so a tile of rows maps the m behind it
// to the one in front as m -> A m + Q.  The tiles' A and Q, a pass over the tiles, and then every tile
// by itself: its states again from the one kept in front of it, its m, and the gradients.
#include "kda_glr.h"

namespace kda {
namespace {

constexpr int WAVES = 8, L = GLR_TILE / WAVES;

// A and Q of every tile
template <typename T, int VEC, bool LOGITS>
__global__ __launch_bounds__(64 * WAVES) void glr_back_kernel(const GlrArgs a) {
    __shared__ float sA[WAVES][64][VEC], sQ[WAVES][64][VEC];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), lane = threadIdx.x & 63;
    const int ctiles = (a.C + 64 * VEC - 1) / (64 * VEC), tile = blockIdx.x / ctiles, c = (blockIdx.x % ctiles * 64 + lane) * VEC;
    const int64_t t0 = (int64_t)tile * GLR_TILE + wave * L, limit = a.seqs.limit();
    const int count = (int)(limit - t0 < 0 ? 0 : limit - t0 < L ? limit - t0 : L);
    float A[VEC], Q[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
        A[i] = 1.f;
        Q[i] = 0.f;
    }
    if (c < a.C && count > 0) {
        uint64_t first, last;
        a.seqs.marks(t0, count, first, last);
        GateConst<VEC, LOGITS> k;
        k.load(a.gates, c);
        const T *d = static_cast<const T *>(a.d_out) + t0 * a.C + c;
        const gate_t<T, LOGITS> *z = static_cast<const gate_t<T, LOGITS> *>(a.gates.gate) + t0 * a.gates.gate_stride + c;
        Raw<T, VEC> rd[L];
        Raw<gate_t<T, LOGITS>, VEC> rz[L];
#pragma unroll
        for (int u = 0; u < L; ++u) {
            const int64_t at = u < count ? u : count - 1;
            rd[u].load(d + at * a.C);
            rz[u].load(z + at * a.gates.gate_stride);
        }
#pragma unroll
        for (int u = L - 1; u >= 0; --u) {
            if (u >= count) continue;
            if (last >> u & 1) {
                float m[VEC] = {};
                if (a.d_sf) load_f32<VEC>(m, a.d_sf + (int64_t)a.seqs.of(t0 + u) * a.C + c);
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    A[i] = 0.f;
                    Q[i] = m[i];
                }
            }
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const float g = make_gate<LOGITS, false, false>(rz[u].get(i), 0.f, k.scale2[i], k.bias2[i], a.gates.lower).a;
                A[i] *= g;
                Q[i] = g * (rd[u].get(i) + Q[i]);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
        sA[wave][lane][i] = A[i];
        sQ[wave][lane][i] = Q[i];
    }
    __syncthreads();
    if (wave || c >= a.C) return;
    float *agg = a.agg + (int64_t)tile * 2 * a.C + c;
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
        float x = 1.f, m = 0.f;
        for (int w = WAVES - 1; w >= 0; --w) {
            m = join(sA[w][lane][i], sQ[w][lane][i], m);
            x *= sA[w][lane][i];
        }
        agg[i] = x;
        agg[a.C + i] = m;
    }
}

template <typename T, int VEC, bool LOGITS, bool NORM, bool GATED>
__global__ __launch_bounds__(64 * WAVES) void glr_bwd_kernel(const GlrArgs a, const float *behind, int blocks) {
    if ((int)blockIdx.x >= blocks) {  // the gradient of a sequence without a row is that of what it handed on
        const int64_t i = (int64_t)(blockIdx.x - blocks) * blockDim.x + threadIdx.x;
        if (i < (int64_t)a.seqs.N * a.C) {
            const int n = (int)(i / a.C);
            if (a.seqs.cu[n + 1] <= a.seqs.cu[n]) a.ds0[i] = a.d_sf ? a.d_sf[i] : 0.f;
        }
        return;
    }
    __shared__ float sA[WAVES][64][VEC], sH[WAVES][64][VEC], sB[WAVES][64][VEC], sQ[WAVES][64][VEC];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), lane = threadIdx.x & 63;
    const int ctiles = (a.C + 64 * VEC - 1) / (64 * VEC), tile = blockIdx.x / ctiles, c = (blockIdx.x % ctiles * 64 + lane) * VEC;
    const int64_t t0 = (int64_t)tile * GLR_TILE + wave * L, limit = a.seqs.limit();
    const int rows = (int)(a.seqs.rows - t0 < 0 ? 0 : a.seqs.rows - t0 < L ? a.seqs.rows - t0 : L);
    const int count = (int)(limit - t0 < 0 ? 0 : limit - t0 < L ? limit - t0 : L);
    const bool there = c < a.C, busy = there && count > 0;
    typedef gate_t<T, LOGITS> Z;
    GateConst<VEC, LOGITS> k;
    uint64_t first = 0, last = 0;
    Raw<T, VEC> rx[L], ri[L], rd[L];
    Raw<Z, VEC> rz[L];
    float av[L][VEC], bv[L][VEC], A[VEC], H[VEC], B[VEC], Q[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
        A[i] = B[i] = 1.f;
        H[i] = Q[i] = 0.f;
    }
    // the state in front of a sequence's first row, what comes back behind its last
    auto front = [&](float(&h)[VEC], int u) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) h[i] = 0.f;
        if (a.s0) load_f32<VEC>(h, a.s0 + (int64_t)a.seqs.of(t0 + u) * a.C + c);
    };
    auto back = [&](float(&m)[VEC], int u) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) m[i] = 0.f;
        if (a.d_sf) load_f32<VEC>(m, a.d_sf + (int64_t)a.seqs.of(t0 + u) * a.C + c);
    };
    if (busy) {
        a.seqs.marks(t0, count, first, last);
        k.load(a.gates, c);
        const T *x = static_cast<const T *>(a.x) + t0 * a.x_stride + c, *in = static_cast<const T *>(a.gates.in_gate) + t0 * a.gates.in_stride + c;
        const T *d = static_cast<const T *>(a.d_out) + t0 * a.C + c;
        const Z *z = static_cast<const Z *>(a.gates.gate) + t0 * a.gates.gate_stride + c;
#pragma unroll
        for (int u = 0; u < L; ++u) {
            const int64_t at = u < count ? u : count - 1;
            rx[u].load(x + at * a.x_stride);
            rz[u].load(z + at * a.gates.gate_stride);
            rd[u].load(d + at * a.C);
            if constexpr (GATED) ri[u].load(in + at * a.gates.in_stride);
            else ri[u].zero();
        }
#pragma unroll
        for (int u = 0; u < L; ++u)
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const Gate g = make_gate<LOGITS, NORM, GATED>(rz[u].get(i), ri[u].get(i), k.scale2[i], k.bias2[i], a.gates.lower);
                av[u][i] = g.a;
                bv[u][i] = g.f * g.i * rx[u].get(i);
            }
#pragma unroll
        for (int u = 0; u < L; ++u) {
            if (u >= count) break;
            if (first >> u & 1) {
                front(H, u);
#pragma unroll
                for (int i = 0; i < VEC; ++i) A[i] = 0.f;
            }
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                A[i] *= av[u][i];
                H[i] = fmaf(av[u][i], H[i], bv[u][i]);
            }
        }
#pragma unroll
        for (int u = L - 1; u >= 0; --u) {
            if (u >= count) continue;
            if (last >> u & 1) {
                back(Q, u);
#pragma unroll
                for (int i = 0; i < VEC; ++i) B[i] = 0.f;
            }
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                B[i] *= av[u][i];
                Q[i] = av[u][i] * (rd[u].get(i) + Q[i]);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
        sA[wave][lane][i] = A[i];
        sH[wave][lane][i] = H[i];
        sB[wave][lane][i] = B[i];
        sQ[wave][lane][i] = Q[i];
    }
    __syncthreads();
    float dz_sum[VEC] = {}, u_sum[VEC] = {};
    T *dx = static_cast<T *>(a.dx) + t0 * a.C + c, *di = static_cast<T *>(a.d_in) + t0 * a.C + c;
    Z *dz = static_cast<Z *>(a.d_gate) + t0 * a.C + c;
    if (busy) {
        float h[VEC], m[VEC];
        load_f32<VEC>(h, a.kept + (int64_t)tile * a.C + c);
        load_f32<VEC>(m, behind + (int64_t)tile * a.C + c);
        for (int w = 0; w < wave; ++w)
#pragma unroll
            for (int i = 0; i < VEC; ++i) h[i] = join(sA[w][lane][i], sH[w][lane][i], h[i]);
        for (int w = WAVES - 1; w > wave; --w)
#pragma unroll
            for (int i = 0; i < VEC; ++i) m[i] = join(sB[w][lane][i], sQ[w][lane][i], m[i]);
        // bv becomes the state in front of its row
#pragma unroll
        for (int u = 0; u < L; ++u) {
            if (u >= count) break;
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
            if (u >= count) continue;
            if (last >> u & 1) back(m, u);
            Raw<T, VEC> ox, oi;
            Raw<Z, VEC> oz;
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const float x = rx[u].get(i);
                const Gate g = make_gate<LOGITS, NORM, GATED>(rz[u].get(i), ri[u].get(i), k.scale2[i], k.bias2[i], a.gates.lower);
                const float lam = rd[u].get(i) + m[i];
                m[i] = g.a * lam;
                const float v = lam * g.i;
                ox.set(i, v * g.f);
                if constexpr (GATED) oi.set(i, v * g.f * x * g.j);
                float dg = m[i] * bv[u][i];
                if constexpr (NORM) dg -= g.f > 0.f ? v * x * g.a * g.a * __builtin_amdgcn_rcpf(g.f) : 0.f;
                if constexpr (LOGITS) {
                    const float du = dg * a.gates.lower * g.p * g.q;
                    const float t = (k.scale2[i] * (1.f / LOG2E)) * du;
                    u_sum[i] += fmaf(k.scale2[i], rz[u].get(i), k.bias2[i]) * du;
                    dz_sum[i] += t;
                    oz.set(i, t);
                } else {
                    oz.set(i, dg);
                }
            }
            ox.store(dx + (int64_t)u * a.C);
            oz.store(dz + (int64_t)u * a.C);
            if constexpr (GATED) oi.store(di + (int64_t)u * a.C);
            if (a.ds0 && first >> u & 1) {
                float *to = a.ds0 + (int64_t)a.seqs.of(t0 + u) * a.C + c;
#pragma unroll
                for (int i = 0; i < VEC; ++i) to[i] = m[i];
            }
        }
    }
    if (there) {  // rows behind the last sequence
        Raw<T, VEC> ox;
        Raw<Z, VEC> oz;
        ox.zero();
        oz.zero();
        for (int u = count; u < rows; ++u) {
            ox.store(dx + (int64_t)u * a.C);
            oz.store(dz + (int64_t)u * a.C);
            if constexpr (GATED) ox.store(di + (int64_t)u * a.C);
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
hipError_t by_input(const GlrArgs &a, const float *behind, hipStream_t stream) {
    const int64_t blocks = (int64_t)((a.C + 64 * VEC - 1) / (64 * VEC)) * a.tiles;
    const int64_t more = a.seqs.cu && a.ds0 ? ((int64_t)a.seqs.N * a.C + 64 * WAVES - 1) / (64 * WAVES) : 0;
    const dim3 grid((unsigned)(blocks + more)), block(64 * WAVES);
    if (a.gates.in_gate) hipLaunchKernelGGL((glr_bwd_kernel<T, VEC, LOGITS, NORM, true>), grid, block, 0, stream, a, behind, (int)blocks);
    else hipLaunchKernelGGL((glr_bwd_kernel<T, VEC, LOGITS, NORM, false>), grid, block, 0, stream, a, behind, (int)blocks);
    return hipGetLastError();
}
template <typename T, int VEC, bool LOGITS>
hipError_t by_norm(const GlrArgs &a, float *behind, hipStream_t stream) {
    const int64_t blocks = (int64_t)((a.C + 64 * VEC - 1) / (64 * VEC)) * a.tiles;
    hipLaunchKernelGGL((glr_back_kernel<T, VEC, LOGITS>), dim3((unsigned)blocks), dim3(64 * WAVES), 0, stream, a);
    hipError_t e = hipGetLastError();
    if (e == hipSuccess) e = launch_glr_carry(a.agg, behind, a.tiles, a.C, true, stream);
    if (e != hipSuccess) return e;
    return a.gates.normalize ? by_input<T, VEC, LOGITS, true>(a, behind, stream) : by_input<T, VEC, LOGITS, false>(a, behind, stream);
}
template <typename T, int VEC>
hipError_t by_gate(const GlrArgs &a, float *behind, hipStream_t stream) {
    return a.gates.log_scale ? by_norm<T, VEC, true>(a, behind, stream) : by_norm<T, VEC, false>(a, behind, stream);
}

}  // namespace

// The workspace: A and H (then A and Q) of the tiles, the m behind them, partial sums and their sums, and the states in
// front of the tiles where the caller has not kept them.
size_t carve_glr_bwd(GlrArgs &a, void *base, bool kept, float *&sums) {
    Pieces w{static_cast<char *>(base)};
    const int64_t n = (int64_t)a.tiles * a.C;
    w.take(a.agg, 3 * n);
    w.take(a.part, a.gates.log_scale ? 2 * n : 0);
    w.take(sums, a.gates.log_scale ? a.C : 0);
    if (!kept) w.take(a.kept, n);
    return w.used;
}

hipError_t launch_glr_bwd(const GlrArgs &a, bool fp32, bool wide, float *sums, float *d_log_scale, float *d_bias, hipStream_t stream) {
    float *behind = a.agg + (int64_t)a.tiles * 2 * a.C;
    hipError_t e;
    if (wide) e = fp32 ? by_gate<float, 4>(a, behind, stream) : by_gate<__bf16, 4>(a, behind, stream);
    else e = fp32 ? by_gate<float, 1>(a, behind, stream) : by_gate<__bf16, 1>(a, behind, stream);
    if (e != hipSuccess || !a.part) return e;
    e = launch_column_sums(ColumnSums{a.part, a.tiles, 2 * a.C, a.C, 1, d_bias, sums}, stream);
    if (e != hipSuccess || !d_log_scale) return e;
    hipLaunchKernelGGL(head_sums_kernel, dim3((unsigned)(a.C / a.gates.K)), dim3(64), 0, stream, sums, a.gates.K, d_log_scale);
    return hipGetLastError();
}

}  // namespace kda
