// kda_glr_bwd.hip -- gradients of the gated linear recurrence (gfx950).
//
// With lambda_t the gradient of h_t and m_t = a_t lambda_t that of h_{t-1}:
//   lambda_t = d out_t + m_{t+1}   (behind a sequence's last row: the gradient of its final state)
//   dx = lambda f i,   di_t = lambda f x i (1 - i),   dg = a lambda h_{t-1} - lambda i x a^2 / f
// (the second term where f = sqrt(1 - a^2), 0 where f is), and through the bounded gate
// du = dg lower p (1 - p), dz = e^A du, d bias = sum dz, d log_scale = sum u du.
// m is a recurrence from the right with the same decays: a tile maps the m behind it to the one in front as
// m -> A m + Q, and the launches are the forward's, from the last tile to the first.  A wave goes through its tile from
// the right, U rows at a time: their states again from the one that the forward kept in front of them, then m and
// the gradients.  Bound by
// memory: four rows read and three written (a gate and an input gate, bf16: 14 bytes a number).  8192 rows of 4096
// channels: A and Q 27 us, the pass over the tiles 5, the rows 102 us (0.49 GB with the kept states, 4.8 TB/s; a large copy
// has 5.0), the sums 9.  With a row's gates kept instead of what its lambda is multiplied by, a wave more than fills half of a
// SIMD's registers: 184 us.
#include "kda_glr.h"

namespace kda {
namespace {

constexpr int WAVES = 4;
static_assert(U == GLR_KEPT, "a state is kept in front of the rows that a wave takes at a time");

// A and Q of every tile
template <typename T, int VEC, bool LOGITS>
__global__ __launch_bounds__(64 * WAVES) void glr_back_kernel(const GlrArgs a) {
    typedef gate_t<T, LOGITS> Z;
    const int wave = blockIdx.x * WAVES + __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    if (wave >= a.tiles.n * a.tiles.columns) return;
    const GlrPlace p = glr_place<VEC>(a, wave);
    if (!p.there) return;
    const int64_t sd = a.C * sizeof(T), sz = a.gates.gate_stride * sizeof(Z);
    const char *d = static_cast<const char *>(a.d_out) + p.t0 * sd, *z = static_cast<const char *>(a.gates.gate) + p.t0 * sz;
    Raw<T, VEC> nd[U];
    Raw<Z, VEC> nz[U];
    auto fetch = [&](int r) {
        load_run(nz, z + r * sz, sz, p.c * (uint32_t)sizeof(Z), p.own - r);
        load_run(nd, d + r * sd, sd, p.c * (uint32_t)sizeof(T), p.own - r);
    };
    const int begin = (p.own - 1) / U * U;
    if (p.own > 0) fetch(begin);
    GateConst<VEC, LOGITS> k;
    k.load(a.gates, p.c);
    float A[VEC], Q[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
        A[i] = 1.f;
        Q[i] = 0.f;
    }
    if (p.own > 0)
        for (int r = begin; r >= 0; r -= U) {
            float av[U][VEC], dv[U][VEC];
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    av[u][i] = make_gate<LOGITS, false, false>(nz[u].get(i), 0.f, k.scale2[i], k.bias2[i], a.gates.lower).a;
                    dv[u][i] = nd[u].get(i);
                }
            if (r > 0) fetch(r - U);
            const uint32_t last = (uint32_t)(p.last >> r) & ((1u << U) - 1);
            auto rows = [&](auto marked) {
                constexpr bool HERE = decltype(marked)::value;
#pragma unroll
                for (int u = U - 1; u >= 0; --u) {
                    if (HERE && r + u >= p.own) continue;
                    if (HERE && last >> u & 1) {
#pragma unroll
                        for (int i = 0; i < VEC; ++i) {
                            A[i] = CUT;
                            Q[i] = 0.f;
                        }
                        if (a.d_sf) load_f32<VEC>(Q, a.d_sf + (int64_t)a.seqs.of(p.t0 + r + u) * a.C + p.c);
                    }
#pragma unroll
                    for (int i = 0; i < VEC; ++i) {
                        A[i] *= av[u][i];
                        Q[i] = av[u][i] * (dv[u][i] + Q[i]);
                    }
                }
            };
            if (last || r + U > p.own) rows(std::true_type{});
            else rows(std::false_type{});
        }
    glr_word<VEC>(a, p.tile, p.c, A, Q);
}

template <typename T, int VEC, bool LOGITS, bool NORM, bool GATED>
__global__ __launch_bounds__(64 * WAVES) void glr_bwd_kernel(const GlrArgs a, int blocks) {
    if ((int)blockIdx.x >= blocks) {  // the gradient of a sequence without a row is that of what it handed on
        const int64_t i = (int64_t)(blockIdx.x - blocks) * blockDim.x + threadIdx.x;
        if (i < (int64_t)a.seqs.N * a.C) {
            const int n = (int)(i / a.C);
            if (a.seqs.cu[n + 1] <= a.seqs.cu[n]) a.ds0[i] = a.d_sf ? a.d_sf[i] : 0.f;
        }
        return;
    }
    typedef gate_t<T, LOGITS> Z;
    const int wave = blockIdx.x * WAVES + __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    if (wave >= a.tiles.n * a.tiles.columns) return;
    const GlrPlace p = glr_place<VEC>(a, wave);
    if (!p.there) return;
    const uint32_t ct = p.c * (uint32_t)sizeof(T), cz = p.c * (uint32_t)sizeof(Z);
    const int64_t sx = a.x_stride * sizeof(T), sz = a.gates.gate_stride * sizeof(Z), si = a.gates.in_stride * sizeof(T), st = a.C * sizeof(T), sg = a.C * sizeof(Z);
    const char *x = static_cast<const char *>(a.x) + p.t0 * sx, *z = static_cast<const char *>(a.gates.gate) + p.t0 * sz;
    const char *in = static_cast<const char *>(a.gates.in_gate) + p.t0 * si, *d = static_cast<const char *>(a.d_out) + p.t0 * st;
    char *dx = static_cast<char *>(a.dx) + p.t0 * st, *di = static_cast<char *>(a.d_in) + p.t0 * st, *dz = static_cast<char *>(a.d_gate) + p.t0 * sg;
    const float *kept = a.kept + p.t0 / GLR_KEPT * a.C + p.c;
    Raw<T, VEC> nx[U], ni[U], nd[U];
    Raw<Z, VEC> nz[U];
    Raw<float, VEC> nh;
    auto fetch = [&](int r) {
        load_run(nz, z + r * sz, sz, cz, p.own - r);
        load_run(nx, x + r * sx, sx, ct, p.own - r);
        if constexpr (GATED) load_run(ni, in + r * si, si, ct, p.own - r);
        load_run(nd, d + r * st, st, ct, p.own - r);
        nh.load(kept + (int64_t)(r / GLR_KEPT) * a.C);
    };
    const int begin = (p.own - 1) / U * U;
    if (p.own > 0) fetch(begin);
    {  // rows behind the last sequence
        Raw<T, VEC> ox;
        Raw<Z, VEC> oz;
        ox.zero();
        oz.zero();
        for (int u = p.own; u < p.count; ++u) {
            ox.store(dx + u * st, ct);
            oz.store(dz + u * sg, cz);
            if constexpr (GATED) ox.store(di + u * st, ct);
        }
    }
    GateConst<VEC, LOGITS> k;
    k.load(a.gates, p.c);
    float m[VEC], dz_sum[VEC] = {}, u_sum[VEC] = {}, slope[VEC];  // u_sum: of log2(e) u dz
#pragma unroll
    for (int i = 0; i < VEC; ++i) slope[i] = k.scale2[i] * (a.gates.lower / LOG2E);  // lower e^A
    glr_front<VEC>(m, a, a.tiles.front, p.tile, p.c, true);
    if (p.own > 0)
        for (int r = begin; r >= 0; r -= U) {
            // What a row's lambda is multiplied by: a for m, f i for dx, f i (1 - i) x for d in, and for dz
            // (a h_{t-1} - f i x a^2 / f^2) lower p (1 - p) e^A (without logits the bracket alone)
            float av[U][VEC], xv[U][VEC], iv[U][VEC], gv[U][VEC], h[VEC];
            Raw<T, VEC> rd[U];
            Raw<Z, VEC> rz[U];
            const uint32_t first = (uint32_t)(p.first >> r) & ((1u << U) - 1), last = (uint32_t)(p.last >> r) & ((1u << U) - 1);
#pragma unroll
            for (int i = 0; i < VEC; ++i) h[i] = nh.get(i);
            auto rows = [&](auto marked) {
                constexpr bool HERE = decltype(marked)::value;
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    rd[u] = nd[u];
                    rz[u] = nz[u];
                    if (HERE && first >> u & 1) {
#pragma unroll
                        for (int i = 0; i < VEC; ++i) h[i] = 0.f;
                        if (a.s0) load_f32<VEC>(h, a.s0 + (int64_t)a.seqs.of(p.t0 + r + u) * a.C + p.c);
                    }
#pragma unroll
                    for (int i = 0; i < VEC; ++i) {
                        const Gate g = make_gate<LOGITS, NORM, GATED>(rz[u].get(i), GATED ? ni[u].get(i) : 0.f, k.scale2[i], k.bias2[i], a.gates.lower);
                        const float fi = g.f * g.i, b = fi * nx[u].get(i);
                        av[u][i] = g.a;
                        xv[u][i] = fi;
                        if constexpr (GATED) iv[u][i] = b * g.j;
                        float w = g.a * h[i];
                        h[i] = w + b;
                        if constexpr (NORM) w = fmaf(-b, g.f > 0.f ? g.a * g.a * __builtin_amdgcn_rcpf(g.f * g.f) : 0.f, w);
                        gv[u][i] = LOGITS ? w * slope[i] * g.p * g.q : w;
                    }
                }
                if (r > 0) fetch(r - U);
                const uint32_t ot = here(ct), og = here(cz);
#pragma unroll
                for (int u = U - 1; u >= 0; --u) {
                    if (HERE && r + u >= p.own) continue;
                    if (HERE && last >> u & 1) {
#pragma unroll
                        for (int i = 0; i < VEC; ++i) m[i] = 0.f;
                        if (a.d_sf) load_f32<VEC>(m, a.d_sf + (int64_t)a.seqs.of(p.t0 + r + u) * a.C + p.c);
                    }
                    Raw<T, VEC> ox, oi;
                    Raw<Z, VEC> oz;
#pragma unroll
                    for (int i = 0; i < VEC; ++i) {
                        const float lam = rd[u].get(i) + m[i];
                        m[i] = av[u][i] * lam;
                        ox.set(i, lam * xv[u][i]);
                        if constexpr (GATED) oi.set(i, lam * iv[u][i]);
                        const float t = lam * gv[u][i];
                        oz.set(i, t);
                        if constexpr (LOGITS) {
                            // u of a logit far out may be infinite, where t is 0 and their product's limit is: held in range
                            const float far = __builtin_amdgcn_fmed3f(fmaf(k.scale2[i], rz[u].get(i), k.bias2[i]), -3e38f, 3e38f);
                            u_sum[i] = fmaf(far, t, u_sum[i]);
                            dz_sum[i] += t;
                        }
                    }
                    ox.store(dx + (r + u) * st, ot);
                    oz.store(dz + (r + u) * sg, og);
                    if constexpr (GATED) oi.store(di + (r + u) * st, ot);
                    if (HERE && a.ds0 && first >> u & 1) {
                        Raw<float, VEC> s;
#pragma unroll
                        for (int i = 0; i < VEC; ++i) s.set(i, m[i]);
                        s.store(a.ds0 + (int64_t)a.seqs.of(p.t0 + r + u) * a.C + p.c);
                    }
                }
            };
            if (first | last || r + U > p.own) rows(std::true_type{});
            else rows(std::false_type{});
        }
    if (LOGITS && a.part) {
        Raw<float, VEC> s, t;
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            s.set(i, dz_sum[i]);
            t.set(i, k.scale2[i] > 0.f ? u_sum[i] / k.scale2[i] : 0.f);  // sum u du, du = dz e^-A
        }
        s.store(a.part + (int64_t)p.tile * 2 * a.C + p.c);
        t.store(a.part + (int64_t)p.tile * 2 * a.C + a.C + p.c);
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
hipError_t by_input(const GlrArgs &a, int64_t waves, hipStream_t stream) {
    const int64_t blocks = (waves + WAVES - 1) / WAVES;
    const int64_t more = a.seqs.cu && a.ds0 ? ((int64_t)a.seqs.N * a.C + 64 * WAVES - 1) / (64 * WAVES) : 0;
    const dim3 grid((unsigned)(blocks + more)), block(64 * WAVES);
    if (a.gates.in_gate) hipLaunchKernelGGL((glr_bwd_kernel<T, VEC, LOGITS, NORM, true>), grid, block, 0, stream, a, (int)blocks);
    else hipLaunchKernelGGL((glr_bwd_kernel<T, VEC, LOGITS, NORM, false>), grid, block, 0, stream, a, (int)blocks);
    return hipGetLastError();
}
template <typename T, int VEC, bool LOGITS>
hipError_t by_norm(GlrArgs a, hipStream_t stream) {
    const int64_t waves = glr_waves(a, VEC);
    if (a.tiles.n > 1) {
        hipLaunchKernelGGL((glr_back_kernel<T, VEC, LOGITS>), dim3((unsigned)((waves + WAVES - 1) / WAVES)), dim3(64 * WAVES), 0, stream, a);
        hipError_t e = hipGetLastError();
        if (e == hipSuccess) e = launch_glr_carry(a, true, stream);
        if (e != hipSuccess) return e;
    }
    return a.gates.normalize ? by_input<T, VEC, LOGITS, true>(a, waves, stream) : by_input<T, VEC, LOGITS, false>(a, waves, stream);
}
template <typename T, int VEC>
hipError_t by_gate(const GlrArgs &a, hipStream_t stream) {
    return a.gates.log_scale ? by_norm<T, VEC, true>(a, stream) : by_norm<T, VEC, false>(a, stream);
}

}  // namespace

// The workspace: the tiles' words (the forward's before, where the states were not kept), partial sums and their sums, and
// those states.
size_t carve_glr_bwd(GlrArgs &a, void *base, bool kept, float *&sums) {
    Pieces w{static_cast<char *>(base)};
    glr_plan(a);
    carve_glr_tiles(a, w);
    w.take(a.part, a.gates.log_scale ? (int64_t)a.tiles.n * 2 * a.C : 0);
    w.take(sums, a.gates.log_scale ? a.C : 0);
    if (!kept) w.take(a.kept, (a.seqs.rows + GLR_KEPT - 1) / GLR_KEPT * a.C);
    return w.used;
}

hipError_t launch_glr_bwd(const GlrArgs &a, bool fp32, bool wide, bool kept, float *sums, float *d_log_scale, float *d_bias, hipStream_t stream) {
    hipError_t e = hipSuccess;
    if (!kept) {
        GlrArgs f = a;
        f.out = nullptr;
        f.sf = nullptr;
        e = launch_glr_fwd(f, fp32, wide, stream);
        if (e != hipSuccess) return e;
    }
    if (wide) e = fp32 ? by_gate<float, 2>(a, stream) : by_gate<__bf16, 2>(a, stream);
    else e = fp32 ? by_gate<float, 1>(a, stream) : by_gate<__bf16, 1>(a, stream);
    if (e != hipSuccess || !a.part) return e;
    e = launch_column_sums(ColumnSums{a.part, a.tiles.n, 2 * a.C, a.C, 1, d_bias, sums}, stream);
    if (e != hipSuccess || !d_log_scale) return e;
    hipLaunchKernelGGL(head_sums_kernel, dim3((unsigned)(a.C / a.gates.K)), dim3(64), 0, stream, sums, a.gates.K, d_log_scale);
    return hipGetLastError();
}

}  // namespace kda
