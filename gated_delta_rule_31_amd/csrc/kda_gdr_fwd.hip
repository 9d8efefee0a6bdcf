// kda_gdr_fwd.hip -- chunkwise prefill of the gated delta rule with one decay per value head
// (formulas and precision: kda_gdr.h).  Two kernels: a pre-pass over all (chunk, value head)
// pairs at once, which forms what does not depend on the state (M, P, the decays, K^T), and
// the chain, serial over a sequence's chunks and parallel over sequences, value heads and
// blocks of 16 value columns.
#include "kda_gdr.h"

namespace kda {
namespace {

constexpr int C = GDR_C;
constexpr int LA = C + 4;  // row stride of the C x C float32 matrices in LDS

// Eight elements down a column of an LDS tile, as parts.
template <int P, typename T>
__device__ __forceinline__ Parts<P> column8(const T *m, int ld, int row, int col) {
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = to_f32(m[(row + i) * ld + col]);
    return cut8<P>(x);
}

// One workgroup of four waves per (chunk slot, value head); wave w owns token rows 16w..16w+15.
template <typename T, int K, int P, bool BWD>
__global__ __launch_bounds__(256) void gdr_prep_kernel(const GdrArgs a) {
    constexpr int PK = gdr_input_parts<T>(), KP = K < 32 ? 32 : K, LK = KP + 8, KS = KP / 32, VEC = 16 / sizeof(T);
    __shared__ __attribute__((aligned(16))) T sK[C * LK], sQ[C * LK];
    __shared__ __attribute__((aligned(16))) float sA[C * LA], sM[C * LA], sD[4 * 16 * 20], sB[C];
    __shared__ double sG[C];
    const int unit = blockIdx.x, hv = unit % a.HV, hk = hv / a.group;
    const int64_t slot = unit / a.HV;
    int64_t row;
    int len;
    if (!gdr_chunk(a, slot, row, len)) return;
    const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6), lr = lane & 15, lg = lane >> 4;

    // k and q rows into LDS, zeros behind the sequence's end and beside a width of 16
    const T *q = static_cast<const T *>(a.q), *k = static_cast<const T *>(a.k);
    for (int i = tid; i < C * KP / VEC; i += 256) {
        const int r = i / (KP / VEC), c = i % (KP / VEC) * VEC;
        f4 x = {}, y = {};
        if (r < len && c < K) {
            const int64_t at = ((row + r) * a.HK + hk) * K + c;
            x = *reinterpret_cast<const f4 *>(k + at);
            y = *reinterpret_cast<const f4 *>(q + at);
        }
        *reinterpret_cast<f4 *>(sK + r * LK + c) = x;
        *reinterpret_cast<f4 *>(sQ + r * LK + c) = y;
    }
    if (w == 0) {
        const int64_t at = (row + lane) * a.HV + hv;
        // log2 units in float64; beyond 2^-1000 a decay is 0 in float32 whatever follows, and
        // the bound keeps -inf out of the differences
        double g = lane < len ? (double)a.g[at] * 1.4426950408889634 : 0.0;
        g = g < -1000.0 ? -1000.0 : g;
#pragma unroll
        for (int d = 1; d < 64; d *= 2) {
            const double up = __shfl_up(g, d);
            if (lane >= d) g += up;
        }
        const double last = __shfl(g, 63);
        const float beta = lane < len ? a.beta[at] : 0.f;
        sG[lane] = g;
        sB[lane] = beta;
        float *dec = a.dec + (int64_t)unit * 4 * C;
        dec[lane] = exp2f((float)g);
        dec[C + lane] = exp2f((float)(last - g));
        dec[2 * C + lane] = beta;
        if (BWD) a.G[(int64_t)unit * C + lane] = g;
    }
    __syncthreads();

    // A and P, tile by tile (P goes to sM until M takes its place)
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        f4 kk = {}, qk = {};
        if (c <= w) {
#pragma unroll
            for (int s = 0; s < KS; ++s) {
                const Parts<PK> b = load8<PK>(sK + (16 * c + lr) * LK + 32 * s + 8 * lg, true);
                mma(kk, load8<PK>(sK + (16 * w + lr) * LK + 32 * s + 8 * lg, true), b);
                mma(qk, load8<PK>(sQ + (16 * w + lr) * LK + 32 * s + 8 * lg, true), b);
            }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int i = 16 * w + 4 * lg + e, j = 16 * c + lr;
            const float d = j <= i ? exp2f((float)(sG[i] - sG[j])) : 0.f;
            sA[i * LA + j] = j < i ? kk[e] * d : 0.f;
            sM[i * LA + j] = j <= i ? qk[e] * d : 0.f;
        }
    }
    __syncthreads();

    // P (or P^T) leaves; K^T (and Q^T) leave once for the value heads of a group
    {
        __bf16 *to = a.P + (int64_t)unit * P * C * C;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            if (BWD) store_frag<P>(to, w, s, lane, column8<P>(sM, LA, 32 * s + 8 * lg, 16 * w + lr));
            else store_frag<P>(to, w, s, lane, cut8<P>(sM + (16 * w + lr) * LA + 32 * s + 8 * lg));
        }
        if (hv % a.group == 0) {
            const int64_t at = (slot * a.HK + hk) * (PK * K * C);
            for (int i = w; i < K / 16 * 2; i += 4) {
                store_frag<PK>(a.Kt + at, i / 2, i % 2, lane, column8<PK>(sK, LK, 32 * (i % 2) + 8 * lg, 16 * (i / 2) + lr));
                if (BWD) store_frag<PK>(a.Qt + at, i / 2, i % 2, lane, column8<PK>(sQ, LK, 32 * (i % 2) + 8 * lg, 16 * (i / 2) + lr));
            }
        }
    }
    // the inverse of block w of 1 + A beta on the diagonal, a column a lane, by substitution
    {
        float x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            float s = i == lr ? 1.f : 0.f;
#pragma unroll
            for (int m = 0; m < i; ++m) s -= sA[(16 * w + i) * LA + 16 * w + m] * (sB[16 * w + m] * x[m]);
            x[i] = s;
        }
        if (lg == 0) {
#pragma unroll
            for (int i = 0; i < 16; ++i) sD[(16 * w + i) * 20 + lr] = x[i];
        }
    }
    __syncthreads();

    // M by columns of blocks, wave w column w: (1 + A_pp beta_p) M_pw = -(A_pw + sum_r A_pr beta_r M_rw).
    // Step e of a product takes k = 4 (lane / 16) + e, which is how an accumulator holds its rows.
    {
        f4 m[4];
#pragma unroll
        for (int p = 0; p < 4; ++p) {
            f4 acc = {};
            if (p >= w) {
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[e] = sA[(16 * p + 4 * lg + e) * LA + 16 * w + lr];
#pragma unroll
                for (int r = 0; r < p; ++r)
                    if (r >= w) {
                        const f4 x = *reinterpret_cast<const f4 *>(sA + (16 * p + lr) * LA + 16 * r + 4 * lg);
#pragma unroll
                        for (int e = 0; e < 4; ++e) acc = __builtin_amdgcn_mfma_f32_16x16x4f32(x[e], m[r][e], acc, 0, 0, 0);
                    }
                const f4 d = *reinterpret_cast<const f4 *>(sD + (16 * p + lr) * 20 + 4 * lg);
                f4 y = {};
#pragma unroll
                for (int e = 0; e < 4; ++e) y = __builtin_amdgcn_mfma_f32_16x16x4f32(d[e], -acc[e], y, 0, 0, 0);
                acc = y;
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                sM[(16 * p + 4 * lg + e) * LA + 16 * w + lr] = acc[e];
                m[p][e] = acc[e] * sB[16 * p + 4 * lg + e];
            }
        }
    }
    __syncthreads();
    {
        const int64_t at = (int64_t)unit * P * C * C;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            store_frag<P>(a.M + at, w, s, lane, cut8<P>(sM + (16 * w + lr) * LA + 32 * s + 8 * lg));
            if (BWD) store_frag<P>(a.Mt + at, w, s, lane, column8<P>(sM, LA, 32 * s + 8 * lg, 16 * w + lr));
        }
    }
}

// What a wave needs of one chunk beside the state: its 16 rows of K, Q, M and P, its channel
// rows of K^T, its values and decays.
template <typename T, int K, int P, bool TRAIN>
struct ChainOps {
    static constexpr int PK = gdr_input_parts<T>(), KS = K < 32 ? 1 : K / 32, NC = (K / 16 + 3) / 4;
    Parts<PK> k[KS], q[TRAIN ? 1 : KS], kt[NC][2];
    Parts<P> m[2], p[TRAIN ? 1 : 2];
    f4 v, b, end, beta;
    float last;

    __device__ __forceinline__ void load(const GdrArgs &a, int64_t slot, int64_t row, int len, int hv, int col, int w, int lane) {
        const int lr = lane & 15, lg = lane >> 4, hk = hv / a.group;
        const int64_t unit = slot * a.HV + hv;
        const int64_t at = ((row + 16 * w + lr) * a.HK + hk) * K + 8 * lg;
        const bool there = 16 * w + lr < len;
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            k[s] = load8<PK>(static_cast<const T *>(a.k) + at + 32 * s, there && 32 * s + 8 * lg < K);
            if (!TRAIN) q[s] = load8<PK>(static_cast<const T *>(a.q) + at + 32 * s, there && 32 * s + 8 * lg < K);
        }
#pragma unroll
        for (int s = 0; s < 2; ++s)
            if (s <= w / 2) {
                m[s] = load_frag<P>(a.M + unit * (P * C * C), w, s, lane);
                if (!TRAIN) p[s] = load_frag<P>(a.P + unit * (P * C * C), w, s, lane);
            }
#pragma unroll
        for (int c = 0; c < NC; ++c)
            if (w + 4 * c < K / 16)
#pragma unroll
                for (int s = 0; s < 2; ++s) kt[c][s] = load_frag<PK>(a.Kt + (slot * a.HK + hk) * (PK * K * C), w + 4 * c, s, lane);
        const float *dec = a.dec + unit * 4 * C + 16 * w + 4 * lg;
        b = *reinterpret_cast<const f4 *>(dec);
        end = *reinterpret_cast<const f4 *>(dec + C);
        beta = *reinterpret_cast<const f4 *>(dec + 2 * C);
        last = a.dec[unit * 4 * C + C - 1];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int r = 16 * w + 4 * lg + e;
            v[e] = r < len ? to_f32(static_cast<const T *>(a.v)[((row + r) * a.HV + hv) * a.V + col]) : 0.f;
        }
    }
};

// One workgroup of four waves per (sequence, value head, 16 value columns).  Wave w owns
// token rows 16w..16w+15 of the chunk and the state's channel tiles w, w + 4, ..; what the
// waves exchange (beta X, Vn, the state) goes through LDS as bf16 parts, columns first.
template <typename T, int K, int P, bool TRAIN>
__global__ __launch_bounds__(256) void gdr_chain_kernel(const GdrArgs a) {
    using Ops = ChainOps<T, K, P, TRAIN>;
    constexpr int KP = K < 32 ? 32 : K, LS = KP + 8, LT = C + 8, KS = Ops::KS, NC = Ops::NC;
    __shared__ __attribute__((aligned(16))) __bf16 sS[P * 16 * LS], sX[P * 16 * LT], sV[P * 16 * LT], sE[P * 16 * LT];
    const int VB = a.V / 16, unit = gdr_xcd_unit(blockIdx.x, gridDim.x);
    const int vb = unit % VB, hv = unit / VB % a.HV, n = unit / VB / a.HV;
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lr = lane & 15, lg = lane >> 4;
    const int col = 16 * vb + lr;
    int64_t row, len, slot;
    gdr_sequence(a, n, row, len, slot);
    const int64_t state = ((int64_t)n * a.HV + hv) * K * a.V;

    if (K < 32)
        for (int i = threadIdx.x; i < P * 16 * LS; i += 256) sS[i] = (__bf16)0.f;
    if (K < 32) __syncthreads();
    f4 S[NC];
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        S[c] = f4{};
        if (w + 4 * c < K / 16) {
            const int ch = 16 * (w + 4 * c) + 4 * lg;
            if (a.s0)
#pragma unroll
                for (int e = 0; e < 4; ++e) S[c][e] = a.s0[state + (int64_t)(ch + e) * a.V + col];
            lds_put4<P>(sS, 16 * LS, LS, lr, ch, S[c]);
        }
    }
    Ops o;
    for (int64_t t = 0; t < len; t += C, ++slot) {
        const int here = (int)(len - t < C ? len - t : C);
        o.load(a, slot, row + t, here, hv, col, w, lane);
        if (TRAIN) {
            float *h = a.h + (slot * a.HV + hv) * ((int64_t)K * a.V);
#pragma unroll
            for (int c = 0; c < NC; ++c)
                if (w + 4 * c < K / 16)
#pragma unroll
                    for (int e = 0; e < 4; ++e) h[(int64_t)(16 * (w + 4 * c) + 4 * lg + e) * a.V + col] = S[c][e];
        }
        gdr_lds_barrier();
        f4 x = {}, y = {};
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            const Parts<P> f = lds_frag<P>(sS, 16 * LS, LS, lr, 32 * s + 8 * lg);
            mma(x, o.k[s], f);
            if (!TRAIN) mma(y, o.q[s], f);
        }
        x = o.v - o.b * x;
        lds_put4<P>(sX, 16 * LT, LT, lr, 16 * w + 4 * lg, o.beta * x);
        gdr_lds_barrier();
#pragma unroll
        for (int s = 0; s < 2; ++s)
            if (s <= w / 2) mma(x, o.m[s], lds_frag<P>(sX, 16 * LT, LT, lr, 32 * s + 8 * lg));
        const f4 vn = o.beta * x;
        if (!TRAIN) lds_put4<P>(sV, 16 * LT, LT, lr, 16 * w + 4 * lg, vn);
        lds_put4<P>(sE, 16 * LT, LT, lr, 16 * w + 4 * lg, o.end * vn);
        gdr_lds_barrier();
#pragma unroll
        for (int c = 0; c < NC; ++c)
            if (w + 4 * c < K / 16) {
                S[c] *= o.last;
#pragma unroll
                for (int s = 0; s < 2; ++s) mma(S[c], o.kt[c][s], lds_frag<P>(sE, 16 * LT, LT, lr, 32 * s + 8 * lg));
                lds_put4<P>(sS, 16 * LS, LS, lr, 16 * (w + 4 * c) + 4 * lg, S[c]);
            }
        if (TRAIN) {
            float *d = a.delta + (slot * a.HV + hv) * ((int64_t)C * a.V);
#pragma unroll
            for (int e = 0; e < 4; ++e) d[(int64_t)(16 * w + 4 * lg + e) * a.V + col] = x[e];
        } else {
            y *= o.b;
#pragma unroll
            for (int s = 0; s < 2; ++s)
                if (s <= w / 2) mma(y, o.p[s], lds_frag<P>(sV, 16 * LT, LT, lr, 32 * s + 8 * lg));
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int r = 16 * w + 4 * lg + e;
                if (r < here) st_out(a.out, a.out_bf16, ((row + t + r) * a.HV + hv) * a.V + col, a.scale * y[e]);
            }
        }
    }
    if (!TRAIN && a.sf)
#pragma unroll
        for (int c = 0; c < NC; ++c)
            if (w + 4 * c < K / 16)
#pragma unroll
                for (int e = 0; e < 4; ++e) a.sf[state + (int64_t)(16 * (w + 4 * c) + 4 * lg + e) * a.V + col] = S[c][e];
}

template <typename F>
hipError_t by_width(int K, F f) {
    switch (K) {
        case 16: return f(std::integral_constant<int, 16>());
        case 32: return f(std::integral_constant<int, 32>());
        case 64: return f(std::integral_constant<int, 64>());
        case 128: return f(std::integral_constant<int, 128>());
    }
    return hipErrorNotSupported;
}

template <typename T, int P, bool BWD>
hipError_t prep(const GdrArgs &a, int K, hipStream_t stream) {
    return by_width(K, [&](auto k) {
        hipLaunchKernelGGL((gdr_prep_kernel<T, decltype(k)::value, P, BWD>), dim3((unsigned)(a.slots * a.HV)), dim3(256), 0, stream, a);
        return hipGetLastError();
    });
}
template <typename T, int P, bool TRAIN>
hipError_t chain(const GdrArgs &a, int K, hipStream_t stream) {
    return by_width(K, [&](auto k) {
        hipLaunchKernelGGL((gdr_chain_kernel<T, decltype(k)::value, P, TRAIN>), dim3((unsigned)((int64_t)a.N * a.HV * (a.V / 16))), dim3(256), 0,
                           stream, a);
        return hipGetLastError();
    });
}

}  // namespace

hipError_t launch_gdr_prep(const GdrArgs &a, bool fp32, int K, bool bwd, hipStream_t stream) {
    if (bwd) return fp32 ? prep<float, 3, true>(a, K, stream) : prep<__bf16, 3, true>(a, K, stream);
    return fp32 ? prep<float, 3, false>(a, K, stream) : prep<__bf16, 2, false>(a, K, stream);
}

hipError_t launch_gdr_fwd_chain(const GdrArgs &a, bool fp32, int K, bool train, hipStream_t stream) {
    if (train) return fp32 ? chain<float, 3, true>(a, K, stream) : chain<__bf16, 3, true>(a, K, stream);
    return fp32 ? chain<float, 3, false>(a, K, stream) : chain<__bf16, 2, false>(a, K, stream);
}

}  // namespace kda
