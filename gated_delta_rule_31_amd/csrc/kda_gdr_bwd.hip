// kda_gdr_bwd.hip -- gradients of the chunkwise gated delta rule with one decay per value head
// (forward formulas: kda_gdr.h).  With dO' = scale dO, per chunk from the last to the first:
//   dVn = P^T dO' + e^{G_C - G} K dS'        dY = dVn + M^T (beta dVn)      E = beta dY = dV
//   dS  = e^{G_C} dS' + Q^T e^G dO' - K^T e^G E
// and then, for every chunk at once, with dP = (dO' Vn^T) D and dA = -(E Vn^T) D (j < i):
//   dQ  = e^G dO' S^T + dP K
//   dK  = e^{G_C - G} Vn dS'^T - e^G E S^T + dP^T Q + dA K + dA^T K
//   dbeta_i = dY_i . delta_i
//   dg_t = sum_{i >= t > j} H_ij + sum_{i >= t} reads_i + sum_{i < t} ends_i + e^{G_C} <S, dS'>
// where H = dP (Q K^T) + dA (K K^T) element by element, reads_i = q_i . (e^G dO' S^T)_i -
// k_i . (e^G E S^T)_i and ends_i = k_i . (e^{G_C - G} Vn dS'^T)_i: the pairs (i, j) whose decay
// holds g_t, the rows that read S through it, and those that reach S' through it.  Summed so,
// no term is added that another one takes away.
//
// Four kernels: the pre-pass and the forward chain (kda_gdr_fwd.hip), which keeps every
// chunk's start state and delta; the chain of gradients, serial backwards over the chunks;
// and one workgroup per (chunk, key head) for the rest, which goes through the value heads of
// its group, so that the shared heads' gradients are summed in a fixed order.  Computed
// operands enter the matrix cores as three bf16 parts (24 bits).
#include "kda_gdr.h"

namespace kda {
namespace {

constexpr int C = GDR_C, P = 3;

__device__ __forceinline__ float ld_any(const void *p, int bf16, int64_t i) {
    return bf16 ? (float)static_cast<const __bf16 *>(p)[i] : static_cast<const float *>(p)[i];
}

// The chain of gradients: workgroups and waves as in the forward chain.
template <typename T, int K>
__global__ __launch_bounds__(256) void gdr_bwd_chain_kernel(const GdrArgs a) {
    constexpr int PK = gdr_input_parts<T>(), KP = K < 32 ? 32 : K, KS = KP / 32, NC = (K / 16 + 3) / 4;
    __shared__ __attribute__((aligned(16))) __bf16 sS[P * 16 * KP], sO[P * 16 * C], sX[P * 16 * C], sB[P * 16 * C], sE[P * 16 * C];
    int vb, hv, n;
    if (!gdr_pair(a, a.V / 16, vb, hv, n)) return;
    const int hk = hv / a.group;
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lr = lane & 15, lg = lane >> 4;
    const int col = 16 * vb + lr;
    int64_t row, len, slot;
    gdr_sequence(a, n, row, len, slot);
    const int64_t state = ((int64_t)n * a.HV + hv) * K * a.V;
    if (K < 32) {
        for (int i = threadIdx.x; i < P * 16 * KP; i += 256) sS[i] = (__bf16)0.f;
        __syncthreads();
    }
    f4 S[NC];
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        S[c] = f4{};
        if (w + 4 * c < K / 16) {
            const int ch = 16 * (w + 4 * c) + 4 * lg;
            if (a.d_sf)
#pragma unroll
                for (int e = 0; e < 4; ++e) S[c][e] = a.d_sf[state + (int64_t)(ch + e) * a.V + col];
            lds_put4<P, 16, KP>(sS, lr, ch, S[c]);
        }
    }
    const int64_t chunks = (len + C - 1) / C;
    for (int64_t j = chunks - 1; j >= 0; --j) {
        const int64_t t = j * C, at = (slot + j) * a.HV + hv;
        const int here = (int)(len - t < C ? len - t : C);
        // this chunk's operands
        Parts<PK> k[KS], kt[NC][2], qt[NC][2];
        Parts<P> m[2], p[2];
        f4 b, end, beta, dO;
        {
            const bool there = 16 * w + lr < here;
            const T *kp = static_cast<const T *>(a.k) + ((row + t + 16 * w + lr) * a.HK + hk) * K + 8 * lg;
#pragma unroll
            for (int s = 0; s < KS; ++s) k[s] = load8<PK>(kp + 32 * s, there && 32 * s + 8 * lg < K);
#pragma unroll
            for (int s = 0; s < 2; ++s)
                if (s >= w / 2) {
                    m[s] = load_frag<P>(a.Mt + at * (P * C * C), w, s, lane);
                    p[s] = load_frag<P>(a.P + at * (P * C * C), w, s, lane);
                }
            const int64_t kq = ((slot + j) * a.HK + hk) * (PK * K * C);
#pragma unroll
            for (int c = 0; c < NC; ++c)
                if (w + 4 * c < K / 16)
#pragma unroll
                    for (int s = 0; s < 2; ++s) {
                        kt[c][s] = load_frag<PK>(a.Kt + kq, w + 4 * c, s, lane);
                        qt[c][s] = load_frag<PK>(a.Qt + kq, w + 4 * c, s, lane);
                    }
            const float *dec = a.dec + at * 4 * C + 16 * w + 4 * lg;
            b = *reinterpret_cast<const f4 *>(dec);
            end = *reinterpret_cast<const f4 *>(dec + C);
            beta = *reinterpret_cast<const f4 *>(dec + 2 * C);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int r = 16 * w + 4 * lg + e;
                dO[e] = r < here ? a.scale * ld_any(a.d_out, a.dout_bf16, ((row + t + r) * a.HV + hv) * a.V + col) : 0.f;
            }
        }
        const float last = a.dec[at * 4 * C + C - 1];
        float *dh = a.dh + at * ((int64_t)K * a.V);
#pragma unroll
        for (int c = 0; c < NC; ++c)
            if (w + 4 * c < K / 16)
#pragma unroll
                for (int e = 0; e < 4; ++e) dh[(int64_t)(16 * (w + 4 * c) + 4 * lg + e) * a.V + col] = S[c][e];
        lds_put4<P, 16, C>(sO, lr, 16 * w + 4 * lg, dO);
        gdr_lds_barrier();
        f4 x = {}, y = {};
#pragma unroll
        for (int s = 0; s < KS; ++s) mma(x, k[s], lds_frag<P, 16, KP>(sS, lr, 32 * s + 8 * lg));
#pragma unroll
        for (int s = 0; s < 2; ++s)
            if (s >= w / 2) mma(y, p[s], lds_frag<P, 16, C>(sO, lr, 32 * s + 8 * lg));
        x = end * x + y;
        lds_put4<P, 16, C>(sX, lr, 16 * w + 4 * lg, beta * x);
        lds_put4<P, 16, C>(sB, lr, 16 * w + 4 * lg, b * dO);
        gdr_lds_barrier();
#pragma unroll
        for (int s = 0; s < 2; ++s)
            if (s >= w / 2) mma(x, m[s], lds_frag<P, 16, C>(sX, lr, 32 * s + 8 * lg));
        const f4 E = beta * x;
        lds_put4<P, 16, C>(sE, lr, 16 * w + 4 * lg, -(b * E));
        gdr_lds_barrier();
#pragma unroll
        for (int c = 0; c < NC; ++c)
            if (w + 4 * c < K / 16) {
                S[c] *= last;
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    mma(S[c], qt[c][s], lds_frag<P, 16, C>(sB, lr, 32 * s + 8 * lg));
                    mma(S[c], kt[c][s], lds_frag<P, 16, C>(sE, lr, 32 * s + 8 * lg));
                }
                lds_put4<P, 16, KP>(sS, lr, 16 * (w + 4 * c) + 4 * lg, S[c]);
            }
        float *dY = a.dY + at * ((int64_t)C * a.V);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int r = 16 * w + 4 * lg + e;
            dY[(int64_t)r * a.V + col] = x[e];
            if (r < here) st_out(a.dv, a.grad_bf16, ((row + t + r) * a.HV + hv) * a.V + col, E[e]);
        }
    }
    if (a.ds0)
#pragma unroll
        for (int c = 0; c < NC; ++c)
            if (w + 4 * c < K / 16)
#pragma unroll
                for (int e = 0; e < 4; ++e) a.ds0[state + (int64_t)(16 * (w + 4 * c) + 4 * lg + e) * a.V + col] = S[c][e];
}

// Eight float32 numbers of a row, zeros where !there.
__device__ __forceinline__ void row8(float (&x)[8], const float *p, bool there) {
    f4 u = {}, v = {};
    if (there) {
        u = *reinterpret_cast<const f4 *>(p);
        v = *reinterpret_cast<const f4 *>(p + 4);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[i] = u[i];
        x[4 + i] = v[i];
    }
}

// One workgroup of four waves per (chunk slot, key head); wave w owns token rows 16w..16w+15.
// The products over V go through LDS in slices of 32 columns.
template <typename T, int K>
__global__ __launch_bounds__(256, 1) void gdr_grads_kernel(const GdrArgs a) {
    constexpr int PK = gdr_input_parts<T>(), KS = K < 32 ? 1 : K / 32, CT = K / 16, LA = C + 4, LH = C + 1;
    __shared__ __attribute__((aligned(16))) __bf16 sS[P * K * 32], sH[P * K * 32], sV[P * C * 32];
    __shared__ __attribute__((aligned(16))) float sP[C * LA], sA[C * LA], sT[C * LH], sReads[C], sEnds[C], sKeep[4];
    __shared__ double sG[C];
    const int unit = blockIdx.x, hk = unit % a.HK;
    const int64_t slot = unit / a.HK;
    int64_t row;
    int len;
    if (!gdr_chunk(a, slot, row, len)) return;
    const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6), lr = lane & 15, lg = lane >> 4;
    const int V = a.V, slices = (V + 31) / 32;
    const T *q = static_cast<const T *>(a.q), *k = static_cast<const T *>(a.k);
    const int64_t kq = (slot * a.HK + hk) * (PK * K * C);

    f4 dq[CT], dk[CT];
#pragma unroll
    for (int c = 0; c < CT; ++c) dq[c] = dk[c] = f4{};
    for (int hv = hk * a.group; hv < (hk + 1) * a.group; ++hv) {
        const int64_t at = slot * a.HV + hv;
        const float *dec = a.dec + at * 4 * C, *h = a.h + at * ((int64_t)K * V), *dh = a.dh + at * ((int64_t)K * V);
        const float *delta = a.delta + at * ((int64_t)C * V), *dY = a.dY + at * ((int64_t)C * V);
        if (tid < C) sG[tid] = a.G[at * C + tid];
        f4 r1[CT], r2[CT], r3[CT], dP[4], dA[4];
#pragma unroll
        for (int c = 0; c < CT; ++c) r1[c] = r2[c] = r3[c] = f4{};
#pragma unroll
        for (int c = 0; c < 4; ++c) dP[c] = dA[c] = f4{};
        const float beta_r = dec[2 * C + 16 * w + lr];
        float keep = 0.f, db = 0.f;
        for (int sl = 0; sl < slices; ++sl) {
            const int r = 16 * w + lr, v0 = 32 * sl + 8 * lg;
            const bool in = v0 < V;
            float xo[8], xv[8], xe[8];
            row8(xv, delta + (int64_t)r * V + v0, in);
            row8(xe, dY + (int64_t)r * V + v0, in);
            const int64_t ov = ((row + r) * a.HV + hv) * V + v0;
            if (a.dout_bf16) {
                const bf16x8 o = in && r < len ? *reinterpret_cast<const bf16x8 *>(static_cast<const __bf16 *>(a.d_out) + ov) : bf16x8{};
#pragma unroll
                for (int i = 0; i < 8; ++i) xo[i] = (float)o[i];
            } else {
                row8(xo, static_cast<const float *>(a.d_out) + ov, in && r < len);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                db += xe[i] * xv[i];
                xv[i] *= beta_r;
                xe[i] *= beta_r;
                xo[i] *= a.scale;
            }
            const Parts<P> fo = cut8<P>(xo), fv = cut8<P>(xv), fe = cut8<P>(xe);
            __syncthreads();  // the last slice has been read
#pragma unroll
            for (int p = 0; p < P; ++p) *reinterpret_cast<bf16x8 *>(sV + p * C * 32 + lds_at<32>(r, 8 * lg)) = fv.v[p];
            for (int i = tid; i < K * 4; i += 256) {
                const int ch = i / 4, c = i % 4 * 8;
                float x[8], y[8];
                row8(x, h + (int64_t)ch * V + 32 * sl + c, 32 * sl + c < V);
                row8(y, dh + (int64_t)ch * V + 32 * sl + c, 32 * sl + c < V);
#pragma unroll
                for (int e = 0; e < 8; ++e) keep += x[e] * y[e];
                const Parts<P> fx = cut8<P>(x), fy = cut8<P>(y);
#pragma unroll
                for (int p = 0; p < P; ++p) {
                    *reinterpret_cast<bf16x8 *>(sS + p * K * 32 + lds_at<32>(ch, c)) = fx.v[p];
                    *reinterpret_cast<bf16x8 *>(sH + p * K * 32 + lds_at<32>(ch, c)) = fy.v[p];
                }
            }
            __syncthreads();
#pragma unroll
            for (int c = 0; c < CT; ++c) {
                const Parts<P> s = lds_frag<P, K, 32>(sS, 16 * c + lr, 8 * lg), d = lds_frag<P, K, 32>(sH, 16 * c + lr, 8 * lg);
                mma(r1[c], fo, s);
                mma(r2[c], fe, s);
                mma(r3[c], fv, d);
            }
#pragma unroll
            for (int c = 0; c < 4; ++c)
                if (c <= w) {
                    const Parts<P> f = lds_frag<P, C, 32>(sV, 16 * c + lr, 8 * lg);
                    mma(dP[c], fo, f);
                    mma(dA[c], fe, f);
                }
        }
        // dbeta: a row's eight-column pieces lie in lanes 16 apart
        db += __shfl_xor(db, 16);
        db += __shfl_xor(db, 32);
        if (lg == 0 && 16 * w + lr < len) a.dbeta[(row + 16 * w + lr) * a.HV + hv] = db;
#pragma unroll
        for (int d = 32; d; d /= 2) keep += __shfl_xor(keep, d);
        if (lane == 0) sKeep[w] = keep;

        // the pairs inside the chunk
        Parts<PK> fk[KS], fq[KS];
        const bool there = 16 * w + lr < len;
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            const int64_t o = ((row + 16 * w + lr) * a.HK + hk) * K + 32 * s + 8 * lg;
            fk[s] = load8<PK>(k + o, there && 32 * s + 8 * lg < K);
            fq[s] = load8<PK>(q + o, there && 32 * s + 8 * lg < K);
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            f4 kk = {}, qk = {};
            if (c <= w)
#pragma unroll
                for (int s = 0; s < KS; ++s) {
                    const Parts<PK> f = load8<PK>(k + ((row + 16 * c + lr) * a.HK + hk) * K + 32 * s + 8 * lg, 16 * c + lr < len && 32 * s + 8 * lg < K);
                    mma(kk, fk[s], f);
                    mma(qk, fq[s], f);
                }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int i = 16 * w + 4 * lg + e, j = 16 * c + lr;
                const float d = j <= i ? exp2f((float)(sG[i] - sG[j])) : 0.f;
                const float p = dP[c][e] * d, m = j < i ? -dA[c][e] * d : 0.f;
                sP[i * LA + j] = p;
                sA[i * LA + j] = m;
                sT[i * LH + j] = p * qk[e] + m * kk[e];
            }
        }
        // rows that read S, and rows that reach S'
        const f4 b = *reinterpret_cast<const f4 *>(dec + 16 * w + 4 * lg), end = *reinterpret_cast<const f4 *>(dec + C + 16 * w + 4 * lg);
        f4 reads = {}, ends = {};
#pragma unroll
        for (int c = 0; c < CT; ++c) {
            f4 qc = {}, kc = {};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int r = 16 * w + 4 * lg + e;
                if (r < len) {
                    qc[e] = to_f32(q[((row + r) * a.HK + hk) * K + 16 * c + lr]);
                    kc[e] = to_f32(k[((row + r) * a.HK + hk) * K + 16 * c + lr]);
                }
            }
            r1[c] *= b;
            r2[c] *= -b;
            r3[c] *= end;
            reads += qc * r1[c] + kc * r2[c];
            ends += kc * r3[c];
            dq[c] += r1[c];
            dk[c] += r2[c] + r3[c];
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            reads[e] = row16_sum(reads[e]);
            ends[e] = row16_sum(ends[e]);
            if (lr == 0) {
                sReads[16 * w + 4 * lg + e] = reads[e];
                sEnds[16 * w + 4 * lg + e] = ends[e];
            }
        }
        __syncthreads();
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            float pr[8], ar[8], pc[8], ac[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                pr[i] = sP[(16 * w + lr) * LA + 32 * s + 8 * lg + i];
                ar[i] = sA[(16 * w + lr) * LA + 32 * s + 8 * lg + i];
                pc[i] = sP[(32 * s + 8 * lg + i) * LA + 16 * w + lr];
                ac[i] = sA[(32 * s + 8 * lg + i) * LA + 16 * w + lr] + ar[i];
            }
            const Parts<P> fpr = cut8<P>(pr), fpc = cut8<P>(pc), fac = cut8<P>(ac);
#pragma unroll
            for (int c = 0; c < CT; ++c) {
                const Parts<PK> kt = load_frag<PK>(a.Kt + kq, c, s, lane), qt = load_frag<PK>(a.Qt + kq, c, s, lane);
                mma(dq[c], fpr, kt);
                mma(dk[c], fac, kt);
                mma(dk[c], fpc, qt);
            }
        }
        // dg: sums of the pairs in each row before t, then over the rows from t on
        if (tid < C) {
            float s = 0.f;
            for (int j = 0; j < C; ++j) {
                const float x = sT[tid * LH + j];
                sT[tid * LH + j] = s;
                s += x;
            }
        }
        __syncthreads();
        if (tid < C) {
            float s = 0.f;
            for (int i = C - 1; i >= tid; --i) s += sT[i * LH + tid];
            float from = sReads[tid], upto = sEnds[tid];
            const float own = upto;
#pragma unroll
            for (int d = 1; d < 64; d *= 2) {
                const float x = __shfl_down(from, d), y = __shfl_up(upto, d);
                if (tid + d < 64) from += x;
                if (tid >= d) upto += y;
            }
            const float last = dec[C - 1];
            if (tid < len) a.dg[(row + tid) * a.HV + hv] = s + from + (upto - own) + last * (sKeep[0] + sKeep[1] + sKeep[2] + sKeep[3]);
        }
        __syncthreads();
    }
#pragma unroll
    for (int c = 0; c < CT; ++c)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int r = 16 * w + 4 * lg + e;
            if (r < len) {
                const int64_t o = ((row + r) * a.HK + hk) * K + 16 * c + lr;
                st_out(a.dq, a.grad_bf16, o, dq[c][e]);
                st_out(a.dk, a.grad_bf16, o, dk[c][e]);
            }
        }
}

template <typename T, int K>
hipError_t launch(const GdrArgs &a, hipStream_t stream) {
    hipLaunchKernelGGL((gdr_bwd_chain_kernel<T, K>), dim3((unsigned)gdr_pair_blocks(a, a.V / 16)), dim3(256), 0, stream, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((gdr_grads_kernel<T, K>), dim3((unsigned)(a.slots * a.HK)), dim3(256), 0, stream, a);
    return hipGetLastError();
}
template <typename T>
hipError_t by_width(const GdrArgs &a, int K, hipStream_t stream) {
    switch (K) {
        case 16: return launch<T, 16>(a, stream);
        case 32: return launch<T, 32>(a, stream);
        case 64: return launch<T, 64>(a, stream);
        case 128: return launch<T, 128>(a, stream);
    }
    return hipErrorNotSupported;
}

}  // namespace

hipError_t launch_gdr_bwd(const GdrArgs &a, bool fp32, int K, hipStream_t stream) {
    hipError_t e = launch_gdr_prep(a, fp32, K, true, stream);
    if (e != hipSuccess) return e;
    e = launch_gdr_fwd_chain(a, fp32, K, true, stream);
    if (e != hipSuccess) return e;
    return fp32 ? by_width<float>(a, K, stream) : by_width<__bf16>(a, K, stream);
}

}  // namespace kda
