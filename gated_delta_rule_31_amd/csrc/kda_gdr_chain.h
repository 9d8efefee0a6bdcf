// The forward chain of the gated delta rule with one decay per value head (formulas and
// precision: kda_gdr.h), serial over a sequence's chunks and parallel over sequences, value heads
// and blocks of value columns: used by the prefill's own kernel and, beside the chain of
// gradients, by the backward pass.
#pragma once

#include "kda_gdr.h"

namespace kda {

// The chain.  One workgroup of four waves per (sequence, value head, 16 NV value columns).
// Wave w owns token rows 16w..16w+15 of the chunk and the state's channel tiles w, w + 4, ..;
// what the waves exchange (beta X, Vn, the state) goes through LDS as bf16 parts, columns first.
// The operands come from memory straight into the registers of the wave that uses them, each
// for the next chunk as soon as this chunk's product has read it, so that they are in flight
// over most of a chunk.  Rows behind the sequence's end read its last row: their beta is 0, so
// nothing of them reaches the state.
//
// Bound by the dependence of a chunk's three phases while a compute unit has one workgroup (2.2
// us a chunk, 8192 tokens x 32 heads, K = V = 128, bf16: 277 to 284 us), by the loads of the
// operands (68 KB a chunk and workgroup, mostly from L2) and instruction issue beyond (96 heads:
// 605 us, 1.3 GB from and to HBM).
//
// TRAIN: for the gradients; every chunk's start state and corrections are kept and there is no
// output.  The LDS arrays are the kernel's, with P = 3 parts: sS [P][16 NV][K], sX, sE and sV [P][16
// NV][64] (sV null for TRAIN), sK [parts of k][64][K], rows of 32 at K = 16.
template <typename T, typename OT, int K, int NV, bool TRAIN>
__device__ __forceinline__ void gdr_chain(const GdrArgs &a, int block, __bf16 *sS, __bf16 *sX, __bf16 *sE, __bf16 *sV, __bf16 *sK) {
    constexpr int C = GDR_C, P = GDR_PARTS, UNIT = TRAIN ? P * C * C : GDR_UNIT;
    constexpr int PK = gdr_input_parts<T>(), KP = K < 32 ? 32 : K, KS = KP / 32, NC = (K / 16 + 3) / 4, W = 16 * NV, SZ = sizeof(T);
    int vb, hv, n;
    if (!gdr_pair(a, block, a.V / W, vb, hv, n)) return;
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lr = lane & 15, lg = lane >> 4, hk = hv / a.group;
    int64_t row, len, slot;
    gdr_sequence(a, n, row, len, slot);
    const int64_t state = ((int64_t)n * a.HV + hv) * K * a.V + W * vb;

    if (K < 32) {
        for (int i = threadIdx.x; i < P * W * KP; i += 256) sS[i] = (__bf16)0.f;
        __syncthreads();
    }
    f4 S[NC][NV];
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int u = 0; u < NV; ++u) {
            S[c][u] = f4{};
            if (K % 64 == 0 || w + 4 * c < K / 16) {
                const int ch = 16 * (w + 4 * c) + 4 * lg;
                if (a.s0)
#pragma unroll
                    for (int e = 0; e < 4; ++e) S[c][u][e] = a.s0[state + (int64_t)(ch + e) * a.V + lr + 16 * u];
                lds_put4<P, W, KP>(sS, 16 * u + lr, ch, S[c][u]);
            }
        }

    const int chunks = (int)((len + C - 1) / C);
    // byte strides of a token, and this lane's offsets from a chunk's first token
    const unsigned kstep = (unsigned)a.HK * K * SZ, vstep = (unsigned)a.HV * a.V * SZ, ostep = (unsigned)a.HV * a.V * sizeof(OT);
    const char *kbase = static_cast<const char *>(a.k) + (row * a.HK + hk) * (K * SZ), *qbase = static_cast<const char *>(a.q) + (row * a.HK + hk) * (K * SZ);
    const char *vbase = static_cast<const char *>(a.v) + ((row * a.HV + hv) * a.V + W * vb) * SZ;
    char *obase = static_cast<char *>(a.out) + ((row * a.HV + hv) * a.V + W * vb) * sizeof(OT);
    const unsigned kcol = (K < 32 ? lg % 2 * 8 : 8 * lg) * SZ;  // beside a width of 16 the state's parts are zero
    const unsigned krow = (16 * w + lr) * kstep + kcol, r0 = 16 * w + 4 * lg;
    Parts<PK> k[KS], q[KS];
    Parts<P> m[2], p[2];
    // rows 0..31 have nothing in M's and P's second 32 columns: waves 0 and 1 multiply zeros that they
    // hold, while the others work, so that a phase has no branches and its parts are interleaved
    m[1] = p[1] = Parts<P>{};
    f4 b, end, beta, nb, nend, nbeta;
    Parts<PK> v, nv;
    bf16x8 one[NV];
#pragma unroll
    for (int u = 0; u < NV; ++u)
#pragma unroll
        for (int i = 0; i < 8; ++i) one[u][i] = (__bf16)(8 * lg + i == 16 * u + lr ? 1.f : 0.f);
    const unsigned vcol = (NV == 1 ? lg % 2 * 8 : 8 * lg) * SZ;
    float last, nlast, blr, nblr;
    auto load_kq = [&](int c) {
        const int64_t t = (int64_t)c * C;
        unsigned at = krow;
        if (t + C > len) at = (unsigned)(16 * w + lr < len - t ? 16 * w + lr : len - t - 1) * kstep + kcol;
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            k[s] = load8<PK>(reinterpret_cast<const T *>(kbase + t * kstep + at + 32 * s * SZ), true);
            if (!TRAIN) q[s] = load8<PK>(reinterpret_cast<const T *>(qbase + t * kstep + at + 32 * s * SZ), true);
        }
    };
    auto load_m = [&](int c) {
        const __bf16 *from = a.M + ((slot + c) * a.HV + hv) * UNIT;
#pragma unroll
        for (int s = 0; s < 2; ++s)
            if (s == 0 || w >= 2) m[s] = load_frag<P>(from, gdr_lower(w, s), lane);
    };
    auto load_p = [&](int c) {
        const __bf16 *from = a.M + ((slot + c) * a.HV + hv) * UNIT + GDR_P_AT;
#pragma unroll
        for (int s = 0; s < 2; ++s)
            if (!TRAIN && (s == 0 || w >= 2)) p[s] = load_frag<P>(from, gdr_lower(w, s), lane);
    };
    auto load_rows = [&](int c) {  // into the second set
        const float *dec = a.dec + ((slot + c) * a.HV + hv) * (4 * C);
        nb = at_offset<f4>(dec, r0 * 4);
        nend = at_offset<f4>(dec + C, r0 * 4);
        nbeta = at_offset<f4>(dec + 2 * C, r0 * 4);
        nlast = dec[C - 1];
        nblr = at_offset<float>(dec, (16 * w + lr) * 4);
        const int64_t t = (int64_t)c * C;
        const unsigned r = 16 * w + lr < len - t ? 16 * w + lr : (unsigned)(len - t - 1);
        nv = load8<PK>(reinterpret_cast<const T *>(vbase + t * vstep + (r * vstep + vcol)), true);
    };
    if (chunks > 0) {
        load_rows(0);
        load_kq(0);
        load_m(0);
        load_p(0);
    }
    for (int c = 0; c < chunks; ++c) {
        const int next = c + 1 < chunks ? c + 1 : c;
        b = nb, end = nend, beta = nbeta, last = nlast, blr = nblr;
        v = nv;
        load_rows(next);
        if (TRAIN) {
            float *h = a.h + ((slot + c) * a.HV + hv) * ((int64_t)K * a.V) + gdr_slice_at(K, W * vb, a.V);
#pragma unroll
            for (int i = 0; i < NC; ++i)
                if (K % 64 == 0 || w + 4 * i < K / 16)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
#pragma unroll
                        for (int u = 0; u < NV; ++u) h[(16 * (w + 4 * i) + 4 * lg + e) * gdr_slice_columns(a.V) + lr + 16 * u] = S[i][u][e];
        }
        gdr_lds_barrier();
        // K's rows also go to LDS, where the state's update reads them by columns
#pragma unroll
        for (int s = 0; s < KS; ++s)
#pragma unroll
            for (int i = 0; i < PK; ++i) *reinterpret_cast<bf16x8 *>(sK + i * C * KP + lds_at<KP>(16 * w + lr, 32 * s + 8 * lg)) = k[s].v[i];
        f4 x[NV], y[NV];
#pragma unroll
        for (int u = 0; u < NV; ++u) x[u] = y[u] = f4{};
#pragma unroll
        for (int s = 0; s < KS; ++s)
#pragma unroll
            for (int u = 0; u < NV; ++u) {
                const Parts<P> f = lds_frag<P, W, KP>(sS, 16 * u + lr, 32 * s + 8 * lg);
                mma(x[u], k[s], f);
                if (!TRAIN) mma(y[u], f, q[s]);  // columns by tokens: a lane gets four columns of a token
            }
        load_kq(next);
#pragma unroll
        for (int u = 0; u < NV; ++u) {
            x[u] *= -b;
            mma(x[u], v, Parts<1>{{one[u]}});
            lds_put4<P, W, C>(sX, 16 * u + lr, r0, beta * x[u]);
        }
        gdr_lds_barrier();
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int u = 0; u < NV; ++u) mma(x[u], m[s], lds_frag<P, W, C>(sX, 16 * u + lr, 32 * s + 8 * lg));
        load_m(next);
#pragma unroll
        for (int u = 0; u < NV; ++u) {
            const f4 vn = beta * x[u];
            lds_put4<P, W, C>(sE, 16 * u + lr, r0, end * vn);
            if (!TRAIN) lds_put4<P, W, C>(sV, 16 * u + lr, r0, vn);
        }
        gdr_lds_barrier();
#pragma unroll
        for (int i = 0; i < NC; ++i)
            if (K % 64 == 0 || w + 4 * i < K / 16) {
                Parts<PK> kt[2];
#pragma unroll
                for (int s = 0; s < 2; ++s) kt[s] = lds_frag_turned<PK, C, KP>(sK, 32 * s + 8 * lg, 16 * (w + 4 * i), lane);
#pragma unroll
                for (int u = 0; u < NV; ++u) {
                    S[i][u] *= last;
#pragma unroll
                    for (int s = 0; s < 2; ++s) mma(S[i][u], kt[s], lds_frag<P, W, C>(sE, 16 * u + lr, 32 * s + 8 * lg));
                    lds_put4<P, W, KP>(sS, 16 * u + lr, 16 * (w + 4 * i) + 4 * lg, S[i][u]);
                }
            }
        const int64_t t = (int64_t)c * C;
        if (TRAIN) {
            float *d = a.delta + ((slot + c) * a.HV + hv) * ((int64_t)C * a.V) + gdr_slice_at(C, W * vb, a.V);
#pragma unroll
            for (int e = 0; e < 4; ++e)
#pragma unroll
                for (int u = 0; u < NV; ++u) d[(r0 + e) * gdr_slice_columns(a.V) + lr + 16 * u] = x[u][e];
        } else {
#pragma unroll
            for (int u = 0; u < NV; ++u) {
                y[u] *= blr;
#pragma unroll
                for (int s = 0; s < 2; ++s)
                    mma(y[u], lds_frag<P, W, C>(sV, 16 * u + lr, 32 * s + 8 * lg), p[s]);
                y[u] *= a.scale;
            }
            load_p(next);
            char *to = obase + t * ostep;
            typedef __attribute__((ext_vector_type(4))) OT ot4;
            if (16 * w + lr < len - t)
#pragma unroll
                for (int u = 0; u < NV; ++u)
                    *reinterpret_cast<ot4 *>(to + ((16 * w + lr) * ostep + (16 * u + 4 * lg) * (unsigned)sizeof(OT))) = __builtin_convertvector(y[u], ot4);
        }
    }
    if (!TRAIN && a.sf)
#pragma unroll
        for (int i = 0; i < NC; ++i)
            if (K % 64 == 0 || w + 4 * i < K / 16)
#pragma unroll
                for (int e = 0; e < 4; ++e)
#pragma unroll
                    for (int u = 0; u < NV; ++u) a.sf[state + (int64_t)(16 * (w + 4 * i) + 4 * lg + e) * a.V + lr + 16 * u] = S[i][u][e];
}

}  // namespace kda
