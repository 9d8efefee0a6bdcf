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
// Three kernels: the pre-pass (kda_gdr_fwd.hip); in one launch the forward chain
// (kda_gdr_chain.h), which keeps every chunk's start state and delta, and the chain of
// gradients, serial backwards over the chunks; and one workgroup per (chunk, key head) for the rest, which goes through the value heads of
// its group, so that the shared heads' gradients are summed in a fixed order.  Computed
// operands enter the matrix cores as three bf16 parts (24 bits).
#include "kda_gdr_chain.h"

namespace kda {
namespace {

constexpr int C = GDR_C, P = GDR_PARTS;

// The chain of gradients: workgroups, waves and operands in flight as in the forward chain, and
// bound alike.  Both chains together, 8192 tokens x 32 heads, K = V = 128, bf16: 718 us, 0.6 GB
// read and 0.9 GB written.
// D: the type of d_out, whose parts are exact until the read's scale meets them.
template <typename T, typename D, int K, int NV>
__device__ __forceinline__ void gdr_bwd_chain(const GdrArgs &a, int block, __bf16 *sS, __bf16 *sX, __bf16 *sE, __bf16 *sB, __bf16 *sK, __bf16 *sQ, __bf16 *sO) {
    constexpr int PK = gdr_input_parts<T>(), PD = gdr_input_parts<D>(), KP = K < 32 ? 32 : K, KS = KP / 32, NC = (K / 16 + 3) / 4, W = 16 * NV;
    constexpr int SZ = sizeof(T), DZ = sizeof(D);
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
    for (int i = 0; i < NC; ++i)
#pragma unroll
        for (int u = 0; u < NV; ++u) {
            S[i][u] = f4{};
            if (K % 64 == 0 || w + 4 * i < K / 16) {
                const int ch = 16 * (w + 4 * i) + 4 * lg;
                if (a.d_sf)
#pragma unroll
                    for (int e = 0; e < 4; ++e) S[i][u][e] = a.d_sf[state + (int64_t)(ch + e) * a.V + lr + 16 * u];
                lds_put4<P, W, KP>(sS, 16 * u + lr, ch, S[i][u]);
            }
        }
    const int chunks = (int)((len + C - 1) / C);
    const unsigned kstep = (unsigned)a.HK * K * SZ, ostep = (unsigned)a.HV * a.V * DZ;
    const char *kbase = static_cast<const char *>(a.k) + (row * a.HK + hk) * (K * SZ), *qbase = static_cast<const char *>(a.q) + (row * a.HK + hk) * (K * SZ);
    const char *obase = static_cast<const char *>(a.d_out) + ((row * a.HV + hv) * a.V + W * vb) * DZ;
    const unsigned kcol = (K < 32 ? lg % 2 * 8 : 8 * lg) * SZ, ocol = (NV == 1 ? lg % 2 * 8 : 8 * lg) * DZ, r0 = 16 * w + 4 * lg;
    bf16x8 one[NV];  // d_out enters as operands, eight columns of a row a lane: dO = dO 1
#pragma unroll
    for (int u = 0; u < NV; ++u)
#pragma unroll
        for (int i = 0; i < 8; ++i) one[u][i] = (__bf16)(8 * lg + i == 16 * u + lr ? 1.f : 0.f);
    Parts<PK> k[KS], q[KS];
    Parts<P> m[2], p[2];
    Parts<PD> o;
    m[0] = p[0] = Parts<P>{};  // rows 32..63 have nothing in the first 32 columns of M^T and P^T
    f4 b, end, beta;
    float last;
    // rows behind the sequence's end read its last row, and what P^T, M^T and the keys hold there meets
    // zeros: d_out is taken as 0, and beta is 0
    auto load_kqo = [&](int c) {
        const int64_t t = (int64_t)c * C;
        const bool there = 16 * w + lr < len - t;
        const unsigned r = there ? 16 * w + lr : (unsigned)(len - t - 1);
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            k[s] = load8<PK>(reinterpret_cast<const T *>(kbase + t * kstep + (r * kstep + kcol) + 32 * s * SZ), true);
            q[s] = load8<PK>(reinterpret_cast<const T *>(qbase + t * kstep + (r * kstep + kcol) + 32 * s * SZ), true);
        }
        o = load8<PD>(reinterpret_cast<const D *>(obase + t * ostep + (r * ostep + ocol)), there);
    };
    auto load_frags = [&](const __bf16 *base, Parts<P> (&f)[2], int c) {
        const __bf16 *from = base + ((slot + c) * a.HV + hv) * (P * C * C);
#pragma unroll
        for (int s = 0; s < 2; ++s)
            if (s == 1 || w < 2) f[s] = load_frag<P>(from, gdr_full(w, s), lane);
    };
    auto load_dec = [&](int c) {
        const float *dec = a.dec + ((slot + c) * a.HV + hv) * (4 * C);
        b = at_offset<f4>(dec, r0 * 4);
        end = at_offset<f4>(dec + C, r0 * 4);
        beta = at_offset<f4>(dec + 2 * C, r0 * 4);
        last = dec[C - 1];
    };
    if (chunks > 0) {
        load_kqo(chunks - 1);
        load_frags(a.P, p, chunks - 1);
        load_dec(chunks - 1);
        load_frags(a.Mt, m, chunks - 1);
    }
    for (int c = chunks - 1; c >= 0; --c) {
        const int next = c > 0 ? c - 1 : 0;
        const int64_t at = (slot + c) * a.HV + hv, t = (int64_t)c * C;
        float *dh = a.dh + at * ((int64_t)K * a.V) + gdr_slice_at(K, W * vb, a.V);
#pragma unroll
        for (int i = 0; i < NC; ++i)
            if (K % 64 == 0 || w + 4 * i < K / 16)
#pragma unroll
                for (int e = 0; e < 4; ++e)
#pragma unroll
                    for (int u = 0; u < NV; ++u) dh[(16 * (w + 4 * i) + 4 * lg + e) * gdr_slice_columns(a.V) + lr + 16 * u] = S[i][u][e];
#pragma unroll
        for (int i = 0; i < PD; ++i) *reinterpret_cast<bf16x8 *>(sO + i * C * 32 + lds_at<32>(16 * w + lr, 8 * lg)) = o.v[i];
        gdr_lds_barrier();
        // behind the barrier: until then other waves may still read the rows of the chunk before (the
        // rows of d_out are read by none of them behind that chunk's second barrier)
#pragma unroll
        for (int s = 0; s < KS; ++s)
#pragma unroll
            for (int i = 0; i < PK; ++i) {
                *reinterpret_cast<bf16x8 *>(sK + i * C * KP + lds_at<KP>(16 * w + lr, 32 * s + 8 * lg)) = k[s].v[i];
                *reinterpret_cast<bf16x8 *>(sQ + i * C * KP + lds_at<KP>(16 * w + lr, 32 * s + 8 * lg)) = q[s].v[i];
            }
        f4 x[NV], y[NV], d[NV];
#pragma unroll
        for (int u = 0; u < NV; ++u) {
            x[u] = y[u] = d[u] = f4{};
            mma(d[u], o, Parts<1>{{one[u]}});
        }
#pragma unroll
        for (int s = 0; s < KS; ++s)
#pragma unroll
            for (int u = 0; u < NV; ++u) mma(x[u], k[s], lds_frag<P, W, KP>(sS, 16 * u + lr, 32 * s + 8 * lg));
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int u = 0; u < NV; ++u) mma(y[u], p[s], lds_frag_turned<PD, C, 32>(sO, 32 * s + 8 * lg, 16 * u, lane));
        load_kqo(next);
        load_frags(a.P, p, next);
#pragma unroll
        for (int u = 0; u < NV; ++u) {
            x[u] = end * x[u] + a.scale * y[u];
            lds_put4<P, W, C>(sX, 16 * u + lr, r0, beta * x[u]);
            lds_put4<P, W, C>(sB, 16 * u + lr, r0, a.scale * b * d[u]);
        }
        gdr_lds_barrier();
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int u = 0; u < NV; ++u) mma(x[u], m[s], lds_frag<P, W, C>(sX, 16 * u + lr, 32 * s + 8 * lg));
        load_frags(a.Mt, m, next);
        f4 E[NV];
#pragma unroll
        for (int u = 0; u < NV; ++u) {
            E[u] = beta * x[u];
            lds_put4<P, W, C>(sE, 16 * u + lr, r0, -(b * E[u]));
        }
#pragma unroll
        for (int i = 0; i < NC; ++i)
#pragma unroll
            for (int u = 0; u < NV; ++u) S[i][u] *= last;
        load_dec(next);
        gdr_lds_barrier();
#pragma unroll
        for (int i = 0; i < NC; ++i)
            if (K % 64 == 0 || w + 4 * i < K / 16) {
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    const Parts<PK> qt = lds_frag_turned<PK, C, KP>(sQ, 32 * s + 8 * lg, 16 * (w + 4 * i), lane);
                    const Parts<PK> kt = lds_frag_turned<PK, C, KP>(sK, 32 * s + 8 * lg, 16 * (w + 4 * i), lane);
#pragma unroll
                    for (int u = 0; u < NV; ++u) {
                        mma(S[i][u], qt, lds_frag<P, W, C>(sB, 16 * u + lr, 32 * s + 8 * lg));
                        mma(S[i][u], kt, lds_frag<P, W, C>(sE, 16 * u + lr, 32 * s + 8 * lg));
                    }
                }
#pragma unroll
                for (int u = 0; u < NV; ++u) lds_put4<P, W, KP>(sS, 16 * u + lr, 16 * (w + 4 * i) + 4 * lg, S[i][u]);
            }
        float *dY = a.dY + at * ((int64_t)C * a.V) + gdr_slice_at(C, W * vb, a.V);
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
            for (int u = 0; u < NV; ++u) {
                dY[(r0 + e) * gdr_slice_columns(a.V) + lr + 16 * u] = x[u][e];
                if (r0 + e < len - t) st_out(a.dv, a.grad_bf16, ((row + t + r0 + e) * a.HV + hv) * a.V + W * vb + lr + 16 * u, E[u][e]);
            }
    }
    if (a.ds0)
#pragma unroll
        for (int i = 0; i < NC; ++i)
            if (K % 64 == 0 || w + 4 * i < K / 16)
#pragma unroll
                for (int e = 0; e < 4; ++e)
#pragma unroll
                    for (int u = 0; u < NV; ++u) a.ds0[state + (int64_t)(16 * (w + 4 * i) + 4 * lg + e) * a.V + lr + 16 * u] = S[i][u][e];
}

// Both chains in one launch: neither needs the other's results, each waits most of its time, and
// a compute unit has room for a workgroup of both.  Groups of eight blocks (one an XCD) take them
// in turn.  Two workgroups a compute unit where the LDS allows it: without that bound the compiler
// takes 264 registers instead of 256 and one fits (1360 against 1262 us for the layer's call).
template <typename T, typename D, int K, int NV>
__global__ __launch_bounds__(256, sizeof(T) == 2 && NV == 1 ? 2 : 1) void gdr_chains_kernel(const GdrArgs a) {
    constexpr int PK = gdr_input_parts<T>(), PD = gdr_input_parts<D>(), KP = K < 32 ? 32 : K, W = 16 * NV;
    __shared__ __attribute__((aligned(16))) __bf16 sS[P * W * KP], sX[P * W * C], sE[P * W * C], sB[P * W * C], sK[PK * C * KP], sQ[PK * C * KP], sO[PD * C * 32];
    const int block = blockIdx.x / 16 * 8 + blockIdx.x % 8;
    if (blockIdx.x / 8 % 2 == 0) gdr_bwd_chain<T, D, K, NV>(a, block, sS, sX, sE, sB, sK, sQ, sO);
    else gdr_chain<T, float, K, NV, true>(a, block, sS, sX, sE, nullptr, sK);
}

// Columns 4 g .. + 3 and 16 + 4 g .. + 3 of a row's 32-column slice: lanes next to each other read
// addresses next to each other, and the products over the slice take their operands' columns in
// this order (staged_at).  The loads are unconditional (a slice of 16 columns reads its first
// quads twice) and nothing is done with what they bring until it is used: a condition or a
// conversion here would wait for them.
template <typename D>
struct Slice8 {
    typedef __attribute__((ext_vector_type(4))) D d4;
    d4 x[2];
    __device__ __forceinline__ void load(const void *p, unsigned bytes, int g, int columns) {
        x[0] = at_offset<d4>(p, bytes + 4 * g * (unsigned)sizeof(D));
        x[1] = at_offset<d4>(p, bytes + (4 * g + (columns > 16 ? 16 : 0)) * (unsigned)sizeof(D));
    }
    __device__ __forceinline__ void get(float (&y)[8], int columns) const {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            y[i] = (float)x[0][i];
            y[4 + i] = columns > 16 ? (float)x[1][i] : 0.f;
        }
    }
    // as operand parts, zeros where !there
    __device__ __forceinline__ Parts<gdr_input_parts<D>()> parts(int columns, bool there) const {
        if constexpr (sizeof(D) == 2) {
            const u32x2 u = there ? __builtin_bit_cast(u32x2, x[0]) : u32x2{}, v = there && columns > 16 ? __builtin_bit_cast(u32x2, x[1]) : u32x2{};
            return {{__builtin_bit_cast(bf16x8, u32x4{u[0], u[1], v[0], v[1]})}};
        } else {
            float y[8];
            get(y, columns);
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = there ? y[i] : 0.f;
            return cut8<gdr_input_parts<D>()>(y);
        }
    }
};
__device__ __forceinline__ int staged_at(int row, int quad) { return lds_at<32>(row, quad % 4 * 8 + quad / 4 * 4); }

// One workgroup of eight waves per (chunk slot, key head).  Wave (w, h) owns token rows
// 16w..16w+15 and the h-th half of the channels; of the C x C products, h = 0 has dP and h = 1
// dA.  The products over V go through LDS in slices of 32 columns, the next slice's rows on
// their way meanwhile.  Bound by issue: cutting float32 states and rows into parts takes the vector
// units about 40% of the time, the products the matrix cores 23% (8192 tokens x 32 heads, K = V =
// 128, bf16: 424 us, 1.05 GB read; its first form, four waves that spilled, took 843 us).
template <typename T, typename D, int K>
__global__ __launch_bounds__(512) void gdr_grads_kernel(const GdrArgs a) {
    constexpr int PK = gdr_input_parts<T>(), PD = gdr_input_parts<D>(), KS = K < 32 ? 1 : K / 32, CT = (K / 16 + 1) / 2, LA = C + 4, KP = K < 32 ? 32 : K, QUADS = K * 8 / 512 ? K * 8 / 512 : 1;
    constexpr bool KQ = PK == 1;  // k and q rows stay in LDS over the heads of a group where they fit
    __shared__ __attribute__((aligned(16))) __bf16 sS[P * K * 32], sH[P * K * 32], sV[P * C * 32], sE[P * C * 32];
    __shared__ __attribute__((aligned(16))) float sP[C * LA], sA[C * LA], sT[C * LA], sSum[2][4][C], sReads[2][2][C], sEnds[2][2][C], sKeep[2][8];
    __shared__ __attribute__((aligned(16))) __bf16 sK[KQ ? C * KP : 8], sQ[KQ ? C * KP : 8];
    __shared__ double sG[C];
    const int unit = blockIdx.x, hk = unit % a.HK;
    const int64_t slot = unit / a.HK;
    int64_t row;
    int len;
    const int w8 = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), w = w8 & 3, half = w8 >> 2;
    if (a.cu) {
        // rows behind the last sequence have no gradient: each slot clears 64 of them, the last slot
        // the first ones.  There are T / 64 + N slots, enough for all T rows, and those counted from
        // the last one hold no chunk, but for one at most.  1000 of 8192 rows used, 16 key and 32 value
        // heads, K = V = 128, bf16: 196 us a call, 185 for the 1000 rows alone; with one workgroup a
        // key head that clears all of them, above 2000.
        int64_t l, s;
        gdr_sequence(a, a.N - 1, row, l, s);
        const int64_t first = row + l + (a.slots - 1 - slot) * C;
        const unsigned es = a.grad_bf16 ? 2 : 4;
        auto clear = [&](void *x, int64_t at, unsigned n) {  // n elements of a row, on 16-byte borders
            char *to = static_cast<char *>(x) + at * es;
            for (unsigned b = (threadIdx.x & 63) * 16; b < n * es; b += 1024) *reinterpret_cast<f4 *>(to + b) = f4{};
        };
        for (int64_t t = first + w8; t < first + C && t < a.T; t += 8) {
            clear(a.dq, (t * a.HK + hk) * K, K);
            clear(a.dk, (t * a.HK + hk) * K, K);
            clear(a.dv, (t * a.HV + hk * a.group) * a.V, a.group * a.V);
            for (int h = threadIdx.x & 63; h < a.group; h += 64) a.dg[t * a.HV + hk * a.group + h] = a.dbeta[t * a.HV + hk * a.group + h] = 0.f;
        }
    }
    if (!gdr_chunk(a, slot, row, len)) return;
    const int V = a.V, slices = (V + 31) / 32;
    // addresses are one of the wave's and a lane's 32-bit offset; rows behind the end read the last
    // row, where dO is taken as 0 and beta is 0
    const T *q = static_cast<const T *>(a.q) + (row * a.HK + hk) * K, *k = static_cast<const T *>(a.k) + (row * a.HK + hk) * K;
    const unsigned kstep = (unsigned)a.HK * K * sizeof(T), dstep = (unsigned)a.HV * V * sizeof(D);
    auto clamped = [&](int i) { return (unsigned)(i < len ? i : len - 1); };
    auto at8 = [](const T *x, unsigned bytes) { return reinterpret_cast<const T *>(reinterpret_cast<const char *>(x) + bytes); };
    const int64_t kq = (slot * a.HK + hk) * (PK * K * C);

    if constexpr (KQ)
        for (int i = threadIdx.x; i < C * K / 8; i += 512) {
            const int j = i / (K / 8), c = i % (K / 8) * 8;
            *reinterpret_cast<bf16x8 *>(sK + lds_at<KP>(j, c)) = load8<1>(at8(k, clamped(j) * kstep + c * (unsigned)sizeof(T)), true).v[0];
            *reinterpret_cast<bf16x8 *>(sQ + lds_at<KP>(j, c)) = load8<1>(at8(q, clamped(j) * kstep + c * (unsigned)sizeof(T)), true).v[0];
        }
    // a slice's rows on their way: corrections, dY and d_out of this lane's row, four columns each of
    // rows of the two states
    Slice8<float> raw_v, raw_e;
    Slice8<D> raw_o;
    float raw_beta;
    f4 hx[QUADS], hy[QUADS];
    auto load = [&](int hv, int sl, int tid) {
        const int64_t at = slot * a.HV + hv;
        const int lane = tid & 63, r = 16 * w + (lane & 15), lg = lane >> 4, left = V - 32 * sl, width = gdr_slice_columns(V);
        const char *dO = static_cast<const char *>(a.d_out) + ((row * a.HV + hv) * V + 32 * sl) * (int64_t)sizeof(D);
        raw_v.load(a.delta + at * ((int64_t)C * V) + C * 32 * sl, r * width * 4u, lg, left);
        raw_e.load(a.dY + at * ((int64_t)C * V) + C * 32 * sl, r * width * 4u, lg, left);
        raw_o.load(dO, clamped(r) * dstep, lg, left);
        raw_beta = at_offset<float>(a.dec + at * 4 * C, (2 * C + r) * 4u);
        const float *h = a.h + at * ((int64_t)K * V) + K * 32 * sl, *dh = a.dh + at * ((int64_t)K * V) + K * 32 * sl;
#pragma unroll
        for (int j = 0; j < QUADS; ++j) {
            const int i = (tid + 512 * j) % (K * 8);
            const unsigned from = (i / 8 * width + i % 8 * 4 % width) * 4u;
            hx[j] = at_offset<f4>(h, from);
            hy[j] = at_offset<f4>(dh, from);
        }
    };
    load(hk * a.group, 0, threadIdx.x);
    f4 dq[CT], dk[CT];
#pragma unroll
    for (int c = 0; c < CT; ++c) dq[c] = dk[c] = f4{};
    for (int hv = hk * a.group; hv < (hk + 1) * a.group; ++hv) {
        // the lane is read anew for each head: what follows from it (a hundred offsets) would else be
        // formed once ahead of the loop and spilled
        int tid = threadIdx.x;
        asm volatile("" : "+v"(tid));
        const int lane = tid & 63, lr = lane & 15, lg = lane >> 4, r = 16 * w + lr;
        const int64_t at = slot * a.HV + hv;
        const float *dec = a.dec + at * 4 * C;
        const double g = a.G[at * C + lane];
        const int turn = hv & 1;  // sums of one head are read while the next is on its way
        f4 r1[CT], r2[CT], r3[CT], pair[4];
#pragma unroll
        for (int c = 0; c < CT; ++c) r1[c] = r2[c] = r3[c] = f4{};
#pragma unroll
        for (int c = 0; c < 4; ++c) pair[c] = f4{};
        float keep = 0.f, db = 0.f;
        for (int sl = 0; sl < slices; ++sl) {
            const int left = V - 32 * sl;
            const float beta_r = raw_beta;
            // half 0 cuts the corrections and half 1 the rows of E; both take both from LDS
            float xe[8], x[8];
            raw_e.get(xe, left);
            if (half == 0) {
                raw_v.get(x, left);
#pragma unroll
                for (int i = 0; i < 8; ++i) db += xe[i] * x[i];
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] = xe[i];
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] *= beta_r;
            const Parts<P> mine = cut8<P>(x);
            const Parts<PD> fd = raw_o.parts(left, r < len);
            unsigned cx[QUADS][2][P], cy[QUADS][2][P];
#pragma unroll
            for (int j = 0; j < QUADS; ++j) {
                if (tid + 512 * j >= K * 8 || (tid + 512 * j) % 8 * 4 >= left) hx[j] = hy[j] = f4{};
#pragma unroll
                for (int e = 0; e < 4; ++e) keep += hx[j][e] * hy[j][e];
                cut2<P>(hx[j][0], hx[j][1], cx[j][0]);
                cut2<P>(hx[j][2], hx[j][3], cx[j][1]);
                cut2<P>(hy[j][0], hy[j][1], cy[j][0]);
                cut2<P>(hy[j][2], hy[j][3], cy[j][1]);
            }
            // the next slice, or the next head's first (the last head's again at the end): one call
            // without a condition, or the registers would be copied, and the copy waits
            __builtin_amdgcn_sched_barrier(0);
            load(sl + 1 < slices || hv + 1 == (hk + 1) * a.group ? hv : hv + 1, sl + 1 < slices ? sl + 1 : 0, tid);
            gdr_lds_barrier();  // the last slice has been read
            if (sl == 0 && w8 == 0) sG[lane] = g;
#pragma unroll
            for (int p = 0; p < P; ++p) *reinterpret_cast<bf16x8 *>((half == 0 ? sV : sE) + p * C * 32 + lds_at<32>(r, 8 * lg)) = mine.v[p];
#pragma unroll
            for (int j = 0; j < QUADS; ++j) {
                const int i = tid + 512 * j;
                if (i < K * 8)
#pragma unroll
                    for (int p = 0; p < P; ++p) {
                        *reinterpret_cast<u32x2 *>(sS + p * K * 32 + staged_at(i / 8, i % 8)) = u32x2{cx[j][0][p], cx[j][1][p]};
                        *reinterpret_cast<u32x2 *>(sH + p * K * 32 + staged_at(i / 8, i % 8)) = u32x2{cy[j][0][p], cy[j][1][p]};
                    }
            }
            gdr_lds_barrier();
            const Parts<P> fv = lds_frag<P, C, 32>(sV, r, 8 * lg), fe = lds_frag<P, C, 32>(sE, r, 8 * lg);
            Parts<P> fpair = fe;  // the whole square of pairs, with no branch: what is above the diagonal is dropped
            if (half == 0)
#pragma unroll
                for (int p = 0; p < P; ++p) fpair.v[p] = p < PD ? fd.v[p < PD ? p : 0] : bf16x8{};
#pragma unroll
            for (int c = 0; c < CT; ++c)
                if (K % 32 == 0 || half * CT + c < K / 16) {
                    const int ch = 16 * (half * CT + c) + lr;
                    const Parts<P> s = lds_frag<P, K, 32>(sS, ch, 8 * lg), d = lds_frag<P, K, 32>(sH, ch, 8 * lg);
                    mma(r1[c], fd, s);
                    mma(r2[c], fe, s);
                    mma(r3[c], fv, d);
                }
#pragma unroll
            for (int c = 0; c < 4; ++c) mma(pair[c], fpair, lds_frag<P, C, 32>(sV, 16 * c + lr, 8 * lg));
        }
        // dbeta: a row's eight-column pieces lie in lanes 16 apart
        db += __shfl_xor(db, 16);
        db += __shfl_xor(db, 32);
        if (half == 0 && lg == 0 && r < len) a.dbeta[(row + r) * a.HV + hv] = db;
#pragma unroll
        for (int d = 32; d; d /= 2) keep += __shfl_xor(keep, d);
        if (lane == 0) sKeep[turn][w8] = keep;

        // the pairs inside the chunk: dP and its share of H, then dA and its
        f4 share[4];
        Parts<PK> f[KS];
        auto rows = [&](const T *x, const __bf16 *tile, int i, int s) {
            if constexpr (KQ) {
                const Parts<PK> y = lds_frag<PK, C, KP>(tile, i, K < 32 ? lg % 2 * 8 : 32 * s + 8 * lg);
                return K < 32 && lg > 1 ? Parts<PK>{} : y;
            } else
                return load8<PK>(at8(x, clamped(i) * kstep + (K < 32 ? lg % 2 * 8 : 32 * s + 8 * lg) * (unsigned)sizeof(T)), K >= 32 || lg < 2);
        };
#pragma unroll
        for (int s = 0; s < KS; ++s) f[s] = rows(half == 0 ? q : k, half == 0 ? sQ : sK, r, s);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            f4 dot = {};
            if (c <= w) {
#pragma unroll
                for (int s = 0; s < KS; ++s) mma(dot, f[s], rows(k, sK, 16 * c + lr, s));
            }
            if (!KQ) __builtin_amdgcn_sched_barrier(0);  // else the loads of all tiles are in registers at once
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int i = 16 * w + 4 * lg + e, j = 16 * c + lr;
                const float d = j < i + (half == 0) ? __builtin_amdgcn_exp2f((float)(sG[i] - sG[j])) : 0.f;
                const float x = c <= w ? pair[c][e] * (half == 0 ? a.scale * d : -d) : 0.f;
                (half == 0 ? sP : sA)[i * LA + j] = x;
                share[c][e] = x * dot[e];
                if (half == 0) sT[i * LA + j] = share[c][e];
            }
        }
        // rows that read S, and rows that reach S'
        const f4 b = *reinterpret_cast<const f4 *>(dec + 16 * w + 4 * lg), end = *reinterpret_cast<const f4 *>(dec + C + 16 * w + 4 * lg);
        f4 reads = {}, ends = {};
#pragma unroll
        for (int c = 0; c < CT; ++c)
            if (K % 32 == 0 || half * CT + c < K / 16) {
                f4 qc, kc;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int i = 16 * w + 4 * lg + e, ch = 16 * (half * CT + c) + lr;
                    if constexpr (KQ) {
                        qc[e] = (float)sQ[lds_at<KP>(i, ch)];
                        kc[e] = (float)sK[lds_at<KP>(i, ch)];
                    } else {
                        qc[e] = to_f32(*at8(q, clamped(i) * kstep + ch * (unsigned)sizeof(T)));
                        kc[e] = to_f32(*at8(k, clamped(i) * kstep + ch * (unsigned)sizeof(T)));
                    }
                }
                r1[c] *= a.scale * b;
                r2[c] *= -b;
                r3[c] *= end;
                reads += qc * r1[c] + kc * r2[c];
                ends += kc * r3[c];
                dq[c] += r1[c];
                dk[c] += r2[c] + r3[c];
            }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float x = row16_sum(reads[e]), y = row16_sum(ends[e]);
            if (lr == 0) {
                sReads[turn][half][16 * w + 4 * lg + e] = x;
                sEnds[turn][half][16 * w + 4 * lg + e] = y;
            }
        }
        __syncthreads();
        if (half == 1)
#pragma unroll
            for (int c = 0; c < 4; ++c)
#pragma unroll
                for (int e = 0; e < 4; ++e) sT[(16 * w + 4 * lg + e) * LA + 16 * c + lr] += share[c][e];
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            float pr[8], ar[8], pc[8], ac[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                pr[i] = sP[r * LA + 32 * s + 8 * lg + i];
                ar[i] = sA[r * LA + 32 * s + 8 * lg + i];
                pc[i] = sP[(32 * s + 8 * lg + i) * LA + r];
                ac[i] = sA[(32 * s + 8 * lg + i) * LA + r] + ar[i];
            }
            const Parts<P> fpr = cut8<P>(pr), fpc = cut8<P>(pc), fac = cut8<P>(ac);
#pragma unroll
            for (int c = 0; c < CT; ++c)
                if (K % 32 == 0 || half * CT + c < K / 16) {
                    Parts<PK> kt, qt;
                    if constexpr (KQ) {
                        kt = lds_frag_turned<PK, C, KP>(sK, 32 * s + 8 * lg, 16 * (half * CT + c), lane);
                        qt = lds_frag_turned<PK, C, KP>(sQ, 32 * s + 8 * lg, 16 * (half * CT + c), lane);
                    } else {
                        kt = load_frag<PK>(a.Kt + kq, gdr_full(half * CT + c, s), lane);
                        qt = load_frag<PK>(a.Qt + kq, gdr_full(half * CT + c, s), lane);
                    }
                    mma(dq[c], fpr, kt);
                    mma(dk[c], fac, kt);
                    mma(dk[c], fpc, qt);
                }
            __builtin_amdgcn_sched_barrier(0);
        }
        __syncthreads();
        // dg.  The pairs: R = H U with U_jt = 1 for j < t sums a row's pairs before t, then the rows
        // from t on are added up; half 0 has t < 32, half 1 the others
#pragma unroll
        for (int c2 = 0; c2 < 2; ++c2) {
            const int c = 2 * half + c2, t = 16 * c + lr;
            f4 R = {};
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                Parts<1> U;
#pragma unroll
                for (int i = 0; i < 8; ++i) U.v[0][i] = (__bf16)(32 * s + 8 * lg + i < t ? 1.f : 0.f);
                mma(R, cut8<P>(sT + r * LA + 32 * s + 8 * lg), U);
            }
            float sum = 0.f;
#pragma unroll
            for (int e = 0; e < 4; ++e) sum += 16 * w + 4 * lg + e >= t ? R[e] : 0.f;
            sum += __shfl_xor(sum, 16);
            sum += __shfl_xor(sum, 32);
            if (lg == 0) sSum[turn][w][t] = sum;
            __builtin_amdgcn_sched_barrier(0);
        }
        __syncthreads();
        if (tid < C) {
            float from = sReads[turn][0][tid] + sReads[turn][1][tid], upto = sEnds[turn][0][tid] + sEnds[turn][1][tid];
            const float own = upto;
#pragma unroll
            for (int d = 1; d < 64; d *= 2) {
                const float x = __shfl_down(from, d), y = __shfl_up(upto, d);
                if (tid + d < 64) from += x;
                if (tid >= d) upto += y;
            }
            float kept = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) kept += sKeep[turn][i];
            const float sum = (sSum[turn][0][tid] + sSum[turn][1][tid]) + (sSum[turn][2][tid] + sSum[turn][3][tid]);
            if (tid < len) a.dg[(row + tid) * a.HV + hv] = sum + from + (upto - own) + dec[C - 1] * kept;
        }
    }
    const int lr = threadIdx.x & 15, lg = threadIdx.x >> 4 & 3;
#pragma unroll
    for (int c = 0; c < CT; ++c)
        if (K % 32 == 0 || half * CT + c < K / 16)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int i = 16 * w + 4 * lg + e;
                if (i < len) {
                    const int64_t o = ((row + i) * a.HK + hk) * K + 16 * (half * CT + c) + lr;
                    st_out(a.dq, a.grad_bf16, o, dq[c][e]);
                    st_out(a.dk, a.grad_bf16, o, dk[c][e]);
                }
            }
}

template <typename T, typename D, int K>
hipError_t launch(const GdrArgs &a, hipStream_t stream) {
    constexpr bool WIDE = sizeof(T) == 2 || K < 128;  // two tiles of float32 rows of 128 channels do not fit the LDS
    if (WIDE && gdr_column_tiles(a) == 2) hipLaunchKernelGGL((gdr_chains_kernel<T, D, K, WIDE ? 2 : 1>), dim3((unsigned)(2 * gdr_pair_blocks(a, a.V / 32))), dim3(256), 0, stream, a);
    else hipLaunchKernelGGL((gdr_chains_kernel<T, D, K, 1>), dim3((unsigned)(2 * gdr_pair_blocks(a, a.V / 16))), dim3(256), 0, stream, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((gdr_grads_kernel<T, D, K>), dim3((unsigned)(a.slots * a.HK)), dim3(512), 0, stream, a);
    return hipGetLastError();
}
template <typename T, typename D>
hipError_t by_width(const GdrArgs &a, int K, hipStream_t stream) {
    switch (K) {
        case 16: return launch<T, D, 16>(a, stream);
        case 32: return launch<T, D, 32>(a, stream);
        case 64: return launch<T, D, 64>(a, stream);
        case 128: return launch<T, D, 128>(a, stream);
    }
    return hipErrorNotSupported;
}

}  // namespace

hipError_t launch_gdr_bwd(const GdrArgs &a, bool fp32, int K, hipStream_t stream) {
    hipError_t e = launch_gdr_prep(a, fp32, K, true, stream);
    if (e != hipSuccess) return e;
    if (a.dout_bf16) return fp32 ? by_width<float, __bf16>(a, K, stream) : by_width<__bf16, __bf16>(a, K, stream);
    return fp32 ? by_width<float, float>(a, K, stream) : by_width<__bf16, float>(a, K, stream);
}

}  // namespace kda
