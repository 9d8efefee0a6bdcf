// kda_gdr_fwd.hip -- chunkwise prefill of the gated delta rule with one decay per value head
// (formulas and precision: kda_gdr.h).  Two kernels: a pre-pass over all (chunk, value head)
// pairs at once, which forms what does not depend on the state (M, P, the decays), and
// the chain, serial over a sequence's chunks and parallel over sequences, value heads and
// blocks of 16 value columns.
#include "kda_gdr_chain.h"

namespace kda {
namespace {

constexpr int C = GDR_C, P = GDR_PARTS;

// Eight elements down a column of an LDS tile, as parts.
template <int P, typename T>
__device__ __forceinline__ Parts<P> column8(const T *m, int ld, int row, int col) {
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = to_f32(m[(row + i) * ld + col]);
    return cut8<P>(x);
}

// The lower 16 x 16 blocks of a C x C float32 matrix in LDS, rows of 20.
constexpr int BLOCKS = 10, LB = 20;
__device__ __forceinline__ int block_at(int p, int r) { return (p * (p + 1) / 2 + r) * 16 * LB; }

// One workgroup of four waves per (chunk slot, value head), and for float32 gradients one per
// (chunk slot, key head) that writes K^T and Q^T.  Wave w owns token rows 16w..16w+15 until A
// is there, then the column blocks w of M.  38 KB of LDS, so that four workgroups share a
// compute unit: a workgroup mostly waits (for its rows, for substitution and products that
// follow one another), and what it writes, 37 KB, is more than it reads.  8192 tokens x 96
// heads, K = 128, bf16: 191 us (183 to 213), 0.18 GB read and 0.46 GB written.
template <typename T, int K, bool BWD>
__global__ __launch_bounds__(256) void gdr_prep_kernel(const GdrArgs a) {
    constexpr int PK = gdr_input_parts<T>(), KP = K < 32 ? 32 : K, LK = KP + 8, KS = KP / 32, VEC = 16 / sizeof(T);
    constexpr bool TURNED = BWD && PK > 1;  // bf16 rows are turned in LDS where they are used
    constexpr int WORK = 2 * BLOCKS * 16 * LB * 4, BYTES = TURNED && C * LK * (int)sizeof(T) > WORK ? C * LK * (int)sizeof(T) : WORK;
    __shared__ __attribute__((aligned(16))) char shared[BYTES];
    __shared__ __attribute__((aligned(16))) float sD[4][16 * LB], sI[4][16 * LB], sP[BWD ? BLOCKS * 16 * LB : 4];
    __shared__ double sG[4][C];
    const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6), lr = lane & 15, lg = lane >> 4;
    const T *q = static_cast<const T *>(a.q), *k = static_cast<const T *>(a.k);
    // blocks go to the eight XCDs in turn: a key head's blocks, which read the same rows, are 8
    // apart and share an L2
    const int i8 = blockIdx.x / 8, each = a.group + TURNED, which_head = i8 % each;
    const int64_t key = (int64_t)(i8 / each) * 8 + blockIdx.x % 8, slot = key / a.HK;
    const int hk = (int)(key % a.HK);
    if (key >= a.slots * a.HK) return;
    int64_t row;
    int len;
    if (!gdr_chunk(a, slot, row, len)) return;
    if (TURNED && which_head == a.group) {  // K^T, Q^T through LDS
        T *tile = reinterpret_cast<T *>(shared);
        for (int which = 0; which < 2; ++which) {
            const T *from = which ? q : k;
            if (which) __syncthreads();
            for (int i = tid; i < C * K / VEC; i += 256) {
                const int r = i / (K / VEC), c = i % (K / VEC) * VEC;
                f4 x = {};
                if (r < len) x = *reinterpret_cast<const f4 *>(from + ((row + r) * a.HK + hk) * K + c);
                *reinterpret_cast<f4 *>(tile + r * LK + c) = x;
            }
            __syncthreads();
            __bf16 *to = (which ? a.Qt : a.Kt) + key * (PK * K * C);
            for (int i = w; i < K / 16 * 2; i += 4)
                store_frag<PK>(to, gdr_full(i / 2, i % 2), lane, column8<PK>(tile, LK, 32 * (i % 2) + 8 * lg, 16 * (i / 2) + lr));
        }
        return;
    }
    const int hv = hk * a.group + which_head;
    const int64_t unit = slot * a.HV + hv;
    float *sA = reinterpret_cast<float *>(shared), *sM = sA + BLOCKS * 16 * LB;

    // log decays in log2 units, summed in float64, lane = token; beyond 2^-1000 a decay is 0 in
    // float32 whatever follows, and the bound keeps -inf out of the differences
    const int64_t at = (row + (lane < len ? lane : 0)) * a.HV + hv;
    double g = (double)a.g[at] * 1.4426950408889634;
    float beta = a.beta[at];
    Parts<PK> fk[KS], fq[KS];
    // rows behind the end read the last row: their beta is 0 and their d_out too, so that what their
    // rows of A, M and P hold reaches nothing
    const char *kbase = reinterpret_cast<const char *>(k + (row * a.HK + hk) * K), *qbase = reinterpret_cast<const char *>(q + (row * a.HK + hk) * K);
    const unsigned kstep = (unsigned)a.HK * K * sizeof(T);
    auto rows8 = [&](const char *base, int r, int s) {
        const unsigned at = (unsigned)(r < len ? r : len - 1) * kstep + (K < 32 ? lg % 2 * 8 : 8 * lg) * (unsigned)sizeof(T);
        Parts<PK> y = load8<PK>(reinterpret_cast<const T *>(base + at + 32 * s * sizeof(T)), true);
        if (K < 32)
#pragma unroll
            for (int p = 0; p < PK; ++p) y.v[p] = lg < 2 ? y.v[p] : bf16x8{};
        return y;
    };
#pragma unroll
    for (int s = 0; s < KS; ++s) {
        fk[s] = rows8(kbase, 16 * w + lr, s);
        fq[s] = rows8(qbase, 16 * w + lr, s);
    }
    if (lane >= len) g = 0.0, beta = 0.f;
    g = g < -1000.0 ? -1000.0 : g;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const double up = __shfl_up(g, d);
        if (lane >= d) g += up;
    }
    sG[w][lane] = g;  // every wave has its own copy: no barrier
    gdr_wave_fence();
    if (w == 0) {
        const double last = __shfl(g, 63);
        float *dec = a.dec + unit * 4 * C;
        dec[lane] = __builtin_amdgcn_exp2f((float)g);
        dec[C + lane] = __builtin_amdgcn_exp2f((float)(last - g));
        dec[2 * C + lane] = beta;
        if (BWD) a.G[unit * C + lane] = g;
    }
    double gi[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) gi[e] = sG[w][16 * w + 4 * lg + e];

    // A and P of the wave's rows; P goes through the wave's rows of sM (BWD: of sP)
    float *rowsP = BWD ? sP : sM;
#pragma unroll
    for (int c = 0; c < 4; ++c)
        if (c <= w) {
            f4 kk = {}, qk = {};
#pragma unroll
            for (int s = 0; s < KS; ++s) {
                const Parts<PK> f = c == w ? fk[s] : rows8(kbase, 16 * c + lr, s);
                mma(kk, fk[s], f);
                mma(qk, fq[s], f);
            }
            const double gj = sG[w][16 * c + lr];
            const float bj = __shfl(beta, 16 * c + lr);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int i = 4 * lg + e;
                const float d = c < w || lr <= i ? __builtin_amdgcn_exp2f((float)(gi[e] - gj)) : 0.f;
                kk[e] = c < w || lr < i ? kk[e] * d : 0.f;
                qk[e] = c < w || lr <= i ? qk[e] * d : 0.f;
                sA[block_at(w, c) + i * LB + lr] = kk[e];
                rowsP[block_at(w, c) + i * LB + lr] = qk[e];
            }
            if (c == w) *reinterpret_cast<f4 *>(sD[w] + lr * LB + 4 * lg) = bj * kk;  // A beta, columns first
        }
    gdr_wave_fence();  // the wave's rows of P and its diagonal block are read by other lanes
    // eight elements of a row, or of a column, of a matrix held by blocks; zeros above the diagonal
    auto row8f = [&](const float *m, int s, float (&x)[8]) {
        const int c = 2 * s + lg / 2;
        const float *from = m + block_at(w, c <= w ? c : w) + lr * LB + lg % 2 * 8;
        const f4 u = *reinterpret_cast<const f4 *>(from), v = *reinterpret_cast<const f4 *>(from + 4);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = c <= w ? (i < 4 ? u[i % 4] : v[i % 4]) : 0.f;
    };
    auto column8f = [&](const float *m, int s, float (&x)[8]) {
        const int p = 2 * s + lg / 2;
        const float *from = m + block_at(p >= w ? p : w, w) + lg % 2 * 8 * LB + lr;
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = p >= w ? from[i * LB] : 0.f;
    };
    float x8[8];
    if (!BWD)
#pragma unroll
        for (int s = 0; s < 2; ++s)
            if (s <= w / 2) {
                row8f(sM, s, x8);
                store_frag<P>(a.M + unit * GDR_UNIT + GDR_P_AT, gdr_lower(w, s), lane, cut8<P>(x8));
            }
    // the inverse of block w of 1 + A beta on the diagonal by substitution, a column a lane: as
    // soon as row m of the inverse is there its part is taken off all rows below
    {
        f4 x[4];
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i / 4][i % 4] = i == lr ? 1.f : 0.f;
#pragma unroll
        for (int m = 0; m < 15; ++m) {
            const float xm = x[m / 4][m % 4];
#pragma unroll
            for (int i4 = (m + 1) / 4; i4 < 4; ++i4) {
                const f4 l = *reinterpret_cast<const f4 *>(sD[w] + m * LB + 4 * i4);  // 0 up to the diagonal
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (4 * i4 + e > m) x[i4][e] -= l[e] * xm;
            }
        }
        if (lg == 0) {
#pragma unroll
            for (int i = 0; i < 16; ++i) sI[w][i * LB + lr] = x[i / 4][i % 4];
        }
    }
    gdr_lds_barrier();

    // M by columns of blocks, wave w column w: (1 + A_pp beta_p) M_pw = -(A_pw + sum_r A_pr beta_r M_rw).
    // Step e of a product takes k = 4 (lane / 16) + e, which is how an accumulator holds its rows.
    f4 m[4];
#pragma unroll
    for (int p = 0; p < 4; ++p)
        if (p >= w) {
            f4 acc;
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[e] = sA[block_at(p, w) + (4 * lg + e) * LB + lr];
#pragma unroll
            for (int r = 0; r < p; ++r)
                if (r >= w) {
                    const f4 x = *reinterpret_cast<const f4 *>(sA + block_at(p, r) + lr * LB + 4 * lg);
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc = __builtin_amdgcn_mfma_f32_16x16x4f32(x[e], m[r][e], acc, 0, 0, 0);
                }
            const f4 d = *reinterpret_cast<const f4 *>(sI[p] + lr * LB + 4 * lg);
            f4 y = {};
#pragma unroll
            for (int e = 0; e < 4; ++e) y = __builtin_amdgcn_mfma_f32_16x16x4f32(d[e], -acc[e], y, 0, 0, 0);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                sM[block_at(p, w) + (4 * lg + e) * LB + lr] = y[e];
                m[p][e] = y[e] * __shfl(beta, 16 * p + 4 * lg + e);
            }
        }
    gdr_lds_barrier();
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        if (s <= w / 2) {
            row8f(sM, s, x8);
            store_frag<P>(a.M + unit * (BWD ? P * C * C : GDR_UNIT), gdr_lower(w, s), lane, cut8<P>(x8));
        }
        if (BWD && s >= w / 2) {
            column8f(sM, s, x8);
            store_frag<P>(a.Mt + unit * (P * C * C), gdr_full(w, s), lane, cut8<P>(x8));
            column8f(sP, s, x8);
            store_frag<P>(a.P + unit * (P * C * C), gdr_full(w, s), lane, cut8<P>(x8));
        }
    }
}

template <typename T, typename OT, int K, int NV>
__global__ __launch_bounds__(256) void gdr_chain_kernel(const GdrArgs a) {
    constexpr int PK = gdr_input_parts<T>(), KP = K < 32 ? 32 : K, W = 16 * NV;
    __shared__ __attribute__((aligned(16))) __bf16 sS[P * W * KP], sX[P * W * C], sE[P * W * C], sV[P * W * C], sK[PK * C * KP];
    gdr_chain<T, OT, K, NV, false>(a, blockIdx.x, sS, sX, sE, sV, sK);
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

template <typename T, bool BWD>
hipError_t prep(const GdrArgs &a, int K, hipStream_t stream) {
    return by_width(K, [&](auto k) {
        hipLaunchKernelGGL((gdr_prep_kernel<T, decltype(k)::value, BWD>), dim3((unsigned)((a.slots * a.HK + 7) / 8 * 8 * (a.group + (BWD && sizeof(T) == 4)))), dim3(256), 0, stream, a);
        return hipGetLastError();
    });
}
template <typename T, typename OT>
hipError_t chain(const GdrArgs &a, int K, hipStream_t stream) {
    return by_width(K, [&](auto k) {
        constexpr int KK = decltype(k)::value;
        if (gdr_column_tiles(a) == 2) hipLaunchKernelGGL((gdr_chain_kernel<T, OT, KK, 2>), dim3((unsigned)gdr_pair_blocks(a, a.V / 32)), dim3(256), 0, stream, a);
        else hipLaunchKernelGGL((gdr_chain_kernel<T, OT, KK, 1>), dim3((unsigned)gdr_pair_blocks(a, a.V / 16)), dim3(256), 0, stream, a);
        return hipGetLastError();
    });
}

}  // namespace

hipError_t launch_gdr_prep(const GdrArgs &a, bool fp32, int K, bool bwd, hipStream_t stream) {
    if (bwd) return fp32 ? prep<float, true>(a, K, stream) : prep<__bf16, true>(a, K, stream);
    return fp32 ? prep<float, false>(a, K, stream) : prep<__bf16, false>(a, K, stream);
}

hipError_t launch_gdr_fwd_chain(const GdrArgs &a, bool fp32, int K, hipStream_t stream) {
    if (a.out_bf16) return fp32 ? chain<float, __bf16>(a, K, stream) : chain<__bf16, __bf16>(a, K, stream);
    return fp32 ? chain<float, float>(a, K, stream) : chain<__bf16, float>(a, K, stream);
}

}  // namespace kda
