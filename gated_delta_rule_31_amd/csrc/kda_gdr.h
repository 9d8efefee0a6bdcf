// Shared parts of the gated-delta-rule kernels with one decay per value head
// (kda_gdr_fwd.hip, kda_gdr_bwd.hip): arguments, the chunk slots of packed sequences, and
// products of float32 numbers on the bf16 matrix cores.
//
// Per chunk of C = 64 tokens that starts from state S, with G the inclusive sum of the log
// decays inside the chunk and D_ij = e^{G_i - G_j} (j <= i):
//   A_ij  = (k_i . k_j) D_ij (j < i)            P_ij = (q_i . k_j) D_ij (j <= i)
//   X     = V - e^G K S                         what the values leave to correct
//   delta = X + M (beta X)                      M = -(1 + A beta)^-1 A, strictly lower
//   Vn    = beta delta
//   O     = scale (e^G Q S + P Vn)              S' = e^{G_C} S + K^T e^{G_C - G} Vn
// (delta_i = X_i - sum_{j<i} A_ij beta_j delta_j is the token loop's v_i - S^T k_i.)  Every
// exponent is <= 0, so unlike a decay per channel nothing has to be rescaled and there is no
// lower bound on g.
//
// Precision.  States, sums and decays are float32 (G itself is summed in float64: e^{G_i-G_j}
// of nearby tokens must not lose the bits that far tokens take).  A product's operands go to
// the matrix cores as sums of bf16 parts: bf16 inputs are one part and exact, float32 numbers
// are cut into 2 parts (16 bits; one part is off by at most 2^-8 of the value, its remainder's
// part by 2^-8 of that) or 3 (24 bits), and the part products that matter are added in
// float32: 2 parts cost 2 (against an exact operand) or 3 instructions, 3 parts 3 or 6, where
// the float32 matrix instruction costs 16 times a bf16 one.
#pragma once

#include "kda_device.h"
#include "kda_internal.h"

namespace kda {

constexpr int GDR_C = 64;  // tokens per chunk

// Workspace of one call; the matrices are stored in the order in which a wave loads its
// matrix-core fragments: [.., 16-row tile][32-column step][part][lane][8].
struct GdrArgs {
    const void *q, *k, *v;       // [rows, HK, K], [rows, HK, K], [rows, HV, V]
    const float *g, *beta;       // [rows, HV]
    const float *s0;             // [N, HV, K, V] or null
    float *sf;                   // [N, HV, K, V] or null
    const int32_t *cu;           // [N + 1] or null
    void *out;                   // [rows, HV, V]
    int64_t T;                   // tokens of a batch row; all tokens with cu
    int N, HK, HV, group, V;     // group = HV / HK
    int out_bf16;
    float scale;
    int64_t slots;               // chunk slots
    int chunks;                  // chunk slots of a batch row (no cu)
    __bf16 *M, *P;               // [slots * HV][parts * 4096]
    __bf16 *Kt;                  // [slots * HK][parts of k * K * 64]
    float *dec;                  // [slots * HV][4 * 64]: e^G, e^{G_C - G}, beta, unused
    // backward
    __bf16 *Mt, *Qt;             // M^T (P holds P^T), Q^T
    double *G;                   // [slots * HV][64], log2 units
    float *h, *dh;               // [slots * HV][K * V]: state at the chunk's start, gradient at its end
    float *delta, *dY;           // [slots * HV][64 * V]
    const void *d_out;           // [rows, HV, V]
    int dout_bf16;
    const float *d_sf;           // [N, HV, K, V] or null
    void *dq, *dk, *dv;
    int grad_bf16;
    float *dg, *dbeta;           // [rows, HV]
    float *ds0;                  // [N, HV, K, V] or null
};

// The parts that numbers are cut into: those of the inputs and those of computed operands.
template <typename T> constexpr int gdr_input_parts() { return sizeof(T) == 2 ? 1 : 3; }

template <int P>
struct Parts {
    bf16x8 v[P];
};

template <int P>
__device__ __forceinline__ void cut(float x, __bf16 (&o)[P]) {
#pragma unroll
    for (int p = 0; p < P; ++p) {
        o[p] = (__bf16)x;
        x -= (float)o[p];
    }
}

template <int P>
__device__ __forceinline__ Parts<P> cut8(const float *x) {
    Parts<P> r;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        __bf16 o[P];
        cut<P>(x[i], o);
#pragma unroll
        for (int p = 0; p < P; ++p) r.v[p][i] = o[p];
    }
    return r;
}

// acc += A B for operands given in parts; the part products below the last part of the
// finer operand are left out.
template <int NA, int NB>
__device__ __forceinline__ void mma(f4 &acc, const Parts<NA> &a, const Parts<NB> &b) {
    constexpr int L = NA > NB ? NA : NB;
#pragma unroll
    for (int s = L - 1; s >= 0; --s)
#pragma unroll
        for (int i = 0; i < NA; ++i)
            if (s - i >= 0 && s - i < NB)
                acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.v[i], b.v[s - i], acc, 0, 0, 0);
}

// Eight consecutive elements of an input as parts; zeros where !there.
template <int PK>
__device__ __forceinline__ Parts<PK> load8(const __bf16 *p, bool there) {
    Parts<PK> r;
    r.v[0] = there ? *reinterpret_cast<const bf16x8 *>(p) : bf16x8{};
    return r;
}
template <int PK>
__device__ __forceinline__ Parts<PK> load8(const float *p, bool there) {
    float x[8] = {};
    if (there) {
        *reinterpret_cast<f4 *>(x) = *reinterpret_cast<const f4 *>(p);
        *reinterpret_cast<f4 *>(x + 4) = *reinterpret_cast<const f4 *>(p + 4);
    }
    return cut8<PK>(x);
}

// A wave's fragment of a workspace matrix: tile r, step s of a matrix with two 32-column steps.
template <int P>
__device__ __forceinline__ Parts<P> load_frag(const __bf16 *m, int r, int s, int lane) {
    Parts<P> f;
#pragma unroll
    for (int p = 0; p < P; ++p)
        f.v[p] = *reinterpret_cast<const bf16x8 *>(m + ((((r * 2 + s) * P + p) * 64) + lane) * 8);
    return f;
}
template <int P>
__device__ __forceinline__ void store_frag(__bf16 *m, int r, int s, int lane, const Parts<P> &f) {
#pragma unroll
    for (int p = 0; p < P; ++p) *reinterpret_cast<bf16x8 *>(m + ((((r * 2 + s) * P + p) * 64) + lane) * 8) = f.v[p];
}

// A fragment out of LDS: part p of row `row` at element `col`, rows of `ld` elements, parts
// `ps` elements apart.
template <int P>
__device__ __forceinline__ Parts<P> lds_frag(const __bf16 *m, int ps, int ld, int row, int col) {
    Parts<P> f;
#pragma unroll
    for (int p = 0; p < P; ++p) f.v[p] = *reinterpret_cast<const bf16x8 *>(m + p * ps + row * ld + col);
    return f;
}
// Four consecutive float32 numbers into LDS as parts.
template <int P>
__device__ __forceinline__ void lds_put4(__bf16 *m, int ps, int ld, int row, int col, const f4 &x) {
    typedef __attribute__((ext_vector_type(4))) __bf16 bf16x4;
    bf16x4 r[P];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        __bf16 o[P];
        cut<P>(x[i], o);
#pragma unroll
        for (int p = 0; p < P; ++p) r[p][i] = o[p];
    }
#pragma unroll
    for (int p = 0; p < P; ++p) *reinterpret_cast<bf16x4 *>(m + p * ps + row * ld + col) = r[p];
}

// Workgroup barrier for LDS traffic only: the waves exchange data through LDS alone, so
// global loads and stores stay in flight across it.
__device__ __forceinline__ void gdr_lds_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// Sequence n: its first token's row, its length and its first chunk slot.  Packed offsets
// are brought into [0, T] and into order, so that no offset a caller passes reads or writes
// outside the tensors; slots of different sequences are disjoint and below T / C + N.
__device__ __forceinline__ void gdr_sequence(const GdrArgs &a, int n, int64_t &row, int64_t &len, int64_t &slot) {
    if (a.cu) {
        int64_t b = a.cu[n], e = a.cu[n + 1];
        b = b < 0 ? 0 : b > a.T ? a.T : b;
        e = e < b ? b : e > a.T ? a.T : e;
        row = b;
        len = e - b;
        slot = b / GDR_C + n;
    } else {
        row = n * a.T;
        len = a.T;
        slot = (int64_t)n * a.chunks;
    }
}

// The chunk at a slot: its first token's row and its length; false if the slot holds none.
__device__ __forceinline__ bool gdr_chunk(const GdrArgs &a, int64_t slot, int64_t &row, int &len) {
    int64_t r, l, s0;
    if (a.cu) {
        int lo = 0, hi = a.N - 1;  // the last sequence whose first slot is <= slot
        while (lo < hi) {
            const int mid = (lo + hi + 1) / 2;
            gdr_sequence(a, mid, r, l, s0);
            if (s0 <= slot) lo = mid;
            else hi = mid - 1;
        }
        gdr_sequence(a, lo, r, l, s0);
    } else {
        gdr_sequence(a, (int)(slot / a.chunks), r, l, s0);
    }
    const int64_t at = (slot - s0) * GDR_C;
    if (at < 0 || at >= l) return false;
    row = r + at;
    len = (int)(l - at < GDR_C ? l - at : GDR_C);
    return true;
}

// Block index to unit: consecutive blocks go to the eight XCDs in turn, so units of one
// eighth of the range run on one XCD and share its L2.
__device__ __forceinline__ int gdr_xcd_unit(int b, int total) {
    const int per = total / 8, left = total % 8, x = b % 8, i = b / 8;
    return x * per + (x < left ? x : left) + i;
}

// the products that do not depend on the state, for every (chunk slot, value head)
hipError_t launch_gdr_prep(const GdrArgs &a, bool fp32, int K, bool bwd, hipStream_t stream);
hipError_t launch_gdr_fwd_chain(const GdrArgs &a, bool fp32, int K, bool train, hipStream_t stream);
hipError_t launch_gdr_bwd(const GdrArgs &a, bool fp32, int K, hipStream_t stream);

}  // namespace kda
