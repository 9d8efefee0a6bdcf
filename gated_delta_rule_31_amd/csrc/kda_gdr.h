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
// are cut into 3 parts (24 bits: one part is off by at most 2^-8 of the value, its remainder's
// part by 2^-8 of that, and so on), and the part products that matter are added in float32: 3
// instructions against an exact operand, 6 against another of 3 parts, where the float32 matrix
// instruction costs 16 times a bf16 one.
#pragma once

#include "kda_device.h"
#include "kda_internal.h"

namespace kda {

constexpr int GDR_C = 64;  // tokens per chunk
// Parts of a computed operand, on its way to the state and to the output alike.  Two parts (16
// bits) of those that reach the output alone left it 4e-6 off in the 2-norm, which a float32
// output shows, for 6% less of a call's time (8192 tokens x 96 heads, K = V = 128, bf16: 728 us
// against 775).
constexpr int GDR_PARTS = 3;

// Workspace of one call; the matrices are stored in the order in which a wave loads its
// matrix-core fragments: [.., fragment][part][lane][8], a fragment being a 16-row tile of 32
// columns.
//
// The prefill's M and P are lower triangles: six fragments of the eight, M's and then P's, 36 KB
// of the GDR_UNIT that every (chunk slot, value head) has.
constexpr int GDR_UNIT = 5 * GDR_C * GDR_C;
__device__ __forceinline__ constexpr int gdr_full(int r, int s) { return r * 2 + s; }               // tile r, step s
__device__ __forceinline__ constexpr int gdr_lower(int r, int s) { return r < 2 ? r : 2 * r - 2 + s; }  // s <= r / 2
constexpr int GDR_P_AT = 6 * GDR_PARTS * 512;  // where a unit's P starts
static_assert(2 * GDR_P_AT <= GDR_UNIT, "M and P of a unit");
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
    __bf16 *M, *P;               // M: [slots * HV][GDR_UNIT], with P behind it; backward: [slots * HV][parts * 4096] each
    __bf16 *Kt;                  // [slots * HK][parts of k * K * 64], float32 gradients only
    float *dec;                  // [slots * HV][4 * 64]: e^G, e^{G_C - G}, beta, unused
    // backward
    __bf16 *Mt, *Qt;             // M^T (P holds P^T), Q^T
    double *G;                   // [slots * HV][64], log2 units
    // by slices of 32 columns (of 16 with V = 16), so that a slice is one run of memory
    float *h, *dh;               // [slots * HV][slices][K][32]: state at the chunk's start, gradient at its end
    float *delta, *dY;           // [slots * HV][slices][64][32]
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

// Two float32 numbers as pairs of bf16 parts, part p of both in one register.
template <int P>
__device__ __forceinline__ void cut2(float x, float y, unsigned (&o)[P]) {
    typedef __attribute__((ext_vector_type(2))) float f2;
    typedef __attribute__((ext_vector_type(2))) __bf16 bf16x2;
#pragma unroll
    for (int p = 0; p < P; ++p) {
        o[p] = __builtin_bit_cast(unsigned, __builtin_convertvector((f2{x, y}), bf16x2));
        if (p + 1 < P) {
            x -= __builtin_bit_cast(float, o[p] << 16);
            y -= __builtin_bit_cast(float, o[p] & 0xffff0000u);
        }
    }
}

typedef __attribute__((ext_vector_type(4))) unsigned u32x4;
typedef __attribute__((ext_vector_type(2))) unsigned u32x2;

template <int P>
__device__ __forceinline__ Parts<P> cut8(const float *x) {
    u32x4 r[P];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        unsigned o[P];
        cut2<P>(x[2 * i], x[2 * i + 1], o);
#pragma unroll
        for (int p = 0; p < P; ++p) r[p][i] = o[p];
    }
    Parts<P> f;
#pragma unroll
    for (int p = 0; p < P; ++p) f.v[p] = __builtin_bit_cast(bf16x8, r[p]);
    return f;
}

// acc += A B for operands given in parts: the part products that matter beside the finer
// operand's last part, smallest first.
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

// A wave's fragment i of a workspace matrix.
template <int P>
__device__ __forceinline__ Parts<P> load_frag(const __bf16 *m, int i, int lane) {
    Parts<P> f;
    const char *from = reinterpret_cast<const char *>(m) + i * P * 1024;
#pragma unroll
    for (int p = 0; p < P; ++p) f.v[p] = *reinterpret_cast<const bf16x8 *>(from + (unsigned)(lane * 16) + p * 1024);
    return f;
}
template <int P>
__device__ __forceinline__ void store_frag(__bf16 *m, int i, int lane, const Parts<P> &f) {
#pragma unroll
    for (int p = 0; p < P; ++p) *reinterpret_cast<bf16x8 *>(m + (((i * P + p) * 64) + lane) * 8) = f.v[p];
}

// Operands in LDS: parts of an R x N matrix (N a multiple of 32), rows of N elements without
// padding.  A row's 16-byte pieces are placed by piece XOR row (for rows shorter than the 64
// banks, XOR of the row's place among those that share a line of banks), so that the sixteen
// rows of a fragment, and the rows that a store writes, fall on different banks.
template <int N>
__device__ __forceinline__ int lds_at(int row, int col) {
    constexpr int PIECES = N / 8, SHARE = 16 / PIECES;  // pieces of a row; rows on one line of banks
    static_assert(N == 32 || N == 64 || N == 128, "rows of at most one line");
    const int turn = N == 32 ? (PIECES - row / SHARE % PIECES) % PIECES : row / SHARE % PIECES;
    return row * N + ((col / 8) ^ turn) * 8 + col % 8;
}
template <int P, int R, int N>
__device__ __forceinline__ Parts<P> lds_frag(const __bf16 *m, int row, int col) {
    Parts<P> f;
#pragma unroll
    for (int p = 0; p < P; ++p) f.v[p] = *reinterpret_cast<const bf16x8 *>(m + p * R * N + lds_at<N>(row, col));
    return f;
}
// Four consecutive float32 numbers of a row into LDS as parts.
template <int P, int R, int N>
__device__ __forceinline__ void lds_put4(__bf16 *m, int row, int col, const f4 &x) {
    unsigned a[P], b[P];
    cut2<P>(x[0], x[1], a);
    cut2<P>(x[2], x[3], b);
#pragma unroll
    for (int p = 0; p < P; ++p) *reinterpret_cast<u32x2 *>(m + p * R * N + lds_at<N>(row, col)) = u32x2{a[p], b[p]};
}

// The transpose of a fragment: eight rows (from row) of column col + lane % 16, out of R x N
// matrices in the same layout.  The instruction turns 4 x 16 tiles: in each sixteen lanes, lane
// 4 i + j gives the address of row i's columns 4 j .. + 3 and receives the rows of its column.
template <int P, int R, int N>
__device__ __forceinline__ Parts<P> lds_frag_turned(const __bf16 *m, int row, int col, int lane) {
    typedef __attribute__((ext_vector_type(4))) short s4;
    typedef __attribute__((address_space(3))) s4 *lds4;
    const int r = row + lane % 16 / 4, c = col + lane % 4 * 4;
    Parts<P> f;
#pragma unroll
    for (int p = 0; p < P; ++p) {
        const s4 x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4)(m + p * R * N + lds_at<N>(r, c)));
        const s4 y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4)(m + p * R * N + lds_at<N>(r + 4, c)));
        f.v[p] = __builtin_bit_cast(bf16x8, __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7));
    }
    return f;
}

// A load or store at a 32-bit byte offset from an address that the whole wave shares.
template <typename V>
__device__ __forceinline__ V at_offset(const void *base, unsigned bytes) {
    return *reinterpret_cast<const V *>(static_cast<const char *>(base) + bytes);
}

// Workgroup barrier for LDS traffic only: the waves exchange data through LDS alone, so
// global loads and stores stay in flight across it.
__device__ __forceinline__ void gdr_lds_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// Between LDS writes and reads by which lanes of one wave hand values to each other.  A wave's LDS
// instructions are carried out in order, so nothing has to be waited for: it keeps the compiler
// from moving one past the other where it could tell a lane's own addresses apart.
__device__ __forceinline__ void gdr_wave_fence() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// Sequence n: its first token's row, its length and its first chunk slot.  Packed offsets are
// brought into [0, T], and a sequence that ends before it starts is empty, so that no offset a
// caller passes reads or writes outside the tensors: rows end at T at most, slots at T / C + N.
// Offsets in order (each at least the one before) give every sequence rows and slots of its own;
// others may share them, and then what is computed is unspecified.
__host__ __device__ __forceinline__ void gdr_sequence(const GdrArgs &a, int n, int64_t &row, int64_t &len, int64_t &slot) {
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
__host__ __device__ __forceinline__ bool gdr_chunk(const GdrArgs &a, int64_t slot, int64_t &row, int &len) {
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

// Where a column tile's element stands in the rows of a matrix kept by slices, and the slice's
// row length.
__device__ __forceinline__ int gdr_slice_columns(int V) { return V < 32 ? V : 32; }
__device__ __forceinline__ int64_t gdr_slice_at(int rows, int col, int V) { return (int64_t)(col / 32) * (rows * 32) + (V < 32 ? col : col % 32); }

// The chains' grids: block b of 8 VB ceil(N HV / 8) takes value block b / 8 % VB of pair
// (b / 8 / VB) 8 + b % 8.  Blocks go to the eight XCDs in turn, so a pair's value blocks, which
// read the same keys, share one XCD's L2, and a long sequence's heads spread over all of them.
// Packed sequences (up to 64) are taken longest first, so that none is left to run alone.
// False for a block without a pair.
__device__ __forceinline__ bool gdr_pair(const GdrArgs &a, int block, int VB, int &vb, int &hv, int &n) {
    const int i = block / 8;
    const int64_t pair = (int64_t)(i / VB) * 8 + block % 8;
    vb = i % VB;
    hv = (int)(pair % a.HV);
    n = (int)(pair / a.HV);
    if (pair >= (int64_t)a.N * a.HV) return false;
    if (a.cu && a.N > 1 && a.N <= 64) {
        const int lane = threadIdx.x & 63;
        int64_t row, len = -1, slot;
        if (lane < a.N) gdr_sequence(a, lane, row, len, slot);
        int rank = 0;
        for (int m = 0; m < a.N; ++m) {
            const int other = __builtin_amdgcn_readlane((int)len, m);
            rank += other > (int)len || (other == (int)len && m < lane);
        }
        n = __builtin_ctzll(__ballot(lane < a.N && rank == n));
    }
    return true;
}
// Tiles of 16 value columns that one workgroup of a chain takes: one while that gives a compute
// unit no more than one workgroup (forward chain, 8192 tokens x 32 heads of 128 columns, bf16: 277
// us, two tiles 339), two from two workgroups a unit on, as a chunk's operands are then loaded half
// as often (64 heads: 395 us, one tile 499; 80 heads 621, 731; 96 heads 610, 725).  The time per
// head is not even: the workgroups of 80 or 96 heads are more than the units, and less than two each.
inline int gdr_column_tiles(const GdrArgs &a) {
    return a.V >= 32 && (int64_t)a.N * a.HV * (a.V / 16) >= 2 * device_cu_count() ? 2 : 1;
}
inline int64_t gdr_pair_blocks(const GdrArgs &a, int VB) { return ((int64_t)a.N * a.HV + 7) / 8 * 8 * VB; }

// the products that do not depend on the state, for every (chunk slot, value head)
hipError_t launch_gdr_prep(const GdrArgs &a, bool fp32, int K, bool bwd, hipStream_t stream);
hipError_t launch_gdr_fwd_chain(const GdrArgs &a, bool fp32, int K, hipStream_t stream);
hipError_t launch_gdr_bwd(const GdrArgs &a, bool fp32, int K, hipStream_t stream);

}  // namespace kda
