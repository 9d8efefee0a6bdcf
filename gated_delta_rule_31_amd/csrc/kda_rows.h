// Shared parts of the kernels that stand around the recurrence in a layer (kda_conv.hip,
// kda_glr_fwd.hip, kda_glr_bwd.hip, kda_norm.hip): where the sequences of a batch begin and end,
// and vectors of channels on their way between memory and float32 registers.
#pragma once

#include <stdint.h>

#include "kda_device.h"
#include "kda_internal.h"

namespace kda {

// The sequences of a batch whose rows are counted from 0 to rows - 1: packed (cu, N + 1 offsets) or
// N of T rows each.  Offsets outside 0..rows or out of order move boundaries, but never an access:
// a sequence's number stays in 0..N-1 and a row in 0..rows-1.
struct Seqs {
    const int32_t *cu;
    int64_t T, rows;  // rows of a sequence (cu: unused); all rows
    int N;

    // rows from here on belong to no sequence
    __host__ __device__ __forceinline__ int64_t limit() const {
        if (!cu) return rows;
        const int64_t e = cu[N];
        return e < 0 ? 0 : e > rows ? rows : e;
    }
    // the last sequence that begins at row t or before it
    __host__ __device__ __forceinline__ int of(int64_t t) const {
        if (!cu) return (int)((uint32_t)t / (uint32_t)T);  // fewer than 2^31 rows
        int lo = 0, hi = N;  // cu[i] <= t for i < lo, cu[i] > t for i >= hi
        while (lo < hi) {
            const int m = (lo + hi) >> 1;
            if (cu[m] <= t) lo = m + 1;
            else hi = m;
        }
        return lo > 0 ? lo - 1 : 0;
    }
    // the first row of sequence n, which row t is in: never behind t
    __host__ __device__ __forceinline__ int64_t begin(int n, int64_t t) const {
        const int64_t b = cu ? (int64_t)cu[n] : (int64_t)n * T;
        return b < 0 ? 0 : b > t ? t : b;
    }
    // bit u: row t0 + u is the first (last) of its sequence, for `count` <= 64 rows from t0 on
    __host__ __device__ __forceinline__ void marks(int64_t t0, int count, uint64_t &first, uint64_t &last) const {
        first = last = 0;
        int64_t left = 0;
        int at = 0;
        if (cu) {
            int hi = N + 1;  // the first offset that is not before t0
            while (at < hi) {
                const int m = (at + hi) >> 1;
                if (cu[m] < t0) at = m + 1;
                else hi = m;
            }
        } else {
            left = t0 ? (int64_t)(((uint32_t)t0 - 1) / (uint32_t)T + 1) * T : 0;
        }
        for (;;) {
            int64_t b;
            if (cu) {
                if (at > N) break;
                b = cu[at++];
            } else {
                if (left > rows) break;
                b = left;
                left += T;
            }
            if (b < t0 || b - t0 > count) break;
            const int u = (int)(b - t0);
            if (u < count) first |= 1ull << u;
            if (u > 0) last |= 1ull << (u - 1);
            if (cu && at <= N && cu[at] == b) {  // sequences without rows, however many: on to the first offset behind them
                for (int hi = N + 1; at < hi;) {
                    const int m = (at + hi) >> 1;
                    if (cu[m] <= b) at = m + 1;
                    else hi = m;
                }
            }
        }
    }
};

// Seqs::marks in scalar registers.
__device__ __forceinline__ void uniform_marks(const Seqs &s, int64_t t0, int count, uint64_t &first, uint64_t &last) {
    uint64_t f, l;
    s.marks(t0, count, f, l);
    first = (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)(f >> 32)) << 32 | (uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)f);
    last = (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)(l >> 32)) << 32 | (uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)l);
}

// VEC neighbouring numbers of type T in the registers that a load gives them.
template <typename T, int VEC>
struct Raw {
    typedef __attribute__((ext_vector_type(VEC))) T vec;
    vec v;
    __device__ __forceinline__ void load(const T *p) { v = *reinterpret_cast<const vec *>(p); }
    __device__ __forceinline__ void store(T *p) const { *reinterpret_cast<vec *>(p) = v; }
    // `off` bytes behind a row that all lanes share
    __device__ __forceinline__ void load(const char *row, uint32_t off) { v = *reinterpret_cast<const vec *>(row + off); }
    __device__ __forceinline__ void store(char *row, uint32_t off) const { *reinterpret_cast<vec *>(row + off) = v; }
    __device__ __forceinline__ float get(int i) const { return to_f32(v[i]); }
    __device__ __forceinline__ void set(int i, float x) { v[i] = from_f32<T>(x); }
    __device__ __forceinline__ void zero() { v = vec{}; }
};
template <typename T>
struct Raw<T, 1> {
    T v;
    __device__ __forceinline__ void load(const T *p) { v = *p; }
    __device__ __forceinline__ void store(T *p) const { *p = v; }
    __device__ __forceinline__ void load(const char *row, uint32_t off) { v = *reinterpret_cast<const T *>(row + off); }
    __device__ __forceinline__ void store(char *row, uint32_t off) const { *reinterpret_cast<T *>(row + off) = v; }
    __device__ __forceinline__ float get(int) const { return to_f32(v); }
    __device__ __forceinline__ void set(int, float x) { v = from_f32<T>(x); }
    __device__ __forceinline__ void zero() { v = T{}; }
};
// The same offset, made anew where it is used: the compiler then addresses by a scalar base and a 32-bit
// offset, where it would keep (and add up) 64-bit addresses in vector registers.
__device__ __forceinline__ uint32_t here(uint32_t off) {
    asm volatile("" : "+v"(off));
    return off;
}

// N rows `stride` bytes apart, of which the last `N - count` are the last of the `count` (> 0) again.
template <int N, typename R>
__device__ __forceinline__ void load_run(R (&r)[N], const char *row, int64_t stride, uint32_t off, int count) {
    const uint32_t at = here(off);
#pragma unroll
    for (int u = 0; u < N; ++u, row += u < count ? stride : 0) r[u].load(row, at);
}
template <int VEC>
__device__ __forceinline__ void load_f32(float (&x)[VEC], const float *p) {
    Raw<float, VEC> r;
    r.load(p);
#pragma unroll
    for (int i = 0; i < VEC; ++i) x[i] = r.get(i);
}

constexpr float LOG2E = 1.4426950408889634f;
// 1 / (1 + e^-x) on the hardware base-2 exponential and reciprocal (1 ulp each); the limits are exact.
__device__ __forceinline__ float sigmoid_f32(float x) { return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-LOG2E * x)); }

// and 1 - that without its cancellation (0 for both where e^-x passes the largest number)
__device__ __forceinline__ float sigmoid_f32(float x, float &rest) {
    const float e = __builtin_amdgcn_exp2f(-LOG2E * x), s = __builtin_amdgcn_rcpf(1.f + e);
    rest = fminf(e, 3e38f) * s;
    return s;
}

// The sums over r < rows of x[r * cols + c], in an order that the sizes alone decide.  Column c goes to
// first[c % D * W + c / D] while c < D * W and to second[c - D * W] from there on; either may be null.
struct ColumnSums {
    const float *x;
    int rows;
    int cols, D, W;
    float *first, *second;
};
hipError_t launch_column_sums(const ColumnSums &a, hipStream_t stream);

// dst[i] = src ? src[i] : 0 for i < bytes (an even number)
hipError_t launch_fill_bytes(void *dst, const void *src, int64_t bytes, hipStream_t stream);

// The pieces of a workspace one behind the other, each on a 256-byte border; with no base only
// the size is counted.
struct Pieces {
    char *base;
    size_t used = 0;
    template <typename T>
    void take(T *&p, int64_t n) {
        p = base ? reinterpret_cast<T *>(base + used) : nullptr;
        used += ((size_t)n * sizeof(T) + 255) / 256 * 256;
    }
};

// The slots of a pool that a request of a decode call starts from and leaves its states in.
struct Slots {
    const int32_t *slots, *start, *lengths;  // [B, cols], [B], [B]; any may be null
    int64_t pool;
    int S, cols;
    __device__ __forceinline__ int tokens(int b) const {
        const int n = lengths ? lengths[b] : S;
        return n < 0 ? 0 : n > S ? S : n;
    }
    // the slot in column i, -1 for one that holds no state
    __device__ __forceinline__ int64_t at(int b, int i) const {
        const int64_t s = slots ? slots[(int64_t)b * cols + i] : b;
        return s < 0 || s >= pool ? -1 : s;
    }
    __device__ __forceinline__ int64_t from(int b) const {
        const int c = start ? start[b] : 0;
        return c < 0 || c >= cols ? -1 : at(b, c);
    }
    // where the state after token i of n goes: to a column of its own, or the last one's to the only column
    __device__ __forceinline__ int64_t to(int b, int i, int n) const { return cols > 1 ? at(b, i) : i + 1 == n ? at(b, 0) : -1; }
};

// ------------------------------------------------------------------ the short convolution

struct ConvArgs {
    const void *x;               // [rows, D], x_stride between rows
    int64_t x_stride;
    const float *weight, *bias;  // [D, W], [D] or null
    const void *s0;              // [N, W - 1, D] or null
    void *sf;                    // [N, W - 1, D] or null
    Seqs seqs;
    int D, W, silu;
    void *out;                   // [rows, D]
    int run, runs;               // rows that a wave goes through, and how many runs there are
    int vecs;                    // vectors of channels in a row
    // gradients
    const void *d_out, *d_sf;    // [rows, D], [N, W - 1, D] or null
    void *dx, *ds0;              // [rows, D], [N, W - 1, D] or null
    float *part;                 // [runs, W + 1, D]
};
struct ConvStepArgs {
    const void *x;               // [B, S, D]
    const float *weight, *bias;
    void *states;                // [pool, W - 1, D]
    Slots slots;
    int B, S, D, W, silu, vecs;
    void *out;
};
constexpr int CONV_FWD_VEC = 2, CONV_BWD_VEC = 4, CONV_STEP_VEC = 2;  // channels of a lane, where rows allow it
void conv_runs(int64_t rows, int vecs, int &run, int &runs);
hipError_t launch_conv_fwd(ConvArgs a, bool fp32, bool wide, hipStream_t stream);
hipError_t launch_conv_bwd(ConvArgs a, bool fp32, bool wide, float *d_weight, float *d_bias, hipStream_t stream);
hipError_t launch_conv_step(ConvStepArgs a, bool fp32, bool wide, hipStream_t stream);

// ------------------------------------------------------------------ the gated linear recurrence

struct GlrGates {
    const void *gate;            // [rows, C]: float32 log decays, or with log_scale logits in the type of x
    const float *log_scale;      // [H] or null
    const float *bias;           // [C] or null
    const void *in_gate;         // [rows, C] or null
    int64_t gate_stride, in_stride;
    float lower;
    int normalize;
    int K;                       // channels that share a log_scale
};
// The tiles that the rows are cut into, and what passes between the launches.
struct GlrTiles {
    int rows, n, columns;        // rows of a tile, tiles, columns of channels
    float *words;                // [n, C, 2]: A and H of every tile
    float *front;                // [n, C]: the state in front of every tile; null: made of the words by whoever needs it
};
struct GlrArgs {
    const void *x;               // [rows, C]
    int64_t x_stride;
    GlrGates gates;
    const float *s0;             // [N, C] or null
    float *sf;                   // [N, C] or null
    Seqs seqs;
    int C;
    void *out;                   // [rows, C], or null: only what is kept is wanted
    float *kept;                 // [ceil(rows / GLR_KEPT), C] or null: the state in front of every GLR_KEPT rows
    GlrTiles tiles;              // workspace
    // gradients
    const void *d_out;           // [rows, C]
    const float *d_sf;           // [N, C] or null
    void *dx, *d_gate, *d_in;    // [rows, C]
    float *ds0;                  // [N, C] or null
    float *part;                 // [n, 2, C] or null
};
struct GlrStepArgs {
    const void *x;               // [B, S, C]
    GlrGates gates;
    float *states;               // [pool, C]
    Slots slots;
    int B, S, C, vecs;
    void *out;
};
constexpr int GLR_KEPT = 8;      // rows between two kept states
size_t carve_glr_fwd(GlrArgs &a, void *base);
size_t carve_glr_bwd(GlrArgs &a, void *base, bool kept, float *&sums);
// wide: two channels at a time
hipError_t launch_glr_fwd(const GlrArgs &a, bool fp32, bool wide, hipStream_t stream);
hipError_t launch_glr_bwd(const GlrArgs &a, bool fp32, bool wide, bool kept, float *sums, float *d_log_scale, float *d_bias, hipStream_t stream);
hipError_t launch_glr_step(GlrStepArgs a, bool fp32, bool wide, hipStream_t stream);

// ------------------------------------------------------------------ norms between blocks

struct NormArgs {
    const void *y, *gate;        // [rows, D]; gate: or null, with strides between tokens of `heads` rows and between those
    int64_t gate_stride, gate_head;
    const void *residual;        // [rows, D] or null
    const float *wa, *wb;        // [D] or null (ones)
    int64_t rows;
    int heads, D;
    float scale, eps;
    int after, before, silu;
    void *h, *n;                 // [rows, D]
    // gradients
    const void *d_h, *d_n;       // [rows, D], either may be null
    const void *h_in;
    void *dy, *d_gate, *d_res;
    float *part;                 // [groups, 2, D]
    int groups;                  // rows of `part`: at most norm_groups of them are written
};
int norm_groups(int64_t rows, int D);
// vec: numbers at a time, 2, 1, or any other number for 16 bytes
hipError_t launch_norm_fwd(NormArgs a, bool fp32, bool h_fp32, int vec, hipStream_t stream);
hipError_t launch_norm_bwd(NormArgs a, bool fp32, bool h_fp32, int vec, float *d_wa, float *d_wb, hipStream_t stream);

}  // namespace kda
