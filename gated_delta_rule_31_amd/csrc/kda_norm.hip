// kda_norm.hip -- what stands between two blocks, and behind a recurrence's heads (gfx950):
//   p = y r w_after, r = 1 / sqrt(mean y^2 + eps)      (or p = y)
//   h = residual + scale act(gate) p                   (act: sigmoid or silu; without a gate 1)
//   n = h r' w_before, r' = 1 / sqrt(mean h^2 + eps)
// and its gradients, every row by itself: one pass over memory, the row in registers between its
// sums.  Bound by memory, a large copy having 5.0 TB/s: 786432 heads of 128, norm and gate, bf16, 118 us (5.1 TB/s), the
// gradients of 131072 of them 37 + 4; gradients between two blocks, 8192 x 7168 with a float32 stream, 261 + 8 us (4.9
// TB/s); one row of 7168, 3.9 us.  Rows of 7168 by 256, 512 or 1024 lanes: 269, 269 and 274 us.
//
// LANES lanes share a row (4, 16, 32 or 64 of a wave, or a whole workgroup), each with NV vectors of
// VEC neighbouring channels, LANES vectors apart.  Workgroups go from row to row and keep the
// weights in registers, and in the backward pass the weights' sums, which they write once.
#include "kda_rows.h"

namespace kda {
namespace {

template <int LANES>
constexpr int THREADS = LANES > 256 ? LANES : 256;

// Sums over the lanes of a row, N at a time; the order is fixed.  Rows of whole workgroups go through
// LDS, by turns in two places, so that one barrier a call is enough.
template <int LANES, int N>
struct RowSum {
    static constexpr int PARTS = LANES > 64 ? LANES / 64 : 1;
    float part[2][N][PARTS];
};
template <int LANES, int N, int M>
__device__ __forceinline__ void row_sum(float (&x)[N], RowSum<LANES, M> &lds, int &turn) {
#pragma unroll
    for (int j = 0; j < N; ++j) {
        if constexpr (LANES < 16) {
#pragma unroll
            for (int d = 1; d < LANES; d *= 2) x[j] += __shfl_xor(x[j], d);
        } else {
            x[j] = row16_sum(x[j]);
        }
        if constexpr (LANES >= 32) x[j] += __shfl_xor(x[j], 16);
        if constexpr (LANES >= 64) x[j] += __shfl_xor(x[j], 32);
    }
    if constexpr (LANES > 64) {
        const int wave = threadIdx.x / 64;
        if ((threadIdx.x & 63) == 0)
#pragma unroll
            for (int j = 0; j < N; ++j) lds.part[turn][j][wave] = x[j];
        __syncthreads();
#pragma unroll
        for (int j = 0; j < N; ++j) {
            float s = 0.f;
#pragma unroll
            for (int w = 0; w < LANES / 64; ++w) s += lds.part[turn][j][w];
            x[j] = s;
        }
        turn ^= 1;
    }
}

template <int VEC, int LANES, int NV>
__device__ __forceinline__ void load_weight(float (&w)[NV][VEC], const float *p, bool on, int lane, int vecs) {
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int i = 0; i < VEC; ++i) w[k][i] = on && p && lane + k * LANES < vecs ? p[(lane + k * LANES) * VEC + i] : 1.f;
}

// Whether a lane keeps its weights from row to row.  A lane of the widest workgroups has 128 registers; with 16 numbers of
// a row it reads them again.
template <int VEC, int LANES, int NV>
constexpr bool KEEP = LANES < 1024 || VEC * NV <= 8;
template <int VEC, int LANES, int NV>
struct Weight {
    float w[KEEP<VEC, LANES, NV> ? NV : 1][VEC];
    const float *p;
    int lane, vecs;
    __device__ __forceinline__ void begin(const float *weight, bool on, int l, int v) {
        p = on ? weight : nullptr;
        lane = l;
        vecs = v;
        if constexpr (KEEP<VEC, LANES, NV>) load_weight<VEC, LANES, NV>(w, p, true, lane, vecs);
    }
    __device__ __forceinline__ float get(int k, int i) const {
        if constexpr (KEEP<VEC, LANES, NV>) return w[k][i];
        else return p && lane + k * LANES < vecs ? p[(lane + k * LANES) * VEC + i] : 1.f;
    }
};

// A lane's sums of a weight's gradient: in registers, or, where a lane of the widest workgroups has 16 numbers of a row, in
// its own places in LDS (1000 rows of 16384: 183 us, 255 with the sums in registers, more of which spill).
template <int VEC, int LANES, int NV>
struct Sums {
    static constexpr bool LDS = !KEEP<VEC, LANES, NV>;
    float s[LDS ? 1 : NV][VEC];
    float *own;
    __device__ __forceinline__ void begin(float *lds) {
        own = lds + threadIdx.x;
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                if constexpr (LDS) own[(k * VEC + i) * LANES] = 0.f;
                else s[k][i] = 0.f;
            }
    }
    __device__ __forceinline__ void add(int k, int i, float x, float y) {
        if constexpr (LDS) own[(k * VEC + i) * LANES] = fmaf(x, y, own[(k * VEC + i) * LANES]);
        else s[k][i] = fmaf(x, y, s[k][i]);
    }
    __device__ __forceinline__ float get(int k, int i) const {
        if constexpr (LDS) return own[(k * VEC + i) * LANES];
        else return s[k][i];
    }
};

// A row's vectors: the row is the same for all lanes of a workgroup (or a row's own where lanes share a wave), so a lane's
// address is one offset.
template <typename T, int VEC, int LANES, int NV>
__device__ __forceinline__ void load_rows(Raw<T, VEC> (&r)[NV], const void *p, int64_t at, int lane, int vecs) {
    const char *row = static_cast<const char *>(p) + at * (int64_t)sizeof(T);
    const uint32_t off = here(lane * (uint32_t)(VEC * sizeof(T)));
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        r[k].zero();
        if (lane + k * LANES < vecs) r[k].load(row + k * (int)(LANES * VEC * sizeof(T)), off);
    }
}
template <int LANES, typename T, int VEC>
__device__ __forceinline__ void store_row(const Raw<T, VEC> &r, void *p, int64_t at, int k, int lane, int vecs) {
    if (lane + k * LANES < vecs) r.store(static_cast<char *>(p) + at * (int64_t)sizeof(T) + k * (int)(LANES * VEC * sizeof(T)), here(lane * (uint32_t)(VEC * sizeof(T))));
}

__device__ __forceinline__ int64_t gate_row(const NormArgs &a, int64_t row) {
    const uint32_t token = (uint32_t)row / (uint32_t)a.heads, head = (uint32_t)row - token * (uint32_t)a.heads;  // fewer than 2^31 rows
    return token * a.gate_stride + head * a.gate_head;
}

// T: y, the gate and n; R: the residual stream
template <typename T, typename R, int VEC, int LANES, int NV>
__global__ __launch_bounds__(THREADS<LANES>) void norm_fwd_kernel(const NormArgs a) {
    constexpr int EACH = THREADS<LANES> / LANES;
    __shared__ RowSum<LANES, 1> lds;
    int turn = 0;
    const int lane = threadIdx.x % LANES, vecs = a.D / VEC;
    const float inv = 1.f / a.D;
    Weight<VEC, LANES, NV> wa, wb;
    wa.begin(a.wa, a.after, lane, vecs);
    wb.begin(a.wb, a.before, lane, vecs);
    for (int64_t row = (int64_t)blockIdx.x * EACH + (EACH > 1 ? threadIdx.x / LANES : 0); row < a.rows; row += (int64_t)gridDim.x * EACH) {
        Raw<T, VEC> y[NV], z[NV];
        Raw<R, VEC> x[NV];
        load_rows<T, VEC, LANES, NV>(y, a.y, row * a.D, lane, vecs);
        if (a.gate) load_rows<T, VEC, LANES, NV>(z, a.gate, gate_row(a, row), lane, vecs);
        if (a.residual) load_rows<R, VEC, LANES, NV>(x, a.residual, row * a.D, lane, vecs);
        float r = a.scale;
        if (a.after) {
            float s[1] = {0.f};
#pragma unroll
            for (int k = 0; k < NV; ++k)
#pragma unroll
                for (int i = 0; i < VEC; ++i) s[0] = fmaf(y[k].get(i), y[k].get(i), s[0]);
            row_sum<LANES>(s, lds, turn);
            r *= __builtin_amdgcn_rsqf(fmaf(s[0], inv, a.eps));
        }
        float h[NV][VEC], q[1] = {0.f};
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            Raw<R, VEC> o;
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                float p = y[k].get(i) * r * wa.get(k, i);
                if (a.gate) {
                    const float g = z[k].get(i), s = sigmoid_f32(g);
                    p *= a.silu ? g * s : s;
                }
                if (a.residual) p += x[k].get(i);
                h[k][i] = p;
                q[0] = fmaf(p, p, q[0]);
                o.set(i, p);
            }
            store_row<LANES>(o, a.h, row * a.D, k, lane, vecs);
        }
        if (!a.before) continue;
        row_sum<LANES>(q, lds, turn);
        const float rh = __builtin_amdgcn_rsqf(fmaf(q[0], inv, a.eps));
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            Raw<T, VEC> o;
#pragma unroll
            for (int i = 0; i < VEC; ++i) o.set(i, h[k][i] * rh * wb.get(k, i));
            store_row<LANES>(o, a.n, row * a.D, k, lane, vecs);
        }
    }
}

// Gradients.  With u = h r', v = y r and <.> the mean over the row:
//   dh = d_h + r' (d_n w_before - u <d_n w_before u>),        d w_before += d_n u,   d residual = dh
//   dp = scale act(gate) dh,   d gate = scale act'(gate) p dh
//   dy = r (dp w_after - v <dp w_after v>),                    d w_after += dp v
template <typename T, typename R, int VEC, int LANES, int NV>
__global__ __launch_bounds__(THREADS<LANES>) void norm_bwd_kernel(const NormArgs a) {
    constexpr int EACH = THREADS<LANES> / LANES;
    __shared__ RowSum<LANES, 3> lds;
    int turn = 0;
    const int lane = threadIdx.x % LANES, vecs = a.D / VEC;
    const float inv = 1.f / a.D;
    Sums<VEC, LANES, NV> da, db;
    __shared__ float in_lds[Sums<VEC, LANES, NV>::LDS ? 2 : 1][Sums<VEC, LANES, NV>::LDS ? NV * VEC * LANES : 1];
    da.begin(in_lds[0]);
    db.begin(in_lds[Sums<VEC, LANES, NV>::LDS ? 1 : 0]);
    Weight<VEC, LANES, NV> wa, wb;
    wa.begin(a.wa, a.after, lane, vecs);
    wb.begin(a.wb, a.before, lane, vecs);
    for (int64_t row = (int64_t)blockIdx.x * EACH + (EACH > 1 ? threadIdx.x / LANES : 0); row < a.rows; row += (int64_t)gridDim.x * EACH) {
        const int64_t at = row * a.D;
        Raw<T, VEC> y[NV], z[NV], dn[NV];
        Raw<R, VEC> h[NV], dh[NV];
        load_rows<T, VEC, LANES, NV>(y, a.y, at, lane, vecs);
        if (a.gate) load_rows<T, VEC, LANES, NV>(z, a.gate, gate_row(a, row), lane, vecs);
        if (a.d_h) load_rows<R, VEC, LANES, NV>(dh, a.d_h, at, lane, vecs);
        if (a.before) {
            load_rows<R, VEC, LANES, NV>(h, a.h_in, at, lane, vecs);
            load_rows<T, VEC, LANES, NV>(dn, a.d_n, at, lane, vecs);
        }
        float s[3] = {0.f, 0.f, 0.f};  // y^2, h^2, d_n w_before h
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                s[0] = fmaf(y[k].get(i), y[k].get(i), s[0]);
                if (a.before) {
                    const float x = h[k].get(i);
                    s[1] = fmaf(x, x, s[1]);
                    s[2] = fmaf(dn[k].get(i) * wb.get(k, i), x, s[2]);
                }
            }
        if (a.before || a.after) row_sum<LANES>(s, lds, turn);
        const float r = a.after ? __builtin_amdgcn_rsqf(fmaf(s[0], inv, a.eps)) : 1.f;
        const float rh = a.before ? __builtin_amdgcn_rsqf(fmaf(s[1], inv, a.eps)) : 0.f, mean = s[2] * inv * rh * rh;
        float dp[NV][VEC], q[1] = {0.f};
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            Raw<R, VEC> ox;
            Raw<T, VEC> oz;
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                float g = a.d_h ? dh[k].get(i) : 0.f;
                if (a.before) {
                    const float x = h[k].get(i), d = dn[k].get(i);
                    g = fmaf(rh, fmaf(d, wb.get(k, i), -x * mean), g);
                    db.add(k, i, d * rh, x);
                    ox.set(i, g);
                }
                g *= a.scale;
                const float v = y[k].get(i) * r;
                if (a.gate) {
                    const float t = z[k].get(i);
                    float f;  // 1 - e
                    const float e = sigmoid_f32(t, f);
                    oz.set(i, g * v * wa.get(k, i) * (a.silu ? e * fmaf(t, f, 1.f) : e * f));
                    g *= a.silu ? t * e : e;
                }
                da.add(k, i, g, v);
                dp[k][i] = g * wa.get(k, i);
                q[0] = fmaf(dp[k][i], v, q[0]);
            }
            if (a.before && a.d_res) store_row<LANES>(ox, a.d_res, at, k, lane, vecs);
            if (a.gate) store_row<LANES>(oz, a.d_gate, at, k, lane, vecs);
        }
        if (a.after) row_sum<LANES>(q, lds, turn);
        const float back = a.after ? q[0] * inv * r : 0.f;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            Raw<T, VEC> o;
#pragma unroll
            for (int i = 0; i < VEC; ++i) o.set(i, a.after ? r * fmaf(-back, y[k].get(i), dp[k][i]) : dp[k][i]);  // without the norm no y, which may be infinite
            store_row<LANES>(o, a.dy, at, k, lane, vecs);
        }
    }
    if (!a.part) return;
    if constexpr (EACH > 1) {  // the rows of a workgroup, in their order
        __shared__ float all[EACH][LANES * NV * VEC];
        const int group = threadIdx.x / LANES;
#pragma unroll
        for (int w = 0; w < 2; ++w) {
            if (w) __syncthreads();
#pragma unroll
            for (int k = 0; k < NV; ++k)
#pragma unroll
                for (int i = 0; i < VEC; ++i) all[group][(lane + k * LANES) * VEC + i] = w ? db.get(k, i) : da.get(k, i);
            __syncthreads();
            for (int c = threadIdx.x; c < a.D; c += THREADS<LANES>) {
                float x = 0.f;
#pragma unroll
                for (int g = 0; g < EACH; ++g) x += all[g][c];
                a.part[((int64_t)blockIdx.x * 2 + w) * a.D + c] = x;
            }
        }
    } else {
#pragma unroll
        for (int k = 0; k < NV; ++k)
            if (lane + k * LANES < vecs)
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    const int64_t at = (int64_t)blockIdx.x * 2 * a.D + (lane + k * LANES) * VEC + i;
                    a.part[at] = da.get(k, i);
                    a.part[at + a.D] = db.get(k, i);
                }
    }
}

// Workgroups: enough to fill the chip, each with rows enough to pay for its weights (and, in the
// backward pass, for the sums that it writes).
template <bool BWD, typename T, typename R, int VEC, int LANES, int NV>
hipError_t launch(NormArgs &a, hipStream_t stream) {
    constexpr int EACH = THREADS<LANES> / LANES;
    const int64_t need = (a.rows + EACH - 1) / EACH, most = BWD ? a.groups : 2048;
    a.groups = (int)(need < most ? need : most);
    const dim3 grid((unsigned)a.groups), block(THREADS<LANES>);
    if constexpr (BWD) hipLaunchKernelGGL((norm_bwd_kernel<T, R, VEC, LANES, NV>), grid, block, 0, stream, a);
    else hipLaunchKernelGGL((norm_fwd_kernel<T, R, VEC, LANES, NV>), grid, block, 0, stream, a);
    return hipGetLastError();
}

template <bool BWD, typename T, typename R, int VEC>
hipError_t by_width(NormArgs &a, hipStream_t stream) {
    const int vecs = a.D / VEC;
    if constexpr (VEC > 2) {
        if (vecs <= 4) return launch<BWD, T, R, VEC, 4, 1>(a, stream);
        if (vecs <= 16) return launch<BWD, T, R, VEC, 16, 1>(a, stream);
        if (vecs <= 32) return launch<BWD, T, R, VEC, 32, 1>(a, stream);
        if (vecs <= 64) return launch<BWD, T, R, VEC, 64, 1>(a, stream);
        if (vecs <= 256) return launch<BWD, T, R, VEC, 256, 1>(a, stream);
        if (vecs <= 512) return launch<BWD, T, R, VEC, 512, 1>(a, stream);
        if (vecs <= 1024) return launch<BWD, T, R, VEC, 512, 2>(a, stream);
        if (vecs <= 2048) return launch<BWD, T, R, VEC, 1024, 2>(a, stream);
        if constexpr (VEC == 4)
            if (vecs <= 4096) return launch<BWD, T, R, VEC, 1024, 4>(a, stream);
    } else {  // rows off a 16-byte border: two numbers at a time where the width is even, one where it is odd
        constexpr int TWO = VEC == 2 ? 1 : 2;
        if (vecs <= 16 * 2 * TWO) return launch<BWD, T, R, VEC, 16, 2 * TWO>(a, stream);
        if (vecs <= 64 * 4 * TWO) return launch<BWD, T, R, VEC, 64, 4 * TWO>(a, stream);
        if (vecs <= 256 * 4 * TWO) return launch<BWD, T, R, VEC, 256, 4 * TWO>(a, stream);
        if (vecs <= 512 * 8 * TWO) return launch<BWD, T, R, VEC, 512, 8 * TWO>(a, stream);
        if (vecs <= 1024 * 8 * TWO) return launch<BWD, T, R, VEC, 1024, 8 * TWO>(a, stream);
    }
    return hipErrorNotSupported;
}

template <bool BWD>
hipError_t by_type(NormArgs &a, bool fp32, bool h_fp32, int vec, hipStream_t stream) {
    if (fp32) return vec > 2 ? by_width<BWD, float, float, 4>(a, stream) : vec == 2 ? by_width<BWD, float, float, 2>(a, stream) : by_width<BWD, float, float, 1>(a, stream);
    if (h_fp32) return vec > 2 ? by_width<BWD, __bf16, float, 8>(a, stream) : vec == 2 ? by_width<BWD, __bf16, float, 2>(a, stream) : by_width<BWD, __bf16, float, 1>(a, stream);
    return vec > 2 ? by_width<BWD, __bf16, __bf16, 8>(a, stream) : vec == 2 ? by_width<BWD, __bf16, __bf16, 2>(a, stream) : by_width<BWD, __bf16, __bf16, 1>(a, stream);
}

}  // namespace

// Workgroups of the backward pass, each with sums of its own: two a compute unit, or the one that fits of the widest.
int norm_groups(int64_t rows, int D) {
    const int most = D > 8192 ? 256 : 512;
    return (int)(rows < most ? rows : most);
}

hipError_t launch_norm_fwd(NormArgs a, bool fp32, bool h_fp32, int vec, hipStream_t stream) {
    return by_type<false>(a, fp32, h_fp32, vec, stream);
}

hipError_t launch_norm_bwd(NormArgs a, bool fp32, bool h_fp32, int vec, float *d_wa, float *d_wb, hipStream_t stream) {
    const hipError_t e = by_type<true>(a, fp32, h_fp32, vec, stream);
    if (e != hipSuccess || !a.part) return e;
    return launch_column_sums(ColumnSums{a.part, a.groups, 2 * a.D, a.D, 1, d_wa, d_wb}, stream);
}

}  // namespace kda
