// kda_gdr_step.hip -- decoding one or several tokens a request over a pool of states, with a
// decay per value head or per channel: the token loop of the gated delta rule in float32,
//   Sbar = e^g S,  d = beta (v - Sbar^T k),  o = scale Sbar^T q + scale (k.q) d,  S = Sbar + k d^T
// (reading Sbar and adding (k.q) d is reading S after its update, without a second pass).
//
// Bound by the state's bytes: one read for each request and head, one write for each kept
// token.  A wave owns CW = 32 value columns of one (request, head): lane (r, c) holds K / RG
// key rows of four columns in registers, so a row's piece is one whole cache line, the sums
// over key rows stay inside the wave, and no wave waits for another.  64 requests x 96 heads, K =
// V = 128, bf16, one token: 146 to 156 us for 0.81 GB over states that do not fit the last-level
// cache (5.2 to 5.5 TB/s; a large device copy reaches 5.0); 24 requests of 1 to 5 tokens x 32
// heads: 37 to 39 us for 0.2 GB.
#include "kda_gdr_step.h"

namespace kda {
namespace {

// Sum over the lanes that differ in the bits of `lane` from STEP upwards.
template <int STEP>
__device__ __forceinline__ float rows_sum(float x) {
#pragma unroll
    for (int d = STEP; d < 64; d *= 2) x += __shfl_xor(x, d);
    return x;
}

template <int N>
__device__ __forceinline__ void load_row(float (&x)[N], const __bf16 *p) {
    if constexpr (N >= 8) {
#pragma unroll
        for (int i = 0; i < N; i += 8) {
            const bf16x8 b = *reinterpret_cast<const bf16x8 *>(p + i);
#pragma unroll
            for (int j = 0; j < 8; ++j) x[i + j] = (float)b[j];
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] = (float)p[i];
    }
}
template <int N>
__device__ __forceinline__ void load_row(float (&x)[N], const float *p) {
    if constexpr (N >= 4) {
#pragma unroll
        for (int i = 0; i < N; i += 4) *reinterpret_cast<f4 *>(x + i) = *reinterpret_cast<const f4 *>(p + i);
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] = p[i];
    }
}

template <typename T, int R, bool CHANNELS>
struct Token {
    float k[R], q[R], v[4], g[CHANNELS ? R : 1], beta;
    __device__ __forceinline__ void load(const GdrStepArgs &a, int64_t bt, int hv, int K, int row, int col) {
        const int64_t at = (bt * a.HK + hv / a.group) * K + row, h = bt * a.HV + hv;
        load_row<R>(k, static_cast<const T *>(a.k) + at);
        load_row<R>(q, static_cast<const T *>(a.q) + at);
        load_row<4>(v, static_cast<const T *>(a.v) + h * a.V + col);
        if constexpr (CHANNELS) load_row<R>(g, a.g + h * K + row);
        else g[0] = a.g[h];
        beta = a.beta[h];
    }
};

template <typename T, int K, int CW, bool CHANNELS>
__global__ __launch_bounds__(256) void gdr_step_kernel(const GdrStepArgs a, int units) {
    constexpr int CQ = CW / 4, RG = 64 / CQ, R = K / RG;  // column quads, row groups, rows of a lane
    const int unit = blockIdx.x * (blockDim.x / 64) + __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    if (unit >= units) return;
    const int VB = a.V / CW, vb = unit % VB, hv = unit / VB % a.HV, b = unit / VB / a.HV;
    const int lane = threadIdx.x & 63, row = lane / CQ * R, col = CW * vb + lane % CQ * 4;
    int len = a.lengths ? a.lengths[b] : a.S;
    len = len < 0 ? 0 : len > a.S ? a.S : len;
    if (len == 0) return;
    Token<T, R, CHANNELS> t;
    t.load(a, (int64_t)b * a.S, hv, K, row, col);

    // slots are read, and bounded, on the device; one outside the pool holds no state
    auto slot = [&](int i) -> int64_t {
        const int64_t s = a.slots ? a.slots[(int64_t)b * a.slot_cols + i] : b;
        return s < 0 || s >= a.pool ? -1 : s;
    };
    const int first = a.start ? a.start[b] : 0;
    const int64_t from = first < 0 || first >= a.slot_cols ? -1 : slot(first);
    f4 S[R];
#pragma unroll
    for (int i = 0; i < R; ++i) S[i] = f4{};
    const int64_t at = (int64_t)hv * K * a.V + (int64_t)row * a.V + col, each = (int64_t)a.HV * K * a.V;
    if (from >= 0)
#pragma unroll
        for (int i = 0; i < R; ++i) S[i] = *reinterpret_cast<const f4 *>(a.states + from * each + at + (int64_t)i * a.V);

    for (int i = 0; i < len; ++i) {
        Token<T, R, CHANNELS> next;
        if (i + 1 < len) next.load(a, (int64_t)b * a.S + i + 1, hv, K, row, col);
        f4 p = {}, r = {};
        float kq = 0.f;
        const float g0 = expf(t.g[0]);
#pragma unroll
        for (int j = 0; j < R; ++j) {
            S[j] *= CHANNELS ? (j ? expf(t.g[j]) : g0) : g0;
            p += t.k[j] * S[j];
            r += t.q[j] * S[j];
            kq += t.k[j] * t.q[j];
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            p[e] = rows_sum<CQ>(p[e]);
            r[e] = rows_sum<CQ>(r[e]);
        }
        kq = rows_sum<CQ>(kq);
        f4 d, o;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            d[e] = t.beta * (t.v[e] - p[e]);
            o[e] = a.scale * (r[e] + kq * d[e]);
        }
#pragma unroll
        for (int j = 0; j < R; ++j) S[j] += t.k[j] * d;
        if (row == 0) {
            const int64_t y = (((int64_t)b * a.S + i) * a.HV + hv) * a.V + col;
#pragma unroll
            for (int e = 0; e < 4; ++e) st_out(a.out, a.out_bf16, y + e, o[e]);
        }
        // a state leaves after every token that has a slot of its own, or after the last
        const int64_t to = a.slot_cols > 1 ? slot(i) : i + 1 == len ? slot(0) : -1;
        if (to >= 0)
#pragma unroll
            for (int j = 0; j < R; ++j)
                __builtin_nontemporal_store(S[j], reinterpret_cast<f4 *>(a.states + to * each + at + (int64_t)j * a.V));
        t = next;
    }
}

template <typename T, int K, int CW, bool CHANNELS>
hipError_t launch(const GdrStepArgs &a, hipStream_t stream) {
    const int64_t units = (int64_t)a.B * a.HV * (a.V / CW);
    const int waves = units > 4 * device_cu_count() ? 4 : 1;  // few waves go to a compute unit each
    hipLaunchKernelGGL((gdr_step_kernel<T, K, CW, CHANNELS>), dim3((unsigned)((units + waves - 1) / waves)), dim3(64 * waves), 0, stream, a,
                       (int)units);
    return hipGetLastError();
}
template <typename T, int K>
hipError_t by_form(const GdrStepArgs &a, hipStream_t stream) {
    if (a.V == 16) return a.channels ? launch<T, K, 16, true>(a, stream) : launch<T, K, 16, false>(a, stream);
    return a.channels ? launch<T, K, 32, true>(a, stream) : launch<T, K, 32, false>(a, stream);
}
template <typename T>
hipError_t by_width(const GdrStepArgs &a, int K, hipStream_t stream) {
    switch (K) {
        case 16: return by_form<T, 16>(a, stream);
        case 32: return by_form<T, 32>(a, stream);
        case 64: return by_form<T, 64>(a, stream);
        case 128: return by_form<T, 128>(a, stream);
    }
    return hipErrorNotSupported;
}

}  // namespace

hipError_t launch_gdr_step(const GdrStepArgs &a, bool fp32, int K, hipStream_t stream) {
    return fp32 ? by_width<float>(a, K, stream) : by_width<__bf16>(a, K, stream);
}

}  // namespace kda
