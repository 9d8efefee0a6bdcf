// kda_draft_verify.hip -- drafted tokens against the target's probabilities.  Draft i holds
// while u_i q_i(x_i) < p_i(x_i); behind the last that holds, one token is drawn from the
// residual max(p - q, 0) (or from p) as the first whose running sum of weights passes u times
// their whole.  The weights are whole numbers of 2^-44, so their sums, and the token drawn,
// do not depend on the order in which they are added: probabilities of float32 are exact down
// to 2^-44, and the whole of 2^19 of them fits 64 bits.
//
// Bound by reading the target's row, and the draft's where a draft was refused.  Two kernels: one
// wave for every 1024 tokens of the row that is drawn from writes the sums of its weights, then one
// workgroup a request walks the sums and looks inside one tile.  192 requests over 131,072 tokens:
// 44 us and 6 us for 0.15 GB (half of the requests have a draft refused; a copy would take 30), 32
// us and 5 us for 0.10 GB where the drafts were certain; one request over 32,768 tokens: 16 to 20
// us a call, the host's time for two launches.
#include "kda_gdr_step.h"

namespace kda {
namespace {

constexpr int TILE = DRAFT_TILE;
typedef unsigned long long u64;

// A weight in units of 2^-44: clamped to [0, 1], cut to whole units, NaN counts as nothing.
__device__ __forceinline__ u64 weight(double w) {
    w = fmin(fmax(w, 0.0), 1.0) * 4096.0;
    const unsigned hi = (unsigned)w;
    return ((u64)hi << 32) + (unsigned)((w - hi) * 4294967296.0);
}

template <typename V>
__device__ __forceinline__ V wave_sum(V x) {
#pragma unroll
    for (int d = 32; d; d /= 2) x += __shfl_xor(x, d);
    return x;
}

// How many drafts hold (one wave, every lane gets it), and how many there were.
__device__ __forceinline__ int accept(const DraftVerifyArgs &a, int b, int &n) {
    const int lane = threadIdx.x & 63;
    n = a.lengths ? a.lengths[b] : a.D;
    n = n < 0 ? 0 : n > a.D ? a.D : n;
    for (int i0 = 0; i0 < n; i0 += 64) {
        const int i = i0 + lane;
        bool holds = false;
        if (i < n) {
            const int x = a.x[(int64_t)b * a.D + i];
            if (x >= 0 && x < a.vocab) {  // a token outside the vocabulary is refused
                const double p = a.target[((int64_t)b * (a.D + 1) + i) * a.vocab + x];
                const double q = a.draft ? a.draft[((int64_t)b * a.D + i) * a.vocab + x] : 1.f;
                holds = a.u[(int64_t)b * (a.D + 1) + i] * q < p;
            }
        }
        const u64 no = __ballot(!holds);
        if (no) return i0 + __builtin_ctzll(no) < n ? i0 + __builtin_ctzll(no) : n;
    }
    return n;
}

// The row that is drawn from: p - q at a token.
struct Row {
    const float *p, *q;  // q: null where nothing is taken off, or the draft is one token
    int x;               // that token, -1 if none
    __device__ __forceinline__ Row(const DraftVerifyArgs &a, int b, int taken, int n) {
        p = a.target + ((int64_t)b * (a.D + 1) + taken) * a.vocab;
        q = taken < n && a.draft ? a.draft + ((int64_t)b * a.D + taken) * a.vocab : nullptr;
        x = taken < n && !a.draft ? a.x[(int64_t)b * a.D + taken] : -1;
    }
    __device__ __forceinline__ double off(int i) const { return q ? (double)q[i] : i == x ? 1.0 : 0.0; }
};

__global__ __launch_bounds__(256) void draft_sums_kernel(const DraftVerifyArgs a) {
    const int64_t unit = (int64_t)blockIdx.x * 4 + threadIdx.x / 64;
    if (unit >= (int64_t)a.B * a.tiles) return;
    const int b = (int)(unit / a.tiles), tile = (int)(unit % a.tiles), lane = threadIdx.x & 63;
    int n;
    const int taken = accept(a, b, n);
    const Row row(a, b, taken, n);
    u64 rest = 0, all = 0;
#pragma unroll 4
    for (int i = tile * TILE + lane; i < (tile + 1) * TILE; i += 64) {
        if (i >= a.vocab) break;
        const double p = row.p[i];
        rest += weight(p - row.off(i));
        all += weight(p);
    }
    rest = wave_sum(rest);
    all = wave_sum(all);
    if (lane == 0) {
        a.sums[unit * 2] = rest;
        a.sums[unit * 2 + 1] = all;
    }
}

// Running sums over the 256 threads of a workgroup; `whole` is all of them.
__device__ __forceinline__ u64 running(u64 x, u64 *s, u64 &whole) {
    const int lane = threadIdx.x & 63, w = threadIdx.x / 64;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const u64 up = __shfl_up(x, d);
        if (lane >= d) x += up;
    }
    __syncthreads();  // s may still be read
    if (lane == 63) s[w] = x;
    __syncthreads();
    u64 before = 0;
    whole = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        before += i < w ? s[i] : 0;
        whole += s[i];
    }
    return before + x;
}

__global__ __launch_bounds__(256) void draft_pick_kernel(const DraftVerifyArgs a) {
    __shared__ u64 s[4], at_sum;
    __shared__ int at_tile, picked;
    const int b = blockIdx.x, tid = threadIdx.x;
    int n;
    const int taken = accept(a, b, n);
    const Row row(a, b, taken, n);
    const u64 *sums = a.sums + (int64_t)b * a.tiles * 2;
    const int each = (a.tiles + 255) / 256;
    u64 rest = 0, all = 0, whole, whole_all;
    for (int i = tid * each; i < (tid + 1) * each && i < a.tiles; ++i) {
        rest += sums[2 * i];
        all += sums[2 * i + 1];
    }
    u64 end = running(rest, s, whole), end_all = running(all, s, whole_all);
    const bool plain = whole == 0;  // nothing is left of the residual: drawn from p itself
    if (plain) {
        end = end_all;
        rest = all;
        whole = whole_all;
    }
    // a uniform number of 1 or more draws the last token that has weight; NaN or one below 0 is taken as
    // 0 and draws the first
    const double t0 = a.u[(int64_t)b * (a.D + 1) + a.D] * (double)whole;
    u64 t = t0 > 0.0 ? t0 < 9.2e18 ? (u64)t0 : ~0ull : 0;
    if (whole && t >= whole) t = whole - 1;
    if (tid == 0) {
        at_tile = 0;
        at_sum = 0;
        picked = 0;  // no weight at all: the first token
    }
    __syncthreads();
    if (end > t && end - rest <= t) {  // the one thread whose tiles hold it
        u64 sum = end - rest;
        for (int i = tid * each; i < (tid + 1) * each && i < a.tiles; ++i) {
            const u64 w = sums[2 * i + plain];
            if (sum + w > t) {
                at_tile = i;
                at_sum = sum;
                break;
            }
            sum += w;
        }
    }
    __syncthreads();
    u64 w[TILE / 256], sum = 0, tile_whole;
    const int first = at_tile * TILE + tid * (TILE / 256);
#pragma unroll
    for (int i = 0; i < TILE / 256; ++i) {
        w[i] = first + i < a.vocab ? weight((double)row.p[first + i] - (plain ? 0.0 : row.off(first + i))) : 0;
        sum += w[i];
    }
    u64 run = at_sum + running(sum, s, tile_whole) - sum;
#pragma unroll
    for (int i = 0; i < TILE / 256; ++i) {
        if (run <= t && run + w[i] > t) picked = first + i;
        run += w[i];
    }
    __syncthreads();
    for (int i = tid; i <= a.D; i += 256)
        a.tokens[(int64_t)b * (a.D + 1) + i] = i < taken ? a.x[(int64_t)b * a.D + i] : i == taken ? picked : -1;
    if (tid == 0) a.accepted[b] = taken;
}

}  // namespace

hipError_t launch_draft_verify(const DraftVerifyArgs &a, hipStream_t stream) {
    const int64_t units = (int64_t)a.B * a.tiles;
    hipLaunchKernelGGL(draft_sums_kernel, dim3((unsigned)((units + 3) / 4)), dim3(256), 0, stream, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(draft_pick_kernel, dim3(a.B), dim3(256), 0, stream, a);
    return hipGetLastError();
}

}  // namespace kda
