// kda_rows_api.hip -- the C entry points of what stands around the recurrence in a layer (the short
// convolution, the gated linear recurrence, the norms between blocks): argument validation, the
// empty cases, workspaces.
#include <initializer_list>

#include "../../include/kda.h"
#include "kda_rows.h"

namespace {

kda_status done(hipError_t e) {
    if (e == hipSuccess) return KDA_OK;
    kda::record_hip_error(e);
    return e == hipErrorNotSupported ? KDA_ERR_UNSUPPORTED : KDA_ERR_HIP;
}

bool type_ok(kda_dtype t) { return t == KDA_F32 || t == KDA_BF16; }
size_t size_of(kda_dtype t) { return t == KDA_F32 ? 4 : 2; }

constexpr int64_t MAX_ROWS = INT32_MAX - 64;    // a row's number, and a tile's end, fit 32 bits
constexpr int64_t MAX_CHANNELS = 1 << 20;
constexpr int64_t MAX_GRID = (int64_t)1 << 31;  // threads of a grid, half of what a launch takes

// Whether rows can be read (and written) `unit` numbers at a time, at most 16 bytes of them in one load: for rows `n` numbers of `size` bytes apart.
struct Units {
    int unit;
    bool ok = true;
    Units &rows(const void *p, size_t size, int64_t n) {
        ok = ok && (!p || ((uintptr_t)p % (unit * size < 16 ? unit * size : 16) == 0 && n % unit == 0));
        return *this;
    }
};
// Whether any of them is off a border of `size` bytes; looked at before a call without rows returns, which fills outputs too.
bool misaligned(size_t size, std::initializer_list<const void *> ps) {
    for (const void *p : ps)
        if ((uintptr_t)p % size != 0) return true;
    return false;
}

// No output may be an input or another output.
template <int I, int O>
bool aliased(const void *const (&ins)[I], const void *const (&outs)[O]) {
    for (int i = 0; i < O; ++i) {
        if (!outs[i]) continue;
        for (const void *p : ins)
            if (p == outs[i]) return true;
        for (int j = 0; j < i; ++j)
            if (outs[j] == outs[i]) return true;
    }
    return false;
}

// The sequences of a batch.  KDA_OK with *empty set: there is no row.
kda_status batch(kda::Seqs &s, const int32_t *cu, int num_seqs, int B, int64_t T, bool *empty) {
    if (B < 0 || T < 0) return KDA_ERR_BAD_SHAPE;
    if (cu && (B != 1 || num_seqs < 0 || (num_seqs == 0 && T > 0))) return KDA_ERR_BAD_ARGUMENT;
    s.cu = cu;
    s.N = cu ? num_seqs : B;
    s.T = T;
    *empty = B == 0 || T == 0 || s.N == 0;
    if (!*empty && T > MAX_ROWS / B) return KDA_ERR_UNSUPPORTED;
    s.rows = *empty ? 0 : B * T;
    return KDA_OK;
}

// dst = src or zeros, n numbers of `size` bytes
kda_status fill(void *dst, const void *src, int64_t n, size_t size, hipStream_t stream) {
    if (!dst || n <= 0) return KDA_OK;
    return done(kda::launch_fill_bytes(dst, src, n * (int64_t)size, stream));
}

kda_status pool_args(kda::Slots &s, const int32_t *slots, int slot_cols, const int32_t *start, const int32_t *lengths, int64_t pool, int B, int S) {
    if (slot_cols != 1 && slot_cols != S) return KDA_ERR_BAD_SHAPE;
    if (!slots && (slot_cols != 1 || start || pool < B)) return KDA_ERR_BAD_ARGUMENT;
    if (start && slot_cols != S) return KDA_ERR_BAD_ARGUMENT;
    s.slots = slots;
    s.start = start;
    s.lengths = lengths;
    s.pool = pool;
    s.S = S;
    s.cols = slot_cols;
    return KDA_OK;
}

kda_status conv_shape(kda_dtype dtype, int D, int W, unsigned flags) {
    if (D <= 0 || W <= 0) return KDA_ERR_BAD_SHAPE;
    if (!type_ok(dtype)) return KDA_ERR_BAD_DTYPE;
    if (flags & ~KDA_SILU) return KDA_ERR_BAD_ARGUMENT;
    if (W < 2 || W > 4 || D > MAX_CHANNELS) return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}
// lanes of all runs, or of all the states' numbers
bool conv_fits(const kda::Seqs &s, int D, int W) {
    int run, runs;
    kda::conv_runs(s.rows, D, run, runs);
    return (int64_t)runs * ((D + 63) / 64 * 64) < MAX_GRID && (int64_t)s.N * (W - 1) * D < MAX_GRID;
}

kda_status glr_gates(kda::GlrGates &g, const void *gate, int64_t gate_stride, const float *log_scale, const float *bias, float lower_bound,
                     const void *in_gate, int64_t in_stride, unsigned flags, int H, int K) {
    if (H <= 0 || K <= 0) return KDA_ERR_BAD_SHAPE;
    if (flags & ~KDA_GLR_NORMALIZE) return KDA_ERR_BAD_ARGUMENT;
    if (log_scale && !(lower_bound < 0.f)) return KDA_ERR_BAD_ARGUMENT;
    if (!log_scale && bias) return KDA_ERR_BAD_ARGUMENT;
    if ((int64_t)H * K > MAX_CHANNELS) return KDA_ERR_UNSUPPORTED;
    g.gate = gate;
    g.log_scale = log_scale;
    g.bias = bias;
    g.in_gate = in_gate;
    g.gate_stride = gate_stride;
    g.in_stride = in_stride;
    g.lower = lower_bound;
    g.normalize = (flags & KDA_GLR_NORMALIZE) != 0;
    g.K = K;
    return KDA_OK;
}
bool glr_fits(const kda::Seqs &s, int C) {
    const int64_t tiles = (s.rows + 63) / 64;  // where there are many
    return tiles * ((C + 63) / 64 * 64) < MAX_GRID && (int64_t)s.N * C < MAX_GRID;
}
// a workspace of which nothing is used is not empty: 0 says that there is no such call
size_t some(size_t bytes) { return bytes ? bytes : 256; }
int64_t glr_kept_rows(int64_t rows) { return (rows + kda::GLR_KEPT - 1) / kda::GLR_KEPT; }

kda_status norm_shape(kda_dtype dtype, kda_dtype h_dtype, int64_t tokens, int heads, int D, float eps, unsigned flags) {
    if (tokens < 0 || heads <= 0 || D <= 0) return KDA_ERR_BAD_SHAPE;
    if (!type_ok(dtype) || !type_ok(h_dtype) || (dtype == KDA_F32 && h_dtype != KDA_F32)) return KDA_ERR_BAD_DTYPE;
    if ((flags & ~(KDA_NORM_AFTER | KDA_NORM_BEFORE | KDA_SILU)) || !(eps >= 0.f)) return KDA_ERR_BAD_ARGUMENT;
    if (D > KDA_NORM_MAX_D || tokens > (int64_t)INT32_MAX / heads) return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}

}  // namespace

extern "C" {

kda_status kda_short_conv_fwd(const void *x, int64_t x_stride, kda_dtype dtype, const float *weight, const float *bias,
                              const void *initial_state, void *final_state, const int32_t *cu_seqlens, int num_seqs, int B,
                              int64_t T, int D, int W, unsigned flags, void *out, hipStream_t stream) {
    kda_status st = conv_shape(dtype, D, W, flags);
    if (st != KDA_OK) return st;
    kda::ConvArgs a{};
    bool empty;
    st = batch(a.seqs, cu_seqlens, num_seqs, B, T, &empty);
    if (st != KDA_OK) return st;
    if (x_stride < D) return KDA_ERR_BAD_SHAPE;
    if (final_state && final_state == initial_state) return KDA_ERR_ALIAS;
    if (misaligned(size_of(dtype), {x, initial_state, final_state, out}) || misaligned(4, {weight, bias, cu_seqlens})) return KDA_ERR_BAD_ARGUMENT;
    if (empty) return fill(final_state, initial_state, (int64_t)a.seqs.N * (W - 1) * D, size_of(dtype), stream);
    if (!conv_fits(a.seqs, D, W)) return KDA_ERR_UNSUPPORTED;
    if (!x || !weight || !out) return KDA_ERR_NULL_POINTER;
    const void *ins[] = {x, weight, bias, initial_state, cu_seqlens}, *outs[] = {out, final_state};
    if (aliased(ins, outs)) return KDA_ERR_ALIAS;
    a.x = x;
    a.x_stride = x_stride;
    a.weight = weight;
    a.bias = bias;
    a.s0 = initial_state;
    a.sf = final_state;
    a.D = D;
    a.W = W;
    a.silu = (flags & KDA_SILU) != 0;
    a.out = out;
    const size_t e = size_of(dtype);
    Units w{kda::CONV_FWD_VEC};
    w.rows(x, e, x_stride).rows(initial_state, e, D).rows(final_state, e, D).rows(out, e, D);
    return done(kda::launch_conv_fwd(a, dtype == KDA_F32, w.ok, stream));
}

size_t kda_short_conv_bwd_workspace_size(kda_dtype dtype, int B, int64_t T, int D, int W) {
    kda::Seqs s{};
    bool empty;
    if (conv_shape(dtype, D, W, 0) != KDA_OK || batch(s, nullptr, 0, B, T, &empty) != KDA_OK || empty || !conv_fits(s, D, W)) return 0;
    // the widest and the narrowest loads go by runs of their own length; both fit
    int run, wide, narrow;
    kda::conv_runs(s.rows, D / kda::CONV_BWD_VEC > 0 ? D / kda::CONV_BWD_VEC : 1, run, wide);
    kda::conv_runs(s.rows, D, run, narrow);
    return (size_t)(wide > narrow ? wide : narrow) * (W + 1) * D * sizeof(float);
}

kda_status kda_short_conv_bwd(const void *x, int64_t x_stride, kda_dtype dtype, const float *weight, const float *bias,
                              const void *initial_state, const int32_t *cu_seqlens, int num_seqs, int B, int64_t T, int D,
                              int W, unsigned flags, const void *d_out, const void *d_final_state, void *dx, float *d_weight,
                              float *d_bias, void *d_initial_state, void *workspace, size_t workspace_bytes, hipStream_t stream) {
    kda_status st = conv_shape(dtype, D, W, flags);
    if (st != KDA_OK) return st;
    kda::ConvArgs a{};
    bool empty;
    st = batch(a.seqs, cu_seqlens, num_seqs, B, T, &empty);
    if (st != KDA_OK) return st;
    if (x_stride < D) return KDA_ERR_BAD_SHAPE;
    if (d_initial_state && d_initial_state == d_final_state) return KDA_ERR_ALIAS;
    if (misaligned(size_of(dtype), {x, initial_state, d_out, d_final_state, dx, d_initial_state}) ||
        misaligned(4, {weight, bias, cu_seqlens, d_weight, d_bias}))
        return KDA_ERR_BAD_ARGUMENT;
    if (empty) {
        st = fill(d_weight, nullptr, (int64_t)D * W, sizeof(float), stream);
        if (st == KDA_OK) st = fill(d_bias, nullptr, D, sizeof(float), stream);
        return st == KDA_OK ? fill(d_initial_state, d_final_state, (int64_t)a.seqs.N * (W - 1) * D, size_of(dtype), stream) : st;
    }
    if (!conv_fits(a.seqs, D, W)) return KDA_ERR_UNSUPPORTED;
    if (!x || !weight || !d_out || !dx) return KDA_ERR_NULL_POINTER;
    const bool sums = d_weight || d_bias;
    if (sums && !workspace) return KDA_ERR_NULL_POINTER;
    const void *ins[] = {x, weight, bias, initial_state, cu_seqlens, d_out, d_final_state};
    const void *outs[] = {dx, d_weight, d_bias, d_initial_state, workspace};
    if (aliased(ins, outs)) return KDA_ERR_ALIAS;
    if (sums && (misaligned(16, {workspace}) || workspace_bytes < kda_short_conv_bwd_workspace_size(dtype, B, T, D, W))) return KDA_ERR_BAD_ARGUMENT;
    a.x = x;
    a.x_stride = x_stride;
    a.weight = weight;
    a.bias = bias;
    a.s0 = initial_state;
    a.D = D;
    a.W = W;
    a.silu = (flags & KDA_SILU) != 0;
    a.d_out = d_out;
    a.d_sf = d_final_state;
    a.dx = dx;
    a.ds0 = d_initial_state;
    a.part = sums ? static_cast<float *>(workspace) : nullptr;
    const size_t e = size_of(dtype);
    Units w{kda::CONV_BWD_VEC};
    w.rows(x, e, x_stride).rows(initial_state, e, D).rows(d_out, e, D).rows(d_final_state, e, D).rows(dx, e, D).rows(d_initial_state, e, D);
    return done(kda::launch_conv_bwd(a, dtype == KDA_F32, w.ok, d_weight, d_bias, stream));
}

kda_status kda_short_conv_step(const void *x, kda_dtype dtype, const float *weight, const float *bias, void *states, int64_t pool,
                               const int32_t *slots, int slot_cols, const int32_t *start, const int32_t *lengths, int B, int S,
                               int D, int W, unsigned flags, void *out, hipStream_t stream) {
    kda_status st = conv_shape(dtype, D, W, flags);
    if (st != KDA_OK) return st;
    if (B < 0 || S < 0 || pool < 0) return KDA_ERR_BAD_SHAPE;
    if (B == 0 || S == 0) return KDA_OK;
    kda::ConvStepArgs a{};
    st = pool_args(a.slots, slots, slot_cols, start, lengths, pool, B, S);
    if (st != KDA_OK) return st;
    if ((int64_t)B * ((D + 63) / 64 * 64) >= MAX_GRID) return KDA_ERR_UNSUPPORTED;
    if (!x || !weight || !states || !out) return KDA_ERR_NULL_POINTER;
    const void *ins[] = {x, weight, bias, slots, start, lengths}, *outs[] = {states, out};
    if (aliased(ins, outs)) return KDA_ERR_ALIAS;
    if (misaligned(size_of(dtype), {x, states, out}) || misaligned(4, {weight, bias, slots, start, lengths})) return KDA_ERR_BAD_ARGUMENT;
    a.x = x;
    a.weight = weight;
    a.bias = bias;
    a.states = states;
    a.B = B;
    a.S = S;
    a.D = D;
    a.W = W;
    a.silu = (flags & KDA_SILU) != 0;
    a.out = out;
    const size_t e = size_of(dtype);
    Units w{kda::CONV_STEP_VEC};
    w.rows(x, e, D).rows(states, e, D).rows(out, e, D);
    return done(kda::launch_conv_step(a, dtype == KDA_F32, w.ok, stream));
}

size_t kda_glr_kept_size(int B, int64_t T, int H, int K) {
    kda::Seqs s{};
    bool empty;
    if (H <= 0 || K <= 0 || (int64_t)H * K > MAX_CHANNELS || batch(s, nullptr, 0, B, T, &empty) != KDA_OK || empty) return 0;
    return (size_t)glr_kept_rows(s.rows) * H * K * sizeof(float);
}

size_t kda_glr_fwd_workspace_size(int B, int64_t T, int H, int K) {
    kda::GlrArgs a{};
    bool empty;
    if (H <= 0 || K <= 0 || (int64_t)H * K > MAX_CHANNELS || batch(a.seqs, nullptr, 0, B, T, &empty) != KDA_OK || empty) return 0;
    a.C = H * K;
    return glr_fits(a.seqs, a.C) ? some(kda::carve_glr_fwd(a, nullptr)) : 0;
}

size_t kda_glr_bwd_workspace_size(int B, int64_t T, int H, int K, int logits, int kept) {
    kda::GlrArgs a{};
    bool empty;
    if (H <= 0 || K <= 0 || (int64_t)H * K > MAX_CHANNELS || batch(a.seqs, nullptr, 0, B, T, &empty) != KDA_OK || empty) return 0;
    a.C = H * K;
    static const float one = 0.f;
    a.gates.log_scale = logits ? &one : nullptr;
    float *sums;
    return glr_fits(a.seqs, a.C) ? some(kda::carve_glr_bwd(a, nullptr, kept != 0, sums)) : 0;
}

kda_status kda_glr_fwd(const void *x, int64_t x_stride, kda_dtype dtype, const void *gate, int64_t gate_stride, const float *log_scale,
                       const float *bias, float lower_bound, const void *in_gate, int64_t in_stride, unsigned flags,
                       const float *initial_state, float *final_state, const int32_t *cu_seqlens, int num_seqs, int B, int64_t T,
                       int H, int K, void *out, float *kept, void *workspace, size_t workspace_bytes, hipStream_t stream) {
    kda::GlrArgs a{};
    if (!type_ok(dtype)) return KDA_ERR_BAD_DTYPE;
    kda_status st = glr_gates(a.gates, gate, gate_stride, log_scale, bias, lower_bound, in_gate, in_stride, flags, H, K);
    if (st != KDA_OK) return st;
    bool empty;
    st = batch(a.seqs, cu_seqlens, num_seqs, B, T, &empty);
    if (st != KDA_OK) return st;
    const int C = a.C = H * K;
    if (x_stride < C || gate_stride < C || (in_gate && in_stride < C)) return KDA_ERR_BAD_SHAPE;
    if (final_state && final_state == initial_state) return KDA_ERR_ALIAS;
    const size_t e = size_of(dtype), gate_size = log_scale ? e : 4;
    if (misaligned(e, {x, in_gate, out}) || misaligned(gate_size, {gate}) ||
        misaligned(4, {log_scale, bias, initial_state, final_state, cu_seqlens, kept}))
        return KDA_ERR_BAD_ARGUMENT;
    if (empty) return fill(final_state, initial_state, (int64_t)a.seqs.N * C, sizeof(float), stream);
    if (!glr_fits(a.seqs, C)) return KDA_ERR_UNSUPPORTED;
    if (!x || !gate || !out || !workspace) return KDA_ERR_NULL_POINTER;
    const void *ins[] = {x, gate, log_scale, bias, in_gate, initial_state, cu_seqlens}, *outs[] = {out, final_state, kept, workspace};
    if (aliased(ins, outs)) return KDA_ERR_ALIAS;
    a.x = x;
    a.x_stride = x_stride;
    a.s0 = initial_state;
    a.sf = final_state;
    a.out = out;
    a.kept = kept;
    if (misaligned(16, {workspace}) || workspace_bytes < kda_glr_fwd_workspace_size(B, T, H, K)) return KDA_ERR_BAD_ARGUMENT;
    kda::carve_glr_fwd(a, workspace);
    Units w{2};
    w.rows(x, e, x_stride).rows(gate, gate_size, gate_stride).rows(in_gate, e, in_stride).rows(out, e, C);
    w.rows(initial_state, 4, C).rows(final_state, 4, C).rows(kept, 4, C);
    return done(kda::launch_glr_fwd(a, dtype == KDA_F32, w.ok, stream));
}

kda_status kda_glr_bwd(const void *x, int64_t x_stride, kda_dtype dtype, const void *gate, int64_t gate_stride, const float *log_scale,
                       const float *bias, float lower_bound, const void *in_gate, int64_t in_stride, unsigned flags,
                       const float *initial_state, const int32_t *cu_seqlens, int num_seqs, int B, int64_t T, int H, int K,
                       const float *kept, const void *d_out, const float *d_final_state, void *dx, void *d_gate, void *d_in_gate,
                       float *d_log_scale, float *d_bias, float *d_initial_state, void *workspace, size_t workspace_bytes,
                       hipStream_t stream) {
    kda::GlrArgs a{};
    if (!type_ok(dtype)) return KDA_ERR_BAD_DTYPE;
    kda_status st = glr_gates(a.gates, gate, gate_stride, log_scale, bias, lower_bound, in_gate, in_stride, flags, H, K);
    if (st != KDA_OK) return st;
    bool empty;
    st = batch(a.seqs, cu_seqlens, num_seqs, B, T, &empty);
    if (st != KDA_OK) return st;
    const int C = a.C = H * K;
    if (x_stride < C || gate_stride < C || (in_gate && in_stride < C)) return KDA_ERR_BAD_SHAPE;
    if (!log_scale && (d_log_scale || d_bias)) return KDA_ERR_BAD_ARGUMENT;
    if (d_initial_state && d_initial_state == d_final_state) return KDA_ERR_ALIAS;
    const size_t e = size_of(dtype), gate_size = log_scale ? e : 4;
    if (misaligned(e, {x, in_gate, d_out, dx, d_in_gate}) || misaligned(gate_size, {gate, d_gate}) ||
        misaligned(4, {log_scale, bias, initial_state, cu_seqlens, kept, d_final_state, d_log_scale, d_bias, d_initial_state}))
        return KDA_ERR_BAD_ARGUMENT;
    if (empty) {
        st = fill(d_log_scale, nullptr, H, sizeof(float), stream);
        if (st == KDA_OK) st = fill(d_bias, nullptr, C, sizeof(float), stream);
        return st == KDA_OK ? fill(d_initial_state, d_final_state, (int64_t)a.seqs.N * C, sizeof(float), stream) : st;
    }
    if (!glr_fits(a.seqs, C)) return KDA_ERR_UNSUPPORTED;
    if (!x || !gate || !d_out || !dx || !d_gate || (in_gate && !d_in_gate) || !workspace) return KDA_ERR_NULL_POINTER;
    const void *ins[] = {x, gate, log_scale, bias, in_gate, initial_state, cu_seqlens, kept, d_out, d_final_state};
    const void *outs[] = {dx, d_gate, in_gate ? d_in_gate : nullptr, d_log_scale, d_bias, d_initial_state, workspace};
    if (aliased(ins, outs)) return KDA_ERR_ALIAS;
    a.x = x;
    a.x_stride = x_stride;
    a.s0 = initial_state;
    a.kept = const_cast<float *>(kept);
    a.d_out = d_out;
    a.d_sf = d_final_state;
    a.dx = dx;
    a.d_gate = d_gate;
    a.d_in = d_in_gate;
    a.ds0 = d_initial_state;
    float *sums;
    if (misaligned(16, {workspace}) || workspace_bytes < kda_glr_bwd_workspace_size(B, T, H, K, log_scale != nullptr, kept != nullptr)) return KDA_ERR_BAD_ARGUMENT;
    kda::carve_glr_bwd(a, workspace, kept != nullptr, sums);
    if (!d_log_scale && !d_bias) a.part = nullptr;
    Units w{2};
    w.rows(x, e, x_stride).rows(gate, gate_size, gate_stride).rows(in_gate, e, in_stride).rows(d_out, e, C).rows(dx, e, C).rows(d_gate, gate_size, C);
    w.rows(in_gate ? d_in_gate : nullptr, e, C).rows(initial_state, 4, C).rows(kept, 4, C).rows(d_final_state, 4, C).rows(d_initial_state, 4, C);
    return done(kda::launch_glr_bwd(a, dtype == KDA_F32, w.ok, kept != nullptr, sums, d_log_scale, d_bias, stream));
}

kda_status kda_glr_step(const void *x, kda_dtype dtype, const void *gate, const float *log_scale, const float *bias, float lower_bound,
                        const void *in_gate, unsigned flags, float *states, int64_t pool, const int32_t *slots, int slot_cols,
                        const int32_t *start, const int32_t *lengths, int B, int S, int H, int K, void *out, hipStream_t stream) {
    kda::GlrStepArgs a{};
    if (!type_ok(dtype)) return KDA_ERR_BAD_DTYPE;
    kda_status st = glr_gates(a.gates, gate, 0, log_scale, bias, lower_bound, in_gate, 0, flags, H, K);
    if (st != KDA_OK) return st;
    if (B < 0 || S < 0 || pool < 0) return KDA_ERR_BAD_SHAPE;
    if (B == 0 || S == 0) return KDA_OK;
    st = pool_args(a.slots, slots, slot_cols, start, lengths, pool, B, S);
    if (st != KDA_OK) return st;
    const int C = a.C = H * K;
    if ((int64_t)B * ((C + 63) / 64 * 64) >= MAX_GRID) return KDA_ERR_UNSUPPORTED;
    if (!x || !gate || !states || !out) return KDA_ERR_NULL_POINTER;
    const void *ins[] = {x, gate, log_scale, bias, in_gate, slots, start, lengths}, *outs[] = {states, out};
    if (aliased(ins, outs)) return KDA_ERR_ALIAS;
    const size_t e = size_of(dtype), gate_size = log_scale ? e : 4;
    if (misaligned(e, {x, in_gate, out}) || misaligned(gate_size, {gate}) || misaligned(4, {log_scale, bias, states, slots, start, lengths}))
        return KDA_ERR_BAD_ARGUMENT;
    a.x = x;
    a.states = states;
    a.B = B;
    a.S = S;
    a.out = out;
    Units w{2};
    w.rows(x, e, C).rows(gate, gate_size, C).rows(in_gate, e, C).rows(states, 4, C).rows(out, e, C);
    return done(kda::launch_glr_step(a, dtype == KDA_F32, w.ok, stream));
}

kda_status kda_block_norm_fwd(const void *y, const void *gate, int64_t gate_stride, int64_t gate_head_stride, kda_dtype dtype, const void *residual, kda_dtype h_dtype,
                              const float *weight_after, const float *weight_before, int64_t tokens, int heads, int D, float scale,
                              float eps, unsigned flags, void *h, void *n, hipStream_t stream) {
    const kda_status st = norm_shape(dtype, h_dtype, tokens, heads, D, eps, flags);
    if (st != KDA_OK) return st;
    const bool before = (flags & KDA_NORM_BEFORE) != 0, after = (flags & KDA_NORM_AFTER) != 0;
    if ((weight_after && !after) || (weight_before && !before)) return KDA_ERR_BAD_ARGUMENT;
    if (gate && (gate_stride < D || (heads > 1 && gate_head_stride < D))) return KDA_ERR_BAD_SHAPE;
    const size_t e = size_of(dtype), he = size_of(h_dtype);
    if (misaligned(e, {y, gate, before ? n : nullptr}) || misaligned(he, {residual, h}) || misaligned(4, {weight_after, weight_before})) return KDA_ERR_BAD_ARGUMENT;
    if (tokens == 0) return KDA_OK;
    if (!y || !h || (before && !n)) return KDA_ERR_NULL_POINTER;
    const void *ins[] = {y, gate, residual, weight_after, weight_before}, *outs[] = {h, before ? n : nullptr};
    if (aliased(ins, outs)) return KDA_ERR_ALIAS;
    kda::NormArgs a{};
    a.y = y;
    a.gate = gate;
    a.gate_stride = gate_stride;
    a.gate_head = heads > 1 ? gate_head_stride : 0;
    a.residual = residual;
    a.wa = weight_after;
    a.wb = weight_before;
    a.rows = tokens * heads;
    a.heads = heads;
    a.D = D;
    a.scale = scale;
    a.eps = eps;
    a.after = after;
    a.before = before;
    a.silu = (flags & KDA_SILU) != 0;
    a.h = h;
    a.n = n;
    auto fits = [&](int unit) {
        Units w{unit};
        w.rows(y, e, D).rows(residual, he, D).rows(h, he, D).rows(before ? n : nullptr, e, D).rows(gate, e, gate_stride).rows(gate, e, a.gate_head);
        return w.ok;
    };
    const int vec = fits(16 / (int)e) ? 16 / (int)e : fits(2) ? 2 : 1;
    return done(kda::launch_norm_fwd(a, dtype == KDA_F32, h_dtype == KDA_F32, vec, stream));
}

size_t kda_block_norm_bwd_workspace_size(int64_t tokens, int heads, int D) {
    if (tokens <= 0 || heads <= 0 || D <= 0 || D > KDA_NORM_MAX_D || tokens > (int64_t)INT32_MAX / heads) return 0;
    return (size_t)kda::norm_groups(tokens * heads, D) * 2 * D * sizeof(float);
}

kda_status kda_block_norm_bwd(const void *y, const void *gate, int64_t gate_stride, int64_t gate_head_stride, kda_dtype dtype, const void *h, kda_dtype h_dtype,
                              const float *weight_after, const float *weight_before, int64_t tokens, int heads, int D, float scale,
                              float eps, unsigned flags, const void *d_h, const void *d_n, void *dy, void *d_gate, void *d_residual,
                              float *d_weight_after, float *d_weight_before, void *workspace, size_t workspace_bytes, hipStream_t stream) {
    kda_status st = norm_shape(dtype, h_dtype, tokens, heads, D, eps, flags);
    if (st != KDA_OK) return st;
    const bool before = (flags & KDA_NORM_BEFORE) != 0, after = (flags & KDA_NORM_AFTER) != 0;
    if ((!after && (weight_after || d_weight_after)) || (!before && (weight_before || d_weight_before))) return KDA_ERR_BAD_ARGUMENT;
    if (gate && (gate_stride < D || (heads > 1 && gate_head_stride < D))) return KDA_ERR_BAD_SHAPE;
    const size_t e = size_of(dtype), he = size_of(h_dtype);
    if (misaligned(e, {y, gate, dy, gate ? d_gate : nullptr, before ? d_n : nullptr}) || misaligned(he, {d_h, before ? h : nullptr, before ? d_residual : nullptr}) ||
        misaligned(4, {weight_after, weight_before, d_weight_after, d_weight_before}))
        return KDA_ERR_BAD_ARGUMENT;
    if (tokens == 0) {
        st = fill(d_weight_after, nullptr, D, sizeof(float), stream);
        return st == KDA_OK ? fill(d_weight_before, nullptr, D, sizeof(float), stream) : st;
    }
    const bool sums = d_weight_after || d_weight_before;
    if (!y || !dy || (gate && !d_gate) || (before ? !h || !d_n : !d_h) || (sums && !workspace)) return KDA_ERR_NULL_POINTER;
    const void *ins[] = {y, gate, before ? h : nullptr, weight_after, weight_before, d_h, before ? d_n : nullptr};
    const void *outs[] = {dy, gate ? d_gate : nullptr, before ? d_residual : nullptr, d_weight_after, d_weight_before, workspace};
    if (aliased(ins, outs)) return KDA_ERR_ALIAS;
    if (sums && (misaligned(16, {workspace}) || workspace_bytes < kda_block_norm_bwd_workspace_size(tokens, heads, D))) return KDA_ERR_BAD_ARGUMENT;
    kda::NormArgs a{};
    a.y = y;
    a.gate = gate;
    a.gate_stride = gate_stride;
    a.gate_head = heads > 1 ? gate_head_stride : 0;
    a.wa = weight_after;
    a.wb = weight_before;
    a.rows = tokens * heads;
    a.heads = heads;
    a.D = D;
    a.scale = scale;
    a.eps = eps;
    a.after = after;
    a.before = before;
    a.silu = (flags & KDA_SILU) != 0;
    a.d_h = d_h;
    a.d_n = d_n;
    a.h_in = h;
    a.dy = dy;
    a.d_gate = d_gate;
    a.d_res = d_residual;
    a.part = sums ? static_cast<float *>(workspace) : nullptr;
    a.groups = kda::norm_groups(a.rows, D);
    auto fits = [&](int unit) {
        Units w{unit};
        w.rows(y, e, D).rows(d_h, he, D).rows(dy, e, D).rows(gate, e, gate_stride).rows(gate, e, a.gate_head).rows(gate ? d_gate : nullptr, e, D);
        w.rows(before ? h : nullptr, he, D).rows(before ? d_n : nullptr, e, D).rows(before ? d_residual : nullptr, he, D);
        return w.ok;
    };
    const int vec = fits(16 / (int)e) ? 16 / (int)e : fits(2) ? 2 : 1;
    return done(kda::launch_norm_bwd(a, dtype == KDA_F32, h_dtype == KDA_F32, vec, d_weight_after, d_weight_before, stream));
}

}  // extern "C"
