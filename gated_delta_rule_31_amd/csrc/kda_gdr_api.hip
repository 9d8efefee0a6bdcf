// kda_gdr_api.hip -- the C entry points of the gated delta rule with one decay per value head
// and of decoding with drafted tokens: argument validation, the empty cases, workspaces.
#include "../../include/kda.h"
#include "kda_gdr.h"
#include "kda_gdr_step.h"

namespace {

kda_status done(hipError_t e) {
    if (e == hipSuccess) return KDA_OK;
    kda::record_hip_error(e);
    return e == hipErrorNotSupported ? KDA_ERR_UNSUPPORTED : KDA_ERR_HIP;
}

bool width_ok(int d) { return d == 16 || d == 32 || d == 64 || d == 128; }
bool type_ok(kda_dtype t) { return t == KDA_F32 || t == KDA_BF16; }
bool aligned(const void *p) { return (uintptr_t)p % 16 == 0; }

constexpr int64_t MAX_UNITS = 1 << 22;  // (chunk slot, value head) or (sequence, value head, column tile)
constexpr int64_t MAX_TOKENS = MAX_UNITS * kda::GDR_C;  // more of them in a row are more slots than that: their count stays in 64 bits

int64_t chunk_slots(int B, int64_t T, int num_seqs, bool varlen) {
    const int64_t C = kda::GDR_C;
    return varlen ? T / C + num_seqs : B * ((T + C - 1) / C);
}

// The pieces of a workspace one behind the other, each on a 256-byte border; with no base only
// the size is counted.
struct Carver {
    char *base;
    size_t used = 0;
    template <typename T>
    void take(T *&p, int64_t n) {
        p = base ? reinterpret_cast<T *>(base + used) : nullptr;
        used += ((size_t)n * sizeof(T) + 255) / 256 * 256;
    }
};

size_t carve_fwd(kda::GdrArgs &a, void *base, bool fp32) {
    // the sizes that callers were told before M and P were kept without their upper fragments: the
    // last 4 KB of a unit, and with float32 inputs the last sixth, are not used
    const int C = kda::GDR_C;
    const int64_t units = a.slots * a.HV;
    Carver w{static_cast<char *>(base)};
    w.take(a.M, units * (fp32 ? 6 * C * C : kda::GDR_UNIT));
    w.take(a.dec, units * 4 * C);
    return w.used;
}

size_t carve_bwd(kda::GdrArgs &a, void *base, bool fp32, int K) {
    const int C = kda::GDR_C, parts = kda::GDR_PARTS, turned_parts = fp32 ? 3 : 0;
    const int64_t units = a.slots * a.HV;
    Carver w{static_cast<char *>(base)};
    w.take(a.M, units * parts * C * C);
    w.take(a.Mt, units * parts * C * C);
    w.take(a.P, units * parts * C * C);
    w.take(a.Kt, a.slots * a.HK * turned_parts * K * C);
    w.take(a.Qt, a.slots * a.HK * turned_parts * K * C);
    w.take(a.dec, units * 4 * C);
    w.take(a.G, units * C);
    w.take(a.h, units * K * a.V);
    w.take(a.dh, units * K * a.V);
    w.take(a.delta, units * C * a.V);
    w.take(a.dY, units * C * a.V);
    return w.used;
}

bool heads_ok(int HK, int HV) { return HK > 0 && HV > 0 && HV % HK == 0; }

// What the prefill and its backward pass share.  KDA_OK with *empty set: nothing to scan.
kda_status chunk_args(kda::GdrArgs &a, const void *q, const void *k, const void *v, kda_dtype in_dtype, const float *g,
                      const float *beta, const float *s0, const int32_t *cu, int num_seqs, int B, int64_t T, int HK,
                      int HV, int K, int V, float scale, bool *empty) {
    if (B < 0 || T < 0 || K <= 0 || V <= 0 || HK <= 0 || HV <= 0) return KDA_ERR_BAD_SHAPE;
    if (!heads_ok(HK, HV)) return KDA_ERR_BAD_SHAPE;
    if (!type_ok(in_dtype)) return KDA_ERR_BAD_DTYPE;
    if (!width_ok(K) || !width_ok(V)) return KDA_ERR_UNSUPPORTED;
    if (cu && (B != 1 || num_seqs < 0 || (num_seqs == 0 && T > 0))) return KDA_ERR_BAD_ARGUMENT;
    const int64_t N = cu ? num_seqs : B;
    a = kda::GdrArgs{};
    a.q = q;
    a.k = k;
    a.v = v;
    a.g = g;
    a.beta = beta;
    a.s0 = s0;
    a.cu = cu;
    a.T = T;
    a.N = (int)N;
    a.HK = HK;
    a.HV = HV;
    a.group = HV / HK;
    a.V = V;
    a.scale = scale;
    *empty = B == 0 || T == 0 || N == 0;
    if (*empty) return KDA_OK;
    if (T > MAX_TOKENS) return KDA_ERR_UNSUPPORTED;
    a.slots = chunk_slots(B, T, num_seqs, cu != nullptr);
    a.chunks = (int)((T + kda::GDR_C - 1) / kda::GDR_C);
    // a chunk's rows are addressed by 32-bit offsets
    if (HK > 65535 || HV > 65535) return KDA_ERR_UNSUPPORTED;
    // a grid has fewer than 2^32 threads
    if (a.slots > MAX_UNITS / HV || N > MAX_UNITS / HV / (V / 16)) return KDA_ERR_UNSUPPORTED;
    if (!q || !k || !v || !g || !beta) return KDA_ERR_NULL_POINTER;
    return KDA_OK;
}

// What a workspace's size depends on; false if the shape is not supported.
bool size_args(kda::GdrArgs &a, kda_dtype in_dtype, int B, int64_t T, int num_seqs, int varlen, int HK, int HV, int K, int V) {
    a = kda::GdrArgs{};
    if (B < 0 || T < 0 || T > MAX_TOKENS || num_seqs < 0 || !heads_ok(HK, HV) || !type_ok(in_dtype) || !width_ok(K) || !width_ok(V)) return false;
    a.HK = HK;
    a.HV = HV;
    a.V = V;
    a.slots = T == 0 ? 0 : chunk_slots(B, T, num_seqs, varlen != 0);
    return a.slots <= MAX_UNITS / HV;
}

}  // namespace

extern "C" {

size_t kda_gdr_chunk_fwd_workspace_size(kda_dtype in_dtype, int B, int64_t T, int num_seqs, int varlen, int HK, int HV,
                                        int K, int V) {
    kda::GdrArgs a;
    return size_args(a, in_dtype, B, T, num_seqs, varlen, HK, HV, K, V) ? carve_fwd(a, nullptr, in_dtype == KDA_F32) : 0;
}

size_t kda_gdr_chunk_bwd_workspace_size(kda_dtype in_dtype, int B, int64_t T, int num_seqs, int varlen, int HK, int HV,
                                        int K, int V) {
    kda::GdrArgs a;
    return size_args(a, in_dtype, B, T, num_seqs, varlen, HK, HV, K, V) ? carve_bwd(a, nullptr, in_dtype == KDA_F32, K) : 0;
}

kda_status kda_gdr_chunk_fwd(const void *q, const void *k, const void *v, kda_dtype in_dtype, const float *g,
                             const float *beta, const float *initial_state, float *final_state,
                             const int32_t *cu_seqlens, int num_seqs, int B, int64_t T, int HK, int HV, int K, int V,
                             float scale, void *out, kda_dtype out_dtype, void *workspace, size_t workspace_bytes,
                             hipStream_t stream) {
    kda::GdrArgs a;
    bool empty;
    const kda_status st = chunk_args(a, q, k, v, in_dtype, g, beta, initial_state, cu_seqlens, num_seqs, B, T, HK, HV, K, V, scale, &empty);
    if (st != KDA_OK) return st;
    if (!type_ok(out_dtype)) return KDA_ERR_BAD_DTYPE;
    if (empty) {
        if (final_state && a.N > 0 && initial_state != final_state)
            return done(kda::launch_fill_copy(final_state, initial_state, (int64_t)a.N * HV * K * V, stream));
        return KDA_OK;
    }
    if (!out || !workspace) return KDA_ERR_NULL_POINTER;
    const void *ins[] = {q, k, v, g, beta, initial_state, cu_seqlens};
    for (const void *p : ins) {
        if (!p) continue;
        if (p == out || p == workspace) return KDA_ERR_ALIAS;
        if (p == (const void *)final_state && p != (const void *)initial_state) return KDA_ERR_ALIAS;
    }
    if (out == (void *)final_state || out == workspace || workspace == (void *)final_state) return KDA_ERR_ALIAS;
    const void *vec[] = {q, k, v, initial_state, final_state, out, workspace};
    for (const void *p : vec)
        if (!aligned(p)) return KDA_ERR_BAD_ARGUMENT;
    if (workspace_bytes < carve_fwd(a, workspace, in_dtype == KDA_F32)) return KDA_ERR_BAD_ARGUMENT;
    a.sf = final_state;
    a.out = out;
    a.out_bf16 = out_dtype == KDA_BF16;
    const hipError_t e = kda::launch_gdr_prep(a, in_dtype == KDA_F32, K, false, stream);
    return done(e != hipSuccess ? e : kda::launch_gdr_fwd_chain(a, in_dtype == KDA_F32, K, stream));
}

kda_status kda_gdr_chunk_bwd(const void *q, const void *k, const void *v, kda_dtype in_dtype, const float *g,
                             const float *beta, const float *initial_state, const int32_t *cu_seqlens, int num_seqs,
                             int B, int64_t T, int HK, int HV, int K, int V, float scale, const void *d_out,
                             kda_dtype dout_dtype, const float *d_final_state, void *dq, void *dk, void *dv,
                             kda_dtype grad_dtype, float *dg, float *dbeta, float *d_initial_state, void *workspace,
                             size_t workspace_bytes, hipStream_t stream) {
    kda::GdrArgs a;
    bool empty;
    const kda_status st = chunk_args(a, q, k, v, in_dtype, g, beta, initial_state, cu_seqlens, num_seqs, B, T, HK, HV, K, V, scale, &empty);
    if (st != KDA_OK) return st;
    if (!type_ok(dout_dtype) || !type_ok(grad_dtype)) return KDA_ERR_BAD_DTYPE;
    if (empty) {
        if (d_initial_state && a.N > 0 && (const float *)d_initial_state != d_final_state)
            return done(kda::launch_fill_copy(d_initial_state, d_final_state, (int64_t)a.N * HV * K * V, stream));
        return KDA_OK;
    }
    if (!d_out || !dq || !dk || !dv || !dg || !dbeta || !workspace) return KDA_ERR_NULL_POINTER;
    const void *ins[] = {q, k, v, g, beta, initial_state, cu_seqlens, d_out, d_final_state};
    const void *outs[] = {dq, dk, dv, dg, dbeta, d_initial_state, workspace};
    for (int i = 0; i < 7; ++i) {
        if (!outs[i]) continue;
        for (const void *p : ins)
            if (p == outs[i]) return KDA_ERR_ALIAS;
        for (int j = 0; j < i; ++j)
            if (outs[j] == outs[i]) return KDA_ERR_ALIAS;
    }
    const void *vec[] = {q, k, v, initial_state, d_out, d_final_state, dq, dk, dv, d_initial_state, workspace};
    for (const void *p : vec)
        if (!aligned(p)) return KDA_ERR_BAD_ARGUMENT;
    if (workspace_bytes < carve_bwd(a, workspace, in_dtype == KDA_F32, K)) return KDA_ERR_BAD_ARGUMENT;
    a.d_out = d_out;
    a.dout_bf16 = dout_dtype == KDA_BF16;
    a.d_sf = d_final_state;
    a.dq = dq;
    a.dk = dk;
    a.dv = dv;
    a.grad_bf16 = grad_dtype == KDA_BF16;
    a.dg = dg;
    a.dbeta = dbeta;
    a.ds0 = d_initial_state;
    return done(kda::launch_gdr_bwd(a, in_dtype == KDA_F32, K, stream));
}

kda_status kda_gdr_recurrent_step(const void *q, const void *k, const void *v, kda_dtype in_dtype, const float *g,
                                  int g_channels, const float *beta, float *states, int64_t pool, const int32_t *slots,
                                  int slot_cols, const int32_t *start, const int32_t *lengths, int B, int S, int HK,
                                  int HV, int K, int V, float scale, void *out, kda_dtype out_dtype,
                                  hipStream_t stream) {
    if (B < 0 || S < 0 || pool < 0 || K <= 0 || V <= 0 || !heads_ok(HK, HV)) return KDA_ERR_BAD_SHAPE;
    if (!type_ok(in_dtype) || !type_ok(out_dtype)) return KDA_ERR_BAD_DTYPE;
    if (!width_ok(K) || !width_ok(V)) return KDA_ERR_UNSUPPORTED;
    if (B == 0 || S == 0) return KDA_OK;
    if (slot_cols != 1 && slot_cols != S) return KDA_ERR_BAD_SHAPE;
    if (!slots && (slot_cols != 1 || start || pool < B)) return KDA_ERR_BAD_ARGUMENT;
    if (start && slot_cols != S) return KDA_ERR_BAD_ARGUMENT;
    if (B > (1 << 24) / HV / (V / 16)) return KDA_ERR_UNSUPPORTED;  // a grid has fewer than 2^32 threads
    if (!q || !k || !v || !g || !beta || !states || !out) return KDA_ERR_NULL_POINTER;
    const void *ins[] = {q, k, v, g, beta, slots, start, lengths};
    for (const void *p : ins)
        if (p && (p == out || p == (const void *)states)) return KDA_ERR_ALIAS;
    if (out == (void *)states) return KDA_ERR_ALIAS;
    const void *vec[] = {q, k, v, g_channels ? g : nullptr, states, out};
    for (const void *p : vec)
        if (!aligned(p)) return KDA_ERR_BAD_ARGUMENT;
    kda::GdrStepArgs a;
    a.q = q;
    a.k = k;
    a.v = v;
    a.g = g;
    a.beta = beta;
    a.states = states;
    a.slots = slots;
    a.start = start;
    a.lengths = lengths;
    a.out = out;
    a.pool = pool;
    a.B = B;
    a.S = S;
    a.HK = HK;
    a.HV = HV;
    a.group = HV / HK;
    a.V = V;
    a.slot_cols = slot_cols;
    a.channels = g_channels != 0;
    a.out_bf16 = out_dtype == KDA_BF16;
    a.scale = scale;
    return done(kda::launch_gdr_step(a, in_dtype == KDA_F32, K, stream));
}

size_t kda_draft_verify_workspace_size(int B, int vocab) {
    if (B < 0 || vocab < 1 || vocab > (1 << 19)) return 0;
    return (size_t)B * ((vocab + kda::DRAFT_TILE - 1) / kda::DRAFT_TILE) * 16;
}

kda_status kda_draft_verify(const float *target_probs, const int32_t *draft_tokens, const float *draft_probs,
                            const float *uniforms, const int32_t *lengths, int B, int D, int vocab, int32_t *tokens,
                            int32_t *accepted, void *workspace, size_t workspace_bytes, hipStream_t stream) {
    if (B < 0 || D < 0 || vocab < 1) return KDA_ERR_BAD_SHAPE;
    // the whole of a row's weights has to fit 64 bits; the second kernel's threads sum the tiles
    if (vocab > (1 << 19) || D == INT32_MAX) return KDA_ERR_UNSUPPORTED;
    if (B == 0) return KDA_OK;
    if (B > (1 << 24) / ((vocab + kda::DRAFT_TILE - 1) / kda::DRAFT_TILE)) return KDA_ERR_UNSUPPORTED;  // likewise
    if (!target_probs || (D && !draft_tokens) || !uniforms || !tokens || !accepted || !workspace) return KDA_ERR_NULL_POINTER;
    const void *ins[] = {target_probs, draft_tokens, draft_probs, uniforms, lengths}, *outs[] = {tokens, accepted, workspace};
    for (int i = 0; i < 3; ++i) {
        for (const void *p : ins)
            if (p && p == outs[i]) return KDA_ERR_ALIAS;
        for (int j = 0; j < i; ++j)
            if (outs[j] == outs[i]) return KDA_ERR_ALIAS;
    }
    if (workspace_bytes < kda_draft_verify_workspace_size(B, vocab) || (uintptr_t)workspace % 8 != 0) return KDA_ERR_BAD_ARGUMENT;
    kda::DraftVerifyArgs a;
    a.target = target_probs;
    a.draft = draft_probs;
    a.x = draft_tokens;
    a.u = uniforms;
    a.lengths = lengths;
    a.tokens = tokens;
    a.accepted = accepted;
    a.sums = static_cast<unsigned long long *>(workspace);
    a.B = B;
    a.D = D;
    a.vocab = vocab;
    a.tiles = (vocab + kda::DRAFT_TILE - 1) / kda::DRAFT_TILE;
    return done(kda::launch_draft_verify(a, stream));
}

}  // extern "C"
