// Launch interface of the decode kernels over a pool of states and of the verification of
// drafted tokens.
#pragma once

#include "kda_device.h"
#include "kda_internal.h"

namespace kda {

struct GdrStepArgs {
    const void *q, *k, *v;      // [B, S, HK, K], [B, S, HK, K], [B, S, HV, V]
    const float *g, *beta;      // [B, S, HV] or [B, S, HV, K] with channels; [B, S, HV]
    float *states;              // [pool, HV, K, V]
    const int32_t *slots;       // [B, slot_cols] or null (slot b)
    const int32_t *start;       // [B]: column of slots whose state a request starts from, or null (0)
    const int32_t *lengths;     // [B] tokens of a request, or null (S)
    void *out;                  // [B, S, HV, V]
    int64_t pool;
    int B, S, HK, HV, group, V, slot_cols;
    int channels, out_bf16;
    float scale;
};
hipError_t launch_gdr_step(const GdrStepArgs &a, bool fp32, int K, hipStream_t stream);

constexpr int DRAFT_TILE = 1024;  // tokens of the vocabulary whose weights are summed together
struct DraftVerifyArgs {
    const float *target;        // [B, D + 1, vocab]
    const float *draft;         // [B, D, vocab] or null
    const int32_t *x;           // [B, D]
    const float *u;             // [B, D + 1]
    const int32_t *lengths;     // [B] or null (D)
    int32_t *tokens;            // [B, D + 1]
    int32_t *accepted;          // [B]
    unsigned long long *sums;   // [B][tiles][2]
    int B, D, vocab, tiles;
};
hipError_t launch_draft_verify(const DraftVerifyArgs &a, hipStream_t stream);

}  // namespace kda
