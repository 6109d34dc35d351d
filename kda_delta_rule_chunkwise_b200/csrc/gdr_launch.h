// Internal launch interface of the gated-delta-rule kernels.
#pragma once

#include "kda_launch.h"

namespace kda {

struct GdrArgs {
    const void *q, *k, *v, *g, *beta;
    const float *state_in;
    const int32_t *cu_seqlens;   // device, N + 1 entries, or nullptr
    int64_t T;                   // rows per batch entry (packed rows when cu_seqlens)
    int N, Hk, H, dk, dv;
    void *o;
    float *state_out;
    uint32_t *err;
    uint32_t epoch;
};

// bf16, tensor cores
cudaError_t launch_gdr_prefill(const GdrArgs &a, cudaStream_t st);

// Token by token in fp32 arithmetic (gdr_token.cu): the decode step for either type, and the
// fp32 prefill.  State entries are slots[n] of P where given.
struct GdrTokenArgs {
    const void *q, *k, *v, *g, *beta;
    const float *state_in;       // nullptr: zeros
    float *state_out;            // nullptr: not written; may equal state_in
    const int32_t *cu_seqlens;   // nullptr: sequence n has rows n T .. n T + T - 1
    const int32_t *slots, *lens; // nullptr: entry n; all T tokens
    int64_t T;
    int N, P, Hk, H, dk, dv;
    void *o;
    uint32_t *err;
};
cudaError_t launch_gdr_token(const GdrTokenArgs &a, bool bf16, cudaStream_t st);

}  // namespace kda
