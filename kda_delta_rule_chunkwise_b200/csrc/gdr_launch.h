// Internal launch interface of the gated-delta-rule kernels.
#pragma once

#include "kda_launch.h"

namespace kda {

struct GdrArgs {
    const void *q, *k, *v, *g, *beta;
    const float *state_in;
    const int32_t *cu_seqlens;   // device, N + 1 entries, or nullptr
    int64_t T;                   // rows per batch entry (packed rows when cu_seqlens)
    int64_t rows;                // of all batch entries
    int N, Hk, H, dk, dv;
    void *o;
    float *state_out;
    uint32_t *err;
    uint32_t epoch;
};

// bf16, tensor cores.  Images of the chunks (gdr_prep.cu) in the caller's workspace, 256-byte
// aligned: keys and queries, the forward's inverses, and the adjoint's for a backward.
struct GdrImages {
    unsigned char *keys, *forward, *adjoint;
    int32_t *order;   // packed sequences from the longest to the shortest, or nullptr (N = 1, dense)
};
size_t gdr_image_bytes(int64_t rows, int N, int Hk, int H, int dk, bool adjoint);
GdrImages gdr_images(void *space, const GdrArgs &a, bool adjoint);
cudaError_t launch_gdr_prep(const GdrArgs &a, const GdrImages &m, cudaStream_t st);
// workspace: gdr_image_bytes(.., false)
cudaError_t launch_gdr_prefill(const GdrArgs &a, void *workspace, cudaStream_t st);

// Backward, bf16.  The images, then three kernels: the forward's chain again, keeping N and the state before
// each 64-token block; the adjoint chain, keeping E and the adjoint state behind each block;
// the gradients of each block (gdr_backward.cu).
struct GdrBackwardSpace {
    float *n, *e;                  // [rows, H, dv]
    unsigned char *s_blocks, *z_blocks;   // [rows / 64 + N + 1, H], fp16 (store_block)
    float *s_scales, *z_scales;           // [rows / 64 + N + 1, H, dv / 16, 2]
    int32_t *owners;               // [rows / 64 + N + 1]: a block's sequence, or -1
};
struct GdrGrads {
    const void *dout;
    const float *dstate_out;       // or nullptr
    void *dq, *dk, *dv, *dg, *dbeta;
    float *dstate_in;              // or nullptr
};
size_t gdr_backward_workspace_bytes(int64_t rows, int N, int Hk, int H, int dk, int dv, bool bf16);
cudaError_t launch_gdr_recompute(const GdrArgs &a, const GdrImages &m, const GdrBackwardSpace &w,
                                 cudaStream_t st);
// workspace: gdr_backward_workspace_bytes bytes, 256-byte aligned
cudaError_t launch_gdr_backward(const GdrArgs &a, const GdrGrads &g, int64_t rows, bool bf16,
                                void *workspace, cudaStream_t st);

// The debug input scan (gdr_debug.cu): g above 0 or NaN; `chunked`: the limits of the bf16 calls on the
// chunks as well, `backward`: and on beta.
struct GdrScanArgs {
    const void *k, *g, *beta;
    const int32_t *cu_seqlens, *lens;   // either may be nullptr
    int64_t T;
    int N, Hk, H, dk;
    bool chunked, backward;
    uint32_t *err;
};
cudaError_t launch_gdr_scan(const GdrScanArgs &a, bool bf16, cudaStream_t st);

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
cudaError_t launch_gdr_token(const GdrTokenArgs &a, bool bf16, cudaStream_t st);   // no cu_seqlens
cudaError_t launch_gdr_token_prefill(const GdrTokenArgs &a, cudaStream_t st);      // fp32; no slots, lens

}  // namespace kda
