// Internal interface of the fp32 backward of the gated delta rule.
#pragma once

#include "gdr_launch.h"

namespace kda {
namespace gdr {

struct TokenBackwardArgs {
    const float *q, *k, *v, *g, *beta, *dout;
    const float *state_in, *dstate_out;
    const int32_t *cu;
    int64_t T;
    int N, Hk, H, dv;
    float *dq, *dk, *dv_out, *dg, *dbeta, *dstate_in;
    // workspace: states before 32-token blocks, the CTAs' token states, the slices' shares
    float *blocks = nullptr, *scratch = nullptr;
    float *part_q = nullptr, *part_k = nullptr;   // [rows, H, slices, dk]
    float *part_g = nullptr, *part_b = nullptr;   // [rows, H, slices]
};
size_t token_backward_workspace_bytes(int64_t rows, int N, int H, int dk, int dv);
cudaError_t launch_token_backward(const GdrArgs &p, const GdrGrads &g, int64_t rows, void *workspace,
                                  cudaStream_t st);

}  // namespace gdr
}  // namespace kda
