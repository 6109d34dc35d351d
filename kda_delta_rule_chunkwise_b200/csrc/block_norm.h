// Internal launch interface of the block norm.
#pragma once

#include "kda_launch.h"

namespace kda {

struct BlockNormArgs {
    const void *x, *y, *gate, *w_post, *w_pre;   // gate may be nullptr
    int64_t rows;
    int width;
    float scale, eps;
    void *x_new, *h;                             // forward
    const void *dx_new, *dh;                     // backward; either may be nullptr (zeros)
    void *dx, *dy, *dgate;
    float *dw_post, *dw_pre;
    float *part;                                 // [block_norm_parts][2][width]
    uint32_t *err;
    uint32_t epoch;
    int stages = 0;                              // of the ring (set by the launcher)
};
constexpr int kBlockNormStages = 8;
constexpr int kBlockNormMaxWidth = 16384;
size_t block_norm_parts(int64_t rows, int width);
cudaError_t launch_block_norm(const BlockNormArgs &a, bool x_bf16, bool bf16, bool backward,
                              cudaStream_t st);

}  // namespace kda
