// Debug input scan of the gated-delta-rule calls (KDA_DEBUG_CHECKS=1): reports inputs outside their
// contract (kda.h) as ERR_INPUT_RANGE in the device error word.  It changes no output.
//
// One warp per (32-token chunk, key head), a token per lane.  Speed is of no concern here.
#include "gdr_common.cuh"
#include "gdr_launch.h"

namespace kda {
namespace gdr {

template <typename Tin>
__global__ void __launch_bounds__(128) gdr_scan_kernel(GdrScanArgs a) {
    const int lane = threadIdx.x & 31;
    const int hk = blockIdx.x % a.Hk, n = blockIdx.x / a.Hk, group = a.H / a.Hk;
    Span span = sequence_span(a.cu_seqlens, n, a.T);
    if (a.lens) span.len = min(max(a.lens[n], 0), span.len);
    const int chunks = (span.len + kChunk - 1) / kChunk;
    const Tin *k = (const Tin *)a.k, *g = (const Tin *)a.g, *beta = (const Tin *)a.beta;
    bool bad = false;
    for (int c = blockIdx.y * 4 + (threadIdx.x >> 5); c < chunks; c += gridDim.y * 4) {
        const bool live = c * kChunk + lane < span.len;
        const int64_t row = span.row + (int64_t)c * kChunk + lane;
        float kk = 0.f;
        if (live && a.chunked)
            for (int i = 0; i < a.dk; ++i) {
                const float x = to_f32(k[(row * a.Hk + hk) * a.dk + i]);
                kk = fmaf(x, x, kk);
            }
        float most = kk;
#pragma unroll
        for (int m = 16; m > 0; m >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, m));
        for (int h = hk * group; live && h < (hk + 1) * group; ++h) {
            const float b = to_f32(beta[row * a.H + h]), step = b * kk;
            bad |= !(to_f32(g[row * a.H + h]) <= 0.f);
            if (a.chunked) bad |= !(step >= 0.f && step <= kMaxStep) || !(b * sqrtf(kk) * sqrtf(most) < kMaxCross);
            if (a.backward) bad |= !(b <= kMaxBeta);
        }
    }
    if (bad) atomicOr(a.err, ERR_INPUT_RANGE);
}

}  // namespace gdr

cudaError_t launch_gdr_scan(const GdrScanArgs &a, bool bf16, cudaStream_t st) {
    const int64_t quads = (a.T + 4 * gdr::kChunk - 1) / (4 * gdr::kChunk);
    const dim3 grid((unsigned)((int64_t)a.N * a.Hk), (unsigned)(quads < 1 ? 1 : quads < 64 ? quads : 64));
    if (bf16) gdr::gdr_scan_kernel<__nv_bfloat16><<<grid, 128, 0, st>>>(a);
    else gdr::gdr_scan_kernel<float><<<grid, 128, 0, st>>>(a);
    return cudaGetLastError();
}

}  // namespace kda
