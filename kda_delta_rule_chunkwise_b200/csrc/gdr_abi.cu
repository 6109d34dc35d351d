// C ABI of the gated delta rule and the block norm (declared in include/kda.h): argument
// checks, then dispatch.
#include "block_norm.h"
#include "gdr_launch.h"

#include "kda.h"

#include <climits>
#include <cmath>

namespace {

bool head_dim(int d) { return d == 64 || d == 128; }
bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
kda_status from_cuda(cudaError_t e) { return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA; }

// The debug input scan ahead of a call, if it is switched on.
kda_status scan_inputs(const kda::GdrScanArgs &a, kda_dtype dtype, cudaStream_t st) {
    if (!kda::debug_checks_enabled()) return KDA_OK;
    return from_cuda(kda::launch_gdr_scan(a, dtype == KDA_BF16, st));
}

// Sizes that the kernels' indexes and the workspaces' byte counts hold.
bool sizes_held(int64_t rows, int N, int H) {
    return rows <= INT32_MAX - 64 && (int64_t)N * H <= INT32_MAX / 8 && rows * H <= (int64_t)1 << 40;
}

// Checks shared by the calls over sequences; KDA_OK if they hold.
kda_status check_sequences(bool packed, int B, int64_t T, int N, int Hk, int H, int dk, int dv,
                           kda_dtype dtype) {
    if (B < 0 || T < 0 || N < 0 || Hk <= 0 || H <= 0 || dk <= 0 || dv <= 0)
        return KDA_ERR_INVALID_ARG;
    if (H % Hk != 0) return KDA_ERR_INVALID_ARG;
    if (dtype != KDA_F32 && dtype != KDA_BF16) return KDA_ERR_INVALID_ARG;
    if (packed ? B != 1 : N != B) return KDA_ERR_INVALID_ARG;
    if (!head_dim(dk) || !head_dim(dv)) return KDA_ERR_UNSUPPORTED;
    if (T > INT32_MAX - 64 || !sizes_held(B * T, N, H)) return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}

// Checks shared by the block norm's two directions.
kda_status check_norm(int64_t rows, int width, float scale, float eps, kda_dtype x_dtype,
                      kda_dtype dtype) {
    if (rows < 0 || width <= 0 || !std::isfinite(scale) || !(eps > 0.f) || !std::isfinite(eps))
        return KDA_ERR_INVALID_ARG;
    for (kda_dtype t : {x_dtype, dtype})
        if (t != KDA_F32 && t != KDA_BF16) return KDA_ERR_INVALID_ARG;
    if (x_dtype == KDA_BF16 && dtype == KDA_F32) return KDA_ERR_UNSUPPORTED;
    if (width > kda::kBlockNormMaxWidth || rows > INT32_MAX - 4096) return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}

}  // namespace

extern "C" {

size_t kda_gdr_prefill_workspace_bytes(int64_t rows, int N, int Hk, int H, int dk, int dv,
                                       kda_dtype dtype) {
    if (rows < 0 || N <= 0 || Hk <= 0 || H <= 0 || H % Hk != 0 || !head_dim(dk) || !head_dim(dv) ||
        !sizes_held(rows, N, H))
        return 0;
    return dtype == KDA_BF16 ? kda::gdr_image_bytes(rows, N, Hk, H, dk, false) : 0;
}

kda_status kda_gdr_chunk_prefill(const void *q, const void *k, const void *v, const void *g,
                                 const void *beta, const float *state_in,
                                 const int32_t *cu_seqlens, int B, int64_t T, int N, int Hk,
                                 int H, int dk, int dv, kda_dtype dtype, void *o,
                                 float *state_out, void *workspace, size_t workspace_bytes,
                                 void *stream) {
    const kda_status s = check_sequences(cu_seqlens != nullptr, B, T, N, Hk, H, dk, dv, dtype);
    if (s != KDA_OK) return s;
    if (B * T > 0 && (!q || !k || !v || !g || !beta || !o)) return KDA_ERR_INVALID_ARG;
    for (const void *p : {q, k, v, (const void *)o, (const void *)state_in,
                          (const void *)state_out})
        if (!aligned16(p)) return KDA_ERR_INVALID_ARG;
    if (N == 0) return KDA_OK;
    const size_t need = kda_gdr_prefill_workspace_bytes(B * T, N, Hk, H, dk, dv, dtype);
    if (need > 0 && (!workspace || workspace_bytes < need ||
                     (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0))
        return KDA_ERR_INVALID_ARG;
    uint32_t *err = kda::device_error_word();
    if (!err) return KDA_ERR_CUDA;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const kda_status scanned = scan_inputs(
        {k, g, beta, cu_seqlens, nullptr, T, N, Hk, H, dk, dtype == KDA_BF16, false, err}, dtype, st);
    if (scanned != KDA_OK) return scanned;
    kda::Profiler::begin(st);
    if (dtype == KDA_BF16) {
        const kda::GdrArgs a{q, k, v, g, beta, state_in, cu_seqlens, T, B * T, N, Hk, H, dk, dv,
                             o, state_out, err, kda::next_launch_epoch()};
        return from_cuda(kda::launch_gdr_prefill(a, workspace, st));
    }
    const kda::GdrTokenArgs a{q, k, v, g, beta, state_in, state_out, cu_seqlens, nullptr,
                              nullptr, T, N, N, Hk, H, dk, dv, o, err};
    return from_cuda(kda::launch_gdr_token_prefill(a, st));
}

kda_status kda_gdr_decode(const void *q, const void *k, const void *v, const void *g,
                          const void *beta, float *state, const int32_t *slots,
                          const int32_t *lens, int N, int P, int L, int Hk, int H, int dk,
                          int dv, kda_dtype dtype, int update_state, void *o, void *stream) {
    if (P < 0 || L < 0) return KDA_ERR_INVALID_ARG;
    const kda_status s = check_sequences(false, N, L, N, Hk, H, dk, dv, dtype);
    if (s != KDA_OK) return s;
    if (!slots && P < N) return KDA_ERR_INVALID_ARG;
    if (N > 0 && L > 0 && (!q || !k || !v || !g || !beta || !state || !o))
        return KDA_ERR_INVALID_ARG;
    if (!aligned16(state)) return KDA_ERR_INVALID_ARG;
    if (N == 0 || L == 0) return KDA_OK;
    uint32_t *err = kda::device_error_word();
    if (!err) return KDA_ERR_CUDA;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const kda_status scanned =
        scan_inputs({k, g, beta, nullptr, lens, L, N, Hk, H, dk, false, false, err}, dtype, st);
    if (scanned != KDA_OK) return scanned;
    kda::Profiler::begin(st);
    const kda::GdrTokenArgs a{q, k, v, g, beta, state, update_state ? state : nullptr, nullptr,
                              slots, lens, L, N, P, Hk, H, dk, dv, o, err};
    return from_cuda(kda::launch_gdr_token(a, dtype == KDA_BF16, st));
}

size_t kda_gdr_backward_workspace_bytes(int64_t rows, int N, int Hk, int H, int dk, int dv,
                                        kda_dtype dtype) {
    if (rows < 0 || N < 0 || Hk <= 0 || H <= 0 || H % Hk != 0 || !head_dim(dk) || !head_dim(dv) ||
        !sizes_held(rows, N, H))
        return 0;
    return kda::gdr_backward_workspace_bytes(rows, N, Hk, H, dk, dv, dtype == KDA_BF16);
}

kda_status kda_gdr_backward(const void *q, const void *k, const void *v, const void *g,
                            const void *beta, const float *state_in, const int32_t *cu_seqlens,
                            int B, int64_t T, int N, int Hk, int H, int dk, int dv,
                            kda_dtype dtype, const void *dout, const float *dstate_out, void *dq,
                            void *dk_out, void *dv_out, void *dg, void *dbeta, float *dstate_in,
                            void *workspace, size_t workspace_bytes, void *stream) {
    const kda_status s = check_sequences(cu_seqlens != nullptr, B, T, N, Hk, H, dk, dv, dtype);
    if (s != KDA_OK) return s;
    const int64_t rows = B * T;
    if (rows > 0 && (!q || !k || !v || !g || !beta || !dout || !dq || !dk_out || !dv_out || !dg ||
                     !dbeta))
        return KDA_ERR_INVALID_ARG;
    for (const void *p : {q, k, v, dout, (const void *)state_in, (const void *)dstate_out,
                          (const void *)dq, (const void *)dk_out, (const void *)dv_out,
                          (const void *)dstate_in})
        if (!aligned16(p)) return KDA_ERR_INVALID_ARG;
    if ((rows / 64 + N + 1) * Hk > INT32_MAX) return KDA_ERR_UNSUPPORTED;
    if (N == 0) return KDA_OK;
    const size_t need = kda_gdr_backward_workspace_bytes(rows, N, Hk, H, dk, dv, dtype);
    if (!workspace || workspace_bytes < need || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
        return KDA_ERR_INVALID_ARG;
    uint32_t *err = kda::device_error_word();
    if (!err) return KDA_ERR_CUDA;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const kda_status scanned = scan_inputs({k, g, beta, cu_seqlens, nullptr, T, N, Hk, H, dk, dtype == KDA_BF16,
                                            dtype == KDA_BF16, err}, dtype, st);
    if (scanned != KDA_OK) return scanned;
    kda::Profiler::begin(st);
    const kda::GdrArgs a{q, k, v, g, beta, state_in, cu_seqlens, T, B * T, N, Hk, H, dk, dv,
                         nullptr, nullptr, err, kda::next_launch_epoch()};
    const kda::GdrGrads gr{dout, dstate_out, dq, dk_out, dv_out, dg, dbeta, dstate_in};
    return from_cuda(kda::launch_gdr_backward(a, gr, rows, dtype == KDA_BF16, workspace, st));
}

kda_status kda_block_norm(const void *x, const void *y, const void *gate, const void *w_post,
                          const void *w_pre, int64_t rows, int width, float scale, float eps,
                          kda_dtype x_dtype, kda_dtype dtype, void *x_new, void *h,
                          void *stream) {
    const kda_status s = check_norm(rows, width, scale, eps, x_dtype, dtype);
    if (s != KDA_OK) return s;
    if (rows == 0) return KDA_OK;
    if (!x || !y || !w_post || !w_pre || !x_new || !h) return KDA_ERR_INVALID_ARG;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    kda::Profiler::begin(st);
    uint32_t *err = kda::device_error_word();
    if (!err) return KDA_ERR_CUDA;
    kda::BlockNormArgs a{x, y, gate, w_post, w_pre, rows, width, scale, eps, x_new, h};
    a.err = err;
    a.epoch = kda::next_launch_epoch();
    return from_cuda(kda::launch_block_norm(a, x_dtype == KDA_BF16, dtype == KDA_BF16, false, st));
}

size_t kda_block_norm_backward_workspace_bytes(int64_t rows, int width) {
    if (rows < 0 || width <= 0 || width > kda::kBlockNormMaxWidth) return 0;
    return kda::block_norm_parts(rows, width) * 2 * (size_t)width * sizeof(float);
}

kda_status kda_block_norm_backward(const void *x, const void *y, const void *gate,
                                   const void *w_post, const void *w_pre, const void *dx_new,
                                   const void *dh, int64_t rows, int width, float scale,
                                   float eps, kda_dtype x_dtype, kda_dtype dtype, void *dx,
                                   void *dy, void *dgate, float *dw_post, float *dw_pre,
                                   void *workspace, size_t workspace_bytes, void *stream) {
    const kda_status s = check_norm(rows, width, scale, eps, x_dtype, dtype);
    if (s != KDA_OK) return s;
    if (!dw_post || !dw_pre) return KDA_ERR_INVALID_ARG;
    if (rows > 0 && (!x || !y || !w_post || !w_pre || !dx || !dy || (gate && !dgate)))
        return KDA_ERR_INVALID_ARG;
    const size_t need = kda_block_norm_backward_workspace_bytes(rows, width);
    if (need > 0 && (!workspace || workspace_bytes < need ||
                     (reinterpret_cast<uintptr_t>(workspace) & 3u) != 0))
        return KDA_ERR_INVALID_ARG;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    kda::Profiler::begin(st);
    uint32_t *err = kda::device_error_word();
    if (!err) return KDA_ERR_CUDA;
    kda::BlockNormArgs a{x, y, gate, w_post, w_pre, rows, width, scale, eps, nullptr, nullptr,
                         dx_new, dh, dx, dy, dgate, dw_post, dw_pre,
                         static_cast<float *>(workspace), err, kda::next_launch_epoch()};
    return from_cuda(kda::launch_block_norm(a, x_dtype == KDA_BF16, dtype == KDA_BF16, true, st));
}

}  // extern "C"
