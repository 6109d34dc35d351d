// Gated delta rule, backward of fp32 inputs, token by token in fp32.
//
// With delta_t = beta_t err_t, err_t = v_t - a_t S_{t-1}^T k_t and Z = dL/dS_t, per token from
// the last to the first:
//     Z += q do^T;   dd = Z^T k;   derr = beta dd = dv;   dbeta = dd . err
//     dq = S_t do;   dk = Z delta - a S_{t-1} derr
//     Z -= k derr^T;  dg = a <S_{t-1}, Z>;  Z *= a
//
// The columns of S and Z are independent: one CTA of 256 threads per (sequence, head, slice of
// 32 columns), each thread with DK / 32 rows x 4 columns of both in registers.  It first walks
// the tokens forward and stores the state before every block of 32 tokens, then the blocks from
// the last: it forms the block's states again (each thread keeps its own part of each token's
// state in the CTA's scratch, so no thread waits for another's), then goes back through them.
// A slice's shares of dq, dk, dg and dbeta go to partial arrays that a second kernel adds up
// over the slices, and dq and dk over the heads of a group, in a fixed order.
//
// What bounds it is the barriers, six a token: two for the sum over all channels and what follows from
// it in each of the walk forward, the block's states formed again and the walk back.  2048 tokens of 4
// heads of 64: 2.34 ms (1.1 us a token); of 16 heads of 128: 3.9 ms.
#include "gdr_common.cuh"
#include "gdr_launch.h"
#include "gdr_token_backward.h"

namespace kda {
namespace gdr {

constexpr int kTB = 32;          // tokens per block
constexpr int kCols = 32;        // columns per CTA
constexpr int kTokenGrid = 296;  // CTAs at most: two per SM

template <int DK>
struct TokenBackwardSmem {
    float k[kTB][DK], q[kTB][DK];
    float v[kTB][kCols], dout[kTB][kCols], delta[kTB][kCols], err[kTB][kCols];
    float a[kTB], beta[kTB], dg[kTB][8];
    float4 red[2][8][8];
    float4 derr[2][8];
};

template <int DK>
__global__ void __launch_bounds__(256, 2) gdr_token_backward_kernel(TokenBackwardArgs a) {
    constexpr int RPT = DK / 32;
    extern __shared__ __align__(16) unsigned char smem_raw[];
    auto &sm = *reinterpret_cast<TokenBackwardSmem<DK> *>(smem_raw);
    const int tid = threadIdx.x, cg = tid & 7, rg = tid >> 3, warp = tid >> 5, lane = tid & 31;
    const int slices = a.dv / kCols;
    const int64_t items = (int64_t)a.N * a.H * slices;
    float4 *scratch = reinterpret_cast<float4 *>(a.scratch) + (int64_t)blockIdx.x * kTB * DK * 8 + tid;

    for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
        const int slice = (int)(item % slices), unit = (int)(item / slices);
        const int h = unit % a.H, n = unit / a.H, hk = h / (a.H / a.Hk);
        const Span span = sequence_span(a.cu, n, a.T);
        const int blocks = (span.len + kTB - 1) / kTB;
        const int64_t slot0 = span.row / kTB + n;
        const int64_t soff = ((int64_t)n * a.H + h) * DK * a.dv + slice * kCols + cg * 4;

        // inputs of a block into shared memory
        auto load = [&](int blk, bool with_grad) {
            const int m = min(kTB, span.len - blk * kTB);
            const int64_t row = span.row + (int64_t)blk * kTB;
            __syncthreads();
            for (int i = tid; i < m * DK; i += 256) {
                const int t = i / DK, c = i % DK;
                const int64_t at = ((row + t) * a.Hk + hk) * DK + c;
                sm.k[t][c] = a.k[at];
                if (with_grad) sm.q[t][c] = a.q[at];
            }
            for (int i = tid; i < m * kCols; i += 256) {
                const int t = i / kCols, j = i % kCols;
                const int64_t at = ((row + t) * a.H + h) * a.dv + slice * kCols + j;
                sm.v[t][j] = a.v[at];
                if (with_grad) sm.dout[t][j] = a.dout[at];
            }
            if (tid < m) {
                sm.a[tid] = decay(a.g[(row + tid) * a.H + h]);
                sm.beta[tid] = a.beta[(row + tid) * a.H + h];
            }
            __syncthreads();
            return m;
        };
        // sum over the channels of each column: a thread's rows are in x
        auto over_channels = [&](float4 x, int b) {
#pragma unroll
            for (int m = 8; m < 32; m <<= 1) {
                x.x += __shfl_xor_sync(0xffffffffu, x.x, m);
                x.y += __shfl_xor_sync(0xffffffffu, x.y, m);
                x.z += __shfl_xor_sync(0xffffffffu, x.z, m);
                x.w += __shfl_xor_sync(0xffffffffu, x.w, m);
            }
            if (lane < 8) sm.red[b][warp][lane] = x;
            __syncthreads();
        };
        auto column = [&](int b) {   // of column tid, after over_channels
            float s = 0.f;
#pragma unroll
            for (int w = 0; w < 8; ++w) s += reinterpret_cast<const float *>(&sm.red[b][w][0])[tid];
            return s;
        };

        float4 s[RPT];
        auto step = [&](int t, int b) {   // one token forward; err and delta of the slice kept
            float4 p = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int i = 0; i < RPT; ++i) {
                const float kr = sm.k[t][rg + 32 * i];
                p.x = fmaf(s[i].x, kr, p.x); p.y = fmaf(s[i].y, kr, p.y);
                p.z = fmaf(s[i].z, kr, p.z); p.w = fmaf(s[i].w, kr, p.w);
            }
            over_channels(p, b);
            const float dec = sm.a[t];
            if (tid < kCols) {
                const float e = sm.v[t][tid] - dec * column(b);
                sm.err[t][tid] = e;
                sm.delta[t][tid] = sm.beta[t] * e;
            }
            __syncthreads();
            const float4 d = *reinterpret_cast<const float4 *>(&sm.delta[t][cg * 4]);
#pragma unroll
            for (int i = 0; i < RPT; ++i) {
                const float kr = sm.k[t][rg + 32 * i];
                s[i].x = fmaf(kr, d.x, dec * s[i].x); s[i].y = fmaf(kr, d.y, dec * s[i].y);
                s[i].z = fmaf(kr, d.z, dec * s[i].z); s[i].w = fmaf(kr, d.w, dec * s[i].w);
            }
        };
        auto block_state = [&](int blk) {
            return reinterpret_cast<float4 *>(a.blocks + ((slot0 + blk) * a.H + h) * DK * a.dv +
                                              slice * kCols + cg * 4);
        };

#pragma unroll
        for (int i = 0; i < RPT; ++i)
            s[i] = a.state_in ? *reinterpret_cast<const float4 *>(a.state_in + soff + (int64_t)(rg + 32 * i) * a.dv)
                              : make_float4(0.f, 0.f, 0.f, 0.f);
        for (int blk = 0; blk < blocks; ++blk) {
            float4 *dst = block_state(blk);
#pragma unroll
            for (int i = 0; i < RPT; ++i) dst[(int64_t)(rg + 32 * i) * a.dv / 4] = s[i];
            if (blk + 1 == blocks) break;
            load(blk, false);
            for (int t = 0; t < kTB; ++t) step(t, t & 1);
        }

        float4 z[RPT];
#pragma unroll
        for (int i = 0; i < RPT; ++i)
            z[i] = a.dstate_out
                       ? *reinterpret_cast<const float4 *>(a.dstate_out + soff + (int64_t)(rg + 32 * i) * a.dv)
                       : make_float4(0.f, 0.f, 0.f, 0.f);
        for (int blk = blocks - 1; blk >= 0; --blk) {
            const int m = load(blk, true);
            const int64_t row = span.row + (int64_t)blk * kTB;
            const float4 *src = block_state(blk);
#pragma unroll
            for (int i = 0; i < RPT; ++i) s[i] = src[(int64_t)(rg + 32 * i) * a.dv / 4];
            for (int t = 0; t < m; ++t) {
#pragma unroll
                for (int i = 0; i < RPT; ++i) scratch[(t * RPT + i) * 256] = s[i];
                step(t, t & 1);
            }
            for (int t = m - 1; t >= 0; --t) {
                const int b = t & 1;
                const float dec = sm.a[t];
                float4 sp[RPT];
#pragma unroll
                for (int i = 0; i < RPT; ++i) sp[i] = scratch[(t * RPT + i) * 256];
                const float4 o = *reinterpret_cast<const float4 *>(&sm.dout[t][cg * 4]);
                float4 p = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int i = 0; i < RPT; ++i) {
                    const float qr = sm.q[t][rg + 32 * i], kr = sm.k[t][rg + 32 * i];
                    z[i].x = fmaf(qr, o.x, z[i].x); z[i].y = fmaf(qr, o.y, z[i].y);
                    z[i].z = fmaf(qr, o.z, z[i].z); z[i].w = fmaf(qr, o.w, z[i].w);
                    p.x = fmaf(z[i].x, kr, p.x); p.y = fmaf(z[i].y, kr, p.y);
                    p.z = fmaf(z[i].z, kr, p.z); p.w = fmaf(z[i].w, kr, p.w);
                }
                over_channels(p, b);
                const int64_t at = (row + t) * a.H + h;
                if (tid < kCols) {
                    const float dd = column(b), de = sm.beta[t] * dd;
                    reinterpret_cast<float *>(sm.derr[b])[tid] = de;
                    a.dv_out[at * a.dv + slice * kCols + tid] = de;
                    float db = dd * sm.err[t][tid];
#pragma unroll
                    for (int x = 16; x > 0; x >>= 1) db += __shfl_xor_sync(0xffffffffu, db, x);
                    if (tid == 0) a.part_b[at * slices + slice] = db;
                }
                __syncthreads();
                const float4 de = sm.derr[b][cg];
                const float4 dl = *reinterpret_cast<const float4 *>(&sm.delta[t][cg * 4]);
                const float ldo = dl.x * o.x + dl.y * o.y + (dl.z * o.z + dl.w * o.w);
                float dg = 0.f;
#pragma unroll
                for (int i = 0; i < RPT; ++i) {
                    const float kr = sm.k[t][rg + 32 * i];
                    const float4 u = make_float4(dec * sp[i].x, dec * sp[i].y, dec * sp[i].z, dec * sp[i].w);
                    float dq = u.x * o.x + u.y * o.y + (u.z * o.z + u.w * o.w) + kr * ldo;
                    float dk = z[i].x * dl.x + z[i].y * dl.y + (z[i].z * dl.z + z[i].w * dl.w) -
                               (u.x * de.x + u.y * de.y + (u.z * de.z + u.w * de.w));
#pragma unroll
                    for (int x = 1; x < 8; x <<= 1) {
                        dq += __shfl_xor_sync(0xffffffffu, dq, x);
                        dk += __shfl_xor_sync(0xffffffffu, dk, x);
                    }
                    if (cg == 0) {
                        const int64_t to = (at * slices + slice) * DK + rg + 32 * i;
                        a.part_q[to] = dq;
                        a.part_k[to] = dk;
                    }
                    z[i].x -= kr * de.x; z[i].y -= kr * de.y; z[i].z -= kr * de.z; z[i].w -= kr * de.w;
                    dg += u.x * z[i].x + u.y * z[i].y + (u.z * z[i].z + u.w * z[i].w);
                    z[i].x *= dec; z[i].y *= dec; z[i].z *= dec; z[i].w *= dec;
                }
#pragma unroll
                for (int x = 16; x > 0; x >>= 1) dg += __shfl_xor_sync(0xffffffffu, dg, x);
                if (lane == 0) sm.dg[t][warp] = dg;
            }
            __syncthreads();
            if (tid < m) {
                float d = 0.f;
#pragma unroll
                for (int w = 0; w < 8; ++w) d += sm.dg[tid][w];
                a.part_g[((row + tid) * a.H + h) * slices + slice] = d;
            }
        }
        if (a.dstate_in)
#pragma unroll
            for (int i = 0; i < RPT; ++i)
                *reinterpret_cast<float4 *>(a.dstate_in + soff + (int64_t)(rg + 32 * i) * a.dv) = z[i];
        __syncthreads();
    }
}

// dq and dk over the slices and the heads of a group, dg and dbeta over the slices, for the rows
// of sequence blockIdx.x.
__global__ void __launch_bounds__(256) gdr_token_gradsum_kernel(TokenBackwardArgs a, int dk) {
    const int n = blockIdx.x, slices = a.dv / kCols, group = a.H / a.Hk;
    const Span span = sequence_span(a.cu, n, a.T);
    for (int r = blockIdx.y; r < span.len; r += gridDim.y) {
        const int64_t row = span.row + r;
        for (int i = threadIdx.x; i < a.Hk * dk; i += 256) {
            const int hk = i / dk, c = i % dk;
            float x = 0.f, y = 0.f;
            for (int p = 0; p < group * slices; ++p) {
                const int64_t at = ((row * a.H + hk * group) * slices + p) * dk + c;
                x += a.part_q[at];
                y += a.part_k[at];
            }
            a.dq[row * a.Hk * dk + i] = x;
            a.dk[row * a.Hk * dk + i] = y;
        }
        for (int i = threadIdx.x; i < a.H; i += 256) {
            float x = 0.f, y = 0.f;
            for (int p = 0; p < slices; ++p) {
                x += a.part_g[(row * a.H + i) * slices + p];
                y += a.part_b[(row * a.H + i) * slices + p];
            }
            a.dg[row * a.H + i] = x;
            a.dbeta[row * a.H + i] = y;
        }
    }
}

static size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }
static int64_t token_grid(int N, int H, int dv) {
    const int64_t items = (int64_t)N * H * (dv / kCols);
    return items < kTokenGrid ? items : kTokenGrid;
}

template <int DK>
static cudaError_t launch_token_backward_t(const TokenBackwardArgs &a, cudaStream_t st) {
    constexpr int bytes = sizeof(TokenBackwardSmem<DK>);
    static_assert(2 * bytes <= 224 * 1024, "two CTAs per SM");
    cudaError_t e = cudaFuncSetAttribute(gdr_token_backward_kernel<DK>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    gdr_token_backward_kernel<DK><<<(unsigned)token_grid(a.N, a.H, a.dv), 256, bytes, st>>>(a);
    e = cudaGetLastError();
    Profiler::mark(st);
    return e;
}

size_t token_backward_workspace_bytes(int64_t rows, int N, int H, int dk, int dv) {
    const size_t slices = dv / kCols, units = (size_t)rows * H * slices;
    return up256((size_t)(rows / kTB + N + 1) * H * dk * dv * 4) +
           up256((size_t)token_grid(N, H, dv) * kTB * dk * kCols * 4) + 2 * up256(units * dk * 4) +
           2 * up256(units * 4);
}

cudaError_t launch_token_backward(const GdrArgs &p, const GdrGrads &g, int64_t rows, void *workspace,
                                  cudaStream_t st) {
    unsigned char *w = static_cast<unsigned char *>(workspace);
    auto take = [&](size_t bytes) {
        float *r = reinterpret_cast<float *>(w);
        w += up256(bytes);
        return r;
    };
    const size_t units = (size_t)rows * p.H * (p.dv / kCols);
    TokenBackwardArgs a{(const float *)p.q, (const float *)p.k, (const float *)p.v, (const float *)p.g,
                        (const float *)p.beta, (const float *)g.dout, p.state_in, g.dstate_out,
                        p.cu_seqlens, p.T, p.N, p.Hk, p.H, p.dv, (float *)g.dq, (float *)g.dk,
                        (float *)g.dv, (float *)g.dg, (float *)g.dbeta, g.dstate_in};
    a.blocks = take((size_t)(rows / kTB + p.N + 1) * p.H * p.dk * p.dv * 4);
    a.scratch = take((size_t)token_grid(p.N, p.H, p.dv) * kTB * p.dk * kCols * 4);
    a.part_q = take(units * p.dk * 4);
    a.part_k = take(units * p.dk * 4);
    a.part_g = take(units * 4);
    a.part_b = take(units * 4);
    cudaError_t e = p.dk == 64 ? launch_token_backward_t<64>(a, st) : launch_token_backward_t<128>(a, st);
    if (e != cudaSuccess || rows == 0) return e;
    const int64_t y = p.T < 1024 ? (p.T > 0 ? p.T : 1) : 1024;
    gdr_token_gradsum_kernel<<<dim3((unsigned)p.N, (unsigned)y), 256, 0, st>>>(a, p.dk);
    e = cudaGetLastError();
    Profiler::mark(st);
    return e;
}

}  // namespace gdr
}  // namespace kda
