// Block norm: what closes one block of a model and opens the next, in one pass.
//
//     n  = y rsqrt(mean y^2 + eps) w_post          norm after the block
//     x' = x + scale sigmoid(gate) n               gate, scaled residual sum
//     h  = x' rsqrt(mean x'^2 + eps) w_pre         norm before the next block
//
// Both directions are bound by HBM: every input is read once and every output written
// once, a row's values stay in registers between the two row sums.  All arithmetic is
// fp32; h is taken from the unrounded x'.
//
// Backward, with r_y, r_x the two rsqrt factors, a = sigmoid(gate), D the width:
//     gx = dh w_pre;   dx = dx' + r_x (gx - x' r_x^2 sum(gx x') / D)
//     dn = scale a dx; gy = dn w_post;  dy = r_y (gy - y r_y^2 sum(gy y) / D)
//     dgate = scale dx n a (1 - a);  dw_pre = sum_rows dh x' r_x;  dw_post = sum_rows dn y r_y
// x' is formed again from x, y and gate (as many bytes as reading it).  The weight
// gradients are summed per CTA over its rows in registers, then over the CTAs by a second
// kernel, both in a fixed order.
#include "block_norm.h"
#include "kda_common.cuh"

namespace kda {
namespace {

// V consecutive elements as loaded: 16 bytes of bf16, 32 of fp32, or one element.  They stay
// packed in registers and are widened where they are used.
template <int V, typename T>
struct Pack {
    static constexpr int WORDS = V == 1 ? 1 : V * (int)sizeof(T) / 4;
    uint32_t w[WORDS];
    __device__ __forceinline__ void load(const T *p) {
        if constexpr (V == 1) {
            w[0] = __float_as_uint(to_f32(*p));
        } else {
#pragma unroll
            for (int i = 0; i < WORDS / 4; ++i) {
                const uint4 u = __ldcs(reinterpret_cast<const uint4 *>(p) + i);
                w[4 * i] = u.x; w[4 * i + 1] = u.y; w[4 * i + 2] = u.z; w[4 * i + 3] = u.w;
            }
        }
    }
    __device__ __forceinline__ void load_shared(const T *p) {   // weights: read by every row
        if constexpr (V == 1) {
            w[0] = __float_as_uint(to_f32(__ldg(p)));
        } else {
#pragma unroll
            for (int i = 0; i < WORDS / 4; ++i) {
                const uint4 u = __ldg(reinterpret_cast<const uint4 *>(p) + i);
                w[4 * i] = u.x; w[4 * i + 1] = u.y; w[4 * i + 2] = u.z; w[4 * i + 3] = u.w;
            }
        }
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < WORDS; ++i) w[i] = 0u;
    }
    __device__ __forceinline__ float get(int j) const {
        if constexpr (V == 1 || sizeof(T) == 4) return __uint_as_float(w[j]);
        else return __uint_as_float((j & 1) ? w[j / 2] & 0xffff0000u : w[j / 2] << 16);
    }
};

template <int V, typename T>
__device__ __forceinline__ void store(T *p, const float (&x)[V]) {
    if constexpr (V == 1) {
        *p = from_f32<T>(x[0]);
    } else if constexpr (sizeof(T) == 2) {
        uint32_t u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
            u[i] = reinterpret_cast<const uint32_t &>(b);
        }
        __stcs(reinterpret_cast<uint4 *>(p), make_uint4(u[0], u[1], u[2], u[3]));
    } else {
#pragma unroll
        for (int i = 0; i < 2; ++i)
            __stcs(reinterpret_cast<float4 *>(p) + i,
                   make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]));
    }
}

// Sums of x and y over the TPR threads of a row, the same bits in each: within a warp by
// shuffles, across warps through shared memory (then the CTA is one row).  `red` is a slot of
// its own for each call between two barriers.
template <int TPR>
__device__ __forceinline__ float2 row_sum(float x, float y, float2 *red) {
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) {
        x += __shfl_xor_sync(0xffffffffu, x, m);
        y += __shfl_xor_sync(0xffffffffu, y, m);
    }
    if constexpr (TPR > 32) {
        if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = make_float2(x, y);
        __syncthreads();
        x = y = 0.f;
#pragma unroll
        for (int w = 0; w < TPR / 32; ++w) {
            const float2 v = red[w];
            x += v.x;
            y += v.y;
        }
    }
    return make_float2(x, y);
}

__device__ __forceinline__ float sigmoid(float x) { return __fdividef(1.f, 1.f + __expf(-x)); }

// V elements per vector, NV vectors per thread, TPR threads per row.
template <int V, int NV, int TPR, typename TX, typename T>
__global__ void __launch_bounds__(TPR > 256 ? TPR : 256) block_norm_kernel(BlockNormArgs a) {
    constexpr int RPC = TPR > 32 ? 1 : 8;   // rows per CTA
    __shared__ float2 red[2][TPR / 32];
    const int t = threadIdx.x % TPR;
    const int64_t row = (int64_t)blockIdx.x * RPC + threadIdx.x / TPR;
    if (RPC > 1 && row >= a.rows) return;   // a whole warp
    const int D = a.width;
    const int64_t at = row * D;
    const bool gated = a.gate != nullptr;

    Pack<V, TX> x[NV];
    Pack<V, T> y[NV], g[NV], wo[NV], wi[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * TPR + t) * V;
        y[i].zero();
        if (c < D) {
            y[i].load((const T *)a.y + at + c);
            x[i].load((const TX *)a.x + at + c);
            if (gated) g[i].load((const T *)a.gate + at + c);
            wo[i].load_shared((const T *)a.w_post + c);
            wi[i].load_shared((const T *)a.w_pre + c);
        }
    }
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) ss = fmaf(y[i].get(j), y[i].get(j), ss);
    const float ry = rsqrtf(row_sum<TPR>(ss, 0.f, red[0]).x / D + a.eps) * a.scale;
    float xn[NV][V];
    ss = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * TPR + t) * V;
        if (c >= D) continue;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const float s = gated ? sigmoid(g[i].get(j)) : 1.f;
            xn[i][j] = fmaf(y[i].get(j) * ry * wo[i].get(j), s, x[i].get(j));
            ss = fmaf(xn[i][j], xn[i][j], ss);
        }
        store<V>((TX *)a.x_new + at + c, xn[i]);
    }
    const float rx = rsqrtf(row_sum<TPR>(ss, 0.f, red[1]).x / D + a.eps);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * TPR + t) * V;
        if (c >= D) continue;
        float h[V];
#pragma unroll
        for (int j = 0; j < V; ++j) h[j] = xn[i][j] * rx * wi[i].get(j);
        store<V>((T *)a.h + at + c, h);
    }
}

// A row's inputs to the backward, as loaded.
template <int V, int NV, int TPR, typename TX, typename T>
struct BackwardRow {
    Pack<V, TX> x[NV], dx[NV];
    Pack<V, T> y[NV], g[NV], dh[NV];
    __device__ __forceinline__ void load(const BlockNormArgs &a, int64_t row, int t) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * TPR + t) * V;
            const int64_t at = row * a.width + c;
            x[i].zero(); dx[i].zero(); y[i].zero(); g[i].zero(); dh[i].zero();
            if (row < a.rows && c < a.width) {
                y[i].load((const T *)a.y + at);
                x[i].load((const TX *)a.x + at);
                if (a.gate) g[i].load((const T *)a.gate + at);
                if (a.dh) dh[i].load((const T *)a.dh + at);
                if (a.dx_new) dx[i].load((const TX *)a.dx_new + at);
            }
        }
    }
};

// A CTA walks rows blockIdx.x RPC + k gridDim.x RPC; the next row is on its way while one is
// worked on.  Its sums of the weight gradients go to part[cta][2][D] (with several rows side by
// side, to part[cta RPC + side]).
template <int V, int NV, int TPR, typename TX, typename T>
__global__ void __launch_bounds__(TPR > 256 ? TPR : 256, TPR > 256 ? 1 : 2)
    block_norm_backward_kernel(BlockNormArgs a) {
    constexpr int RPC = TPR > 32 ? 1 : 8;
    __shared__ float2 red[2][3][TPR / 32];
    const int t = threadIdx.x % TPR, side = threadIdx.x / TPR;
    const int D = a.width;
    const bool gated = a.gate != nullptr;
    const float inv_d = 1.f / D;
    float dwo[NV][V], dwi[NV][V];
    Pack<V, T> wo[NV], wi[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        wo[i].zero(), wi[i].zero();
        if ((i * TPR + t) * V < D) {
            wo[i].load_shared((const T *)a.w_post + (i * TPR + t) * V);
            wi[i].load_shared((const T *)a.w_pre + (i * TPR + t) * V);
        }
#pragma unroll
        for (int j = 0; j < V; ++j) dwo[i][j] = dwi[i][j] = 0.f;
    }
    BackwardRow<V, NV, TPR, TX, T> next;
    const int64_t first = (int64_t)blockIdx.x * RPC + side, step = (int64_t)gridDim.x * RPC;
    next.load(a, first, t);
    int turn = 0;
    for (int64_t row = first; row < a.rows; row += step, turn ^= 1) {
        const BackwardRow<V, NV, TPR, TX, T> in = next;
        next.load(a, row + step, t);
        const int64_t at = row * D;
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j) ss = fmaf(in.y[i].get(j), in.y[i].get(j), ss);
        const float ry = rsqrtf(row_sum<TPR>(ss, 0.f, red[turn][0]).x / D + a.eps);
        // x' and the gate; the two sums of the second norm
        float xn[NV][V], s[NV][V], sx = 0.f, sg = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j) {
                s[i][j] = gated ? sigmoid(in.g[i].get(j)) : 1.f;
                xn[i][j] = fmaf(in.y[i].get(j) * ry * wo[i].get(j), a.scale * s[i][j], in.x[i].get(j));
                sx = fmaf(xn[i][j], xn[i][j], sx);
                sg = fmaf(in.dh[i].get(j) * wi[i].get(j), xn[i][j], sg);
            }
        const float2 two = row_sum<TPR>(sx, sg, red[turn][1]);
        const float rx = rsqrtf(two.x / D + a.eps), kx = rx * rx * rx * (two.y * inv_d);
        float gy[NV][V], sy = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * TPR + t) * V;
            float dx[V], dg[V];
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float h = in.dh[i].get(j), yn = in.y[i].get(j) * ry;
                dwi[i][j] = fmaf(h, xn[i][j] * rx, dwi[i][j]);
                dx[j] = in.dx[i].get(j) + rx * (h * wi[i].get(j)) - kx * xn[i][j];
                const float dn = a.scale * dx[j] * s[i][j];
                dg[j] = dn * (1.f - s[i][j]) * (yn * wo[i].get(j));
                dwo[i][j] = fmaf(dn, yn, dwo[i][j]);
                gy[i][j] = dn * wo[i].get(j);
                sy = fmaf(gy[i][j], in.y[i].get(j), sy);
            }
            if (c < D) {
                store<V>((TX *)a.dx + at + c, dx);
                if (gated) store<V>((T *)a.dgate + at + c, dg);
            }
        }
        const float ky = ry * ry * ry * (row_sum<TPR>(sy, 0.f, red[turn][2]).x * inv_d);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * TPR + t) * V;
            float d[V];
#pragma unroll
            for (int j = 0; j < V; ++j) d[j] = fmaf(ry, gy[i][j], -ky * in.y[i].get(j));
            if (c < D) store<V>((T *)a.dy + at + c, d);
        }
    }
    float *part = a.part + ((int64_t)blockIdx.x * RPC + side) * 2 * D;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * TPR + t) * V;
        if (c >= D) continue;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            part[c + j] = dwo[i][j];
            part[D + c + j] = dwi[i][j];
        }
    }
}

// Column sums of part[parts][2 D] in a fixed order: 32 columns and 8 groups of rows per CTA.
__global__ void __launch_bounds__(256) block_norm_weights_kernel(const float *part, int parts,
                                                                 int D, float *dw_post,
                                                                 float *dw_pre) {
    __shared__ float red[8][33];
    const int col = blockIdx.x * 32 + (threadIdx.x & 31), group = threadIdx.x >> 5;
    float s = 0.f;
    if (col < 2 * D)
#pragma unroll 8
        for (int i = group; i < parts; i += 8) s += part[(int64_t)i * 2 * D + col];
    red[group][threadIdx.x & 31] = s;
    __syncthreads();
    if (group == 0 && col < 2 * D) {
        s = 0.f;
#pragma unroll
        for (int g = 0; g < 8; ++g) s += red[g][threadIdx.x];
        (col < D ? dw_post[col] : dw_pre[col - D]) = s;
    }
}

constexpr int kSMs = 148;

// Rows of partial weight gradients: as many CTAs as run at once, or as there are rows.
int64_t grid_of(int64_t rows, int rpc, bool backward) {
    const int64_t all = (rows + rpc - 1) / rpc;
    return backward ? (all < 2 * kSMs ? all : 2 * kSMs) : all;
}

template <int V, int NV, int TPR, typename TX, typename T>
cudaError_t launch_t(BlockNormArgs a, bool backward, cudaStream_t st) {
    constexpr int RPC = TPR > 32 ? 1 : 8, threads = TPR > 32 ? TPR : 256;
    const int64_t grid = grid_of(a.rows, RPC, backward);
    if (!backward) {
        block_norm_kernel<V, NV, TPR, TX, T><<<(unsigned)grid, threads, 0, st>>>(a);
    } else {
        if (grid > 0) {
            block_norm_backward_kernel<V, NV, TPR, TX, T><<<(unsigned)grid, threads, 0, st>>>(a);
            const cudaError_t e = cudaGetLastError();
            if (e != cudaSuccess) return e;
            Profiler::mark(st);
        }
        block_norm_weights_kernel<<<(2 * a.width + 31) / 32, 256, 0, st>>>(
            a.part, (int)grid * RPC, a.width, a.dw_post, a.dw_pre);
    }
    const cudaError_t e = cudaGetLastError();
    Profiler::mark(st);
    return e;
}

// Threads per row: one vector a thread up to 512 of them; a row's values and the next one's
// then fit the registers in either direction.
template <int V, typename TX, typename T>
cudaError_t launch_v(const BlockNormArgs &a, bool b, cudaStream_t st) {
    const int vecs = (a.width + V - 1) / V;
    if (vecs <= 32) return launch_t<V, 1, 32, TX, T>(a, b, st);
    if (vecs <= 64) return launch_t<V, 1, 64, TX, T>(a, b, st);
    if (vecs <= 128) return launch_t<V, 1, 128, TX, T>(a, b, st);
    if (vecs <= 256) return launch_t<V, 1, 256, TX, T>(a, b, st);
    if (vecs <= 512) return launch_t<V, 1, 512, TX, T>(a, b, st);
    if (vecs <= 1024) return launch_t<V, 2, 512, TX, T>(a, b, st);
    if constexpr (V == 8) {
        return launch_t<V, 4, 512, TX, T>(a, b, st);
    } else {
        if (vecs <= 4096) return launch_t<V, 8, 512, TX, T>(a, b, st);
        return launch_t<V, 32, 512, TX, T>(a, b, st);
    }
}

bool vectors(const BlockNormArgs &a) {
    if (a.width % 8) return false;
    for (const void *p : {a.x, a.y, a.gate, a.w_post, a.w_pre, a.dx_new, a.dh, (const void *)a.x_new,
                          (const void *)a.h, (const void *)a.dx, (const void *)a.dy,
                          (const void *)a.dgate})
        if (reinterpret_cast<uintptr_t>(p) & 15u) return false;
    return true;
}

}  // namespace

size_t block_norm_parts(int64_t rows, int width) {
    // rows side by side only where a row has at most 32 vectors; an upper bound for both
    const int rpc = width <= 256 ? 8 : 1;
    const int64_t one = grid_of(rows, 1, true), many = grid_of(rows, rpc, true) * rpc;
    return (size_t)(one > many ? one : many);
}

cudaError_t launch_block_norm(const BlockNormArgs &a, bool x_bf16, bool bf16, bool backward,
                              cudaStream_t st) {
    using bf = __nv_bfloat16;
    const bool v = vectors(a);
    if (x_bf16) return v ? launch_v<8, bf, bf>(a, backward, st) : launch_v<1, bf, bf>(a, backward, st);
    if (bf16) return v ? launch_v<8, float, bf>(a, backward, st) : launch_v<1, float, bf>(a, backward, st);
    return v ? launch_v<8, float, float>(a, backward, st) : launch_v<1, float, float>(a, backward, st);
}

}  // namespace kda
