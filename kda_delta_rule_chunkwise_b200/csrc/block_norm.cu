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

template <int V> struct Floats { float v[V]; };

template <int V, typename T>
__device__ __forceinline__ Floats<V> load(const T *p) {
    Floats<V> r;
    if constexpr (V == 1) {
        r.v[0] = to_f32(*p);
    } else if constexpr (sizeof(T) == 2) {
        const uint4 w = *reinterpret_cast<const uint4 *>(p);
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            r.v[2 * i] = __uint_as_float(u[i] << 16);
            r.v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float4 w = reinterpret_cast<const float4 *>(p)[i];
            r.v[4 * i] = w.x; r.v[4 * i + 1] = w.y; r.v[4 * i + 2] = w.z; r.v[4 * i + 3] = w.w;
        }
    }
    return r;
}

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
        *reinterpret_cast<uint4 *>(p) = make_uint4(u[0], u[1], u[2], u[3]);
    } else {
#pragma unroll
        for (int i = 0; i < 2; ++i)
            reinterpret_cast<float4 *>(p)[i] =
                make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
    }
}

// Sum over the TPR threads of a row, the same bits in each: within a warp by shuffles,
// across warps through shared memory (then the CTA is one row).  `red` is a slot of its own
// for each call between two barriers.
template <int TPR>
__device__ __forceinline__ float row_sum(float x, float *red) {
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) x += __shfl_xor_sync(0xffffffffu, x, m);
    if constexpr (TPR > 32) {
        if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = x;
        __syncthreads();
        x = 0.f;
#pragma unroll
        for (int w = 0; w < TPR / 32; ++w) x += red[w];
    }
    return x;
}

__device__ __forceinline__ float sigmoid(float x) { return 1.f / (1.f + expf(-x)); }

// V elements per vector, NV vectors per thread, TPR threads per row.
template <int V, int NV, int TPR, typename TX, typename T>
__global__ void __launch_bounds__(TPR > 256 ? TPR : 256) block_norm_kernel(BlockNormArgs a) {
    constexpr int RPC = TPR > 32 ? 1 : 8;   // rows per CTA
    __shared__ float red[2][TPR / 32];
    const int t = threadIdx.x % TPR;
    const int64_t row = (int64_t)blockIdx.x * RPC + threadIdx.x / TPR;
    if (RPC > 1 && row >= a.rows) return;   // a whole warp
    const int D = a.width;
    const TX *x = (const TX *)a.x + row * D;
    const T *y = (const T *)a.y + row * D, *gate = (const T *)a.gate;
    if (gate) gate += row * D;

    Floats<V> xv[NV], yv[NV], gv[NV];
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * TPR + t) * V;
        if (c < D) {
            yv[i] = load<V>(y + c);
            xv[i] = load<V>(x + c);
            if (gate) gv[i] = load<V>(gate + c);
        }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i)
        if ((i * TPR + t) * V < D)
#pragma unroll
            for (int j = 0; j < V; ++j) ss = fmaf(yv[i].v[j], yv[i].v[j], ss);
    const float ry = rsqrtf(row_sum<TPR>(ss, red[0]) / D + a.eps) * a.scale;
    ss = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * TPR + t) * V;
        if (c >= D) continue;
        const Floats<V> w = load<V>((const T *)a.w_post + c);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const float g = gate ? sigmoid(gv[i].v[j]) : 1.f;
            xv[i].v[j] = fmaf(yv[i].v[j] * ry * w.v[j], g, xv[i].v[j]);
            ss = fmaf(xv[i].v[j], xv[i].v[j], ss);
        }
        store<V>((TX *)a.x_new + row * D + c, xv[i].v);
    }
    const float rx = rsqrtf(row_sum<TPR>(ss, red[1]) / D + a.eps);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * TPR + t) * V;
        if (c >= D) continue;
        const Floats<V> w = load<V>((const T *)a.w_pre + c);
        float h[V];
#pragma unroll
        for (int j = 0; j < V; ++j) h[j] = xv[i].v[j] * rx * w.v[j];
        store<V>((T *)a.h + row * D + c, h);
    }
}

// A CTA walks rows blockIdx.x RPC + k gridDim.x RPC; its sums of the weight gradients go to
// part[cta][2][D] (with several rows side by side, to part[cta * RPC + side]).
template <int V, int NV, int TPR, typename TX, typename T>
__global__ void __launch_bounds__(TPR > 256 ? TPR : 256) block_norm_backward_kernel(BlockNormArgs a) {
    constexpr int RPC = TPR > 32 ? 1 : 8;
    __shared__ float red[2][4][TPR / 32];
    const int t = threadIdx.x % TPR, side = threadIdx.x / TPR;
    const int D = a.width;
    const T *gate = (const T *)a.gate;
    const float inv_d = 1.f / D;
    float wo[NV][V], wi[NV][V];
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) wo[i][j] = wi[i][j] = 0.f;
    int turn = 0;
    for (int64_t row = (int64_t)blockIdx.x * RPC + side; row < a.rows;
         row += (int64_t)gridDim.x * RPC, turn ^= 1) {
        const int64_t at = row * D;
        Floats<V> xv[NV], yv[NV], gv[NV], hv[NV], dv[NV];
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * TPR + t) * V;
            if (c >= D) continue;
            yv[i] = load<V>((const T *)a.y + at + c);
            xv[i] = load<V>((const TX *)a.x + at + c);
            if (gate) gv[i] = load<V>(gate + at + c);
            if (a.dh) hv[i] = load<V>((const T *)a.dh + at + c);
            if (a.dx_new) dv[i] = load<V>((const TX *)a.dx_new + at + c);
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if ((i * TPR + t) * V >= D) continue;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                gv[i].v[j] = gate ? sigmoid(gv[i].v[j]) : 1.f;
                if (!a.dh) hv[i].v[j] = 0.f;
                if (!a.dx_new) dv[i].v[j] = 0.f;
                ss = fmaf(yv[i].v[j], yv[i].v[j], ss);
            }
        }
        const float ry = rsqrtf(row_sum<TPR>(ss, red[turn][0]) / D + a.eps);
        // x' in place of x; the two sums of the second norm
        float sx = 0.f, sg = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * TPR + t) * V;
            if (c >= D) continue;
            const Floats<V> w = load<V>((const T *)a.w_post + c), u = load<V>((const T *)a.w_pre + c);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float s = a.scale * gv[i].v[j];
                xv[i].v[j] = fmaf(yv[i].v[j] * ry * w.v[j], s, xv[i].v[j]);
                sx = fmaf(xv[i].v[j], xv[i].v[j], sx);
                sg = fmaf(hv[i].v[j] * u.v[j], xv[i].v[j], sg);
            }
        }
        sx = row_sum<TPR>(sx, red[turn][1]);
        sg = row_sum<TPR>(sg, red[turn][2]);
        const float rx = rsqrtf(sx / D + a.eps), kx = rx * rx * rx * (sg * inv_d);
        float sy = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * TPR + t) * V;
            if (c >= D) continue;
            const Floats<V> w = load<V>((const T *)a.w_post + c), u = load<V>((const T *)a.w_pre + c);
            float dg[V];
#pragma unroll
            for (int j = 0; j < V; ++j) {
                wi[i][j] = fmaf(hv[i].v[j], xv[i].v[j] * rx, wi[i][j]);
                const float d = dv[i].v[j] + rx * (hv[i].v[j] * u.v[j]) - kx * xv[i].v[j];
                dv[i].v[j] = d;                              // dx
                const float s = a.scale * d, yn = yv[i].v[j] * ry, g = gv[i].v[j];
                const float dn = s * g;
                dg[j] = dn * (1.f - g) * (yn * w.v[j]);
                wo[i][j] = fmaf(dn, yn, wo[i][j]);
                hv[i].v[j] = dn * w.v[j];                    // gy
                sy = fmaf(hv[i].v[j], yv[i].v[j], sy);
            }
            store<V>((TX *)a.dx + at + c, dv[i].v);
            if (gate) store<V>((T *)a.dgate + at + c, dg);
        }
        sy = row_sum<TPR>(sy, red[turn][3]);
        const float ky = ry * ry * ry * (sy * inv_d);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * TPR + t) * V;
            if (c >= D) continue;
            float d[V];
#pragma unroll
            for (int j = 0; j < V; ++j) d[j] = fmaf(ry, hv[i].v[j], -ky * yv[i].v[j]);
            store<V>((T *)a.dy + at + c, d);
        }
    }
    float *part = a.part + ((int64_t)blockIdx.x * RPC + side) * 2 * D;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * TPR + t) * V;
        if (c >= D) continue;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            part[c + j] = wo[i][j];
            part[D + c + j] = wi[i][j];
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

// Threads per row: two vectors a thread from 512 vectors on, one below (a row's latency then
// counts more than the number of its threads).
template <int V, typename TX, typename T>
cudaError_t launch_v(const BlockNormArgs &a, bool b, cudaStream_t st) {
    const int vecs = (a.width + V - 1) / V;
    if (vecs <= 32) return launch_t<V, 1, 32, TX, T>(a, b, st);
    if (vecs <= 64) return launch_t<V, 1, 64, TX, T>(a, b, st);
    if (vecs <= 128) return launch_t<V, 1, 128, TX, T>(a, b, st);
    if (vecs <= 256) return launch_t<V, 1, 256, TX, T>(a, b, st);
    if (vecs <= 512) return launch_t<V, 2, 256, TX, T>(a, b, st);
    if (vecs <= 1024) return launch_t<V, 2, 512, TX, T>(a, b, st);
    if constexpr (V == 8) {
        return launch_t<V, 2, 1024, TX, T>(a, b, st);
    } else {
        if (vecs <= 4096) return launch_t<V, 8, 512, TX, T>(a, b, st);
        return launch_t<V, 16, 1024, TX, T>(a, b, st);
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
