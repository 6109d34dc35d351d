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

#include <type_traits>

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
    __device__ __forceinline__ void load_staged(const unsigned char *tile, int c) {   // V > 1
        const uint4 *p = reinterpret_cast<const uint4 *>(tile + (size_t)c * sizeof(T));
#pragma unroll
        for (int i = 0; i < (WORDS + 3) / 4; ++i) {
            const uint4 u = p[i];
            w[4 * i] = u.x;
            if constexpr (WORDS > 1) { w[4 * i + 1] = u.y; w[4 * i + 2] = u.z; w[4 * i + 3] = u.w; }
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

// Sums of x over the TPR threads of a row, the same bits in each: within a warp by shuffles,
// across warps through shared memory.  Every thread of the CTA takes part.  `red` is a slot of
// its own for each call between two barriers.
template <int TPR>
__device__ __forceinline__ float row_sum(float x, float *red) {
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) x += __shfl_xor_sync(0xffffffffu, x, m);
    constexpr int NW = TPR / 32;   // warps of a row
    if (NW > 1 && (threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = x;
    __syncthreads();
    if constexpr (NW > 1) {
        x = red[threadIdx.x / TPR * NW + (threadIdx.x & (NW - 1))];
#pragma unroll
        for (int m = NW / 2; m > 0; m >>= 1) x += __shfl_xor_sync(0xffffffffu, x, m);
    }
    return x;
}
// The same of two sums at once.
template <int TPR>
__device__ __forceinline__ float2 row_sum2(float x, float y, float2 *red) {
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) {
        x += __shfl_xor_sync(0xffffffffu, x, m);
        y += __shfl_xor_sync(0xffffffffu, y, m);
    }
    constexpr int NW = TPR / 32;
    if (NW > 1 && (threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = make_float2(x, y);
    __syncthreads();
    if constexpr (NW > 1) {
        const float2 v = red[threadIdx.x / TPR * NW + (threadIdx.x & (NW - 1))];
        x = v.x, y = v.y;
#pragma unroll
        for (int m = NW / 2; m > 0; m >>= 1) {
            x += __shfl_xor_sync(0xffffffffu, x, m);
            y += __shfl_xor_sync(0xffffffffu, y, m);
        }
    }
    return make_float2(x, y);
}

__device__ __forceinline__ float sigmoid(float x) { return __fdividef(1.f, 1.f + __expf(-x)); }


// The inputs of the rows that a CTA works on: NT / TPR rows side by side, TPR threads and NV
// vectors of V elements each.  STAGED: they come through a ring of `stages` row groups in
// shared memory, each filled by one bulk copy per tensor (the rows of a group are contiguous),
// so that as many bytes are in flight as the ring holds; a stage is filled again as soon as the
// first barrier after its reading has passed, each tensor's copy issued by a warp of its own.
// Otherwise (widths or addresses that are no multiple of 16 bytes, rows too wide for the ring)
// each thread loads its own elements.
template <int V, int NV, int TPR, int NT, bool BACK, bool STAGED, typename TX, typename T>
struct RowSource {
    static constexpr int RPC = NT / TPR;
    Pack<V, TX> x[NV], dx[BACK ? NV : 1];
    Pack<V, T> y[NV], g[NV], dh[BACK ? NV : 1];

    static __device__ __forceinline__ uint32_t stage_bytes(const BlockNormArgs &a) {
        return (uint32_t)RPC * a.width *
               ((BACK ? 2 : 1) * sizeof(TX) + ((BACK ? 2 : 1) + (a.gate ? 1 : 0)) * sizeof(T));
    }
    // What this thread copies for each group: lane 0 of warp w has tensor w of y, x, gate, dh,
    // dx_new (`bytes` per row, 0: none), and warp 0's also announces all tensors' bytes.
    struct Copier {
        const unsigned char *src;
        uint32_t bytes, offset, total;
    };
    static __device__ __forceinline__ Copier copier(const BlockNormArgs &a) {
        Copier c{nullptr, 0u, 0u, 0u};
        if (threadIdx.x & 31) return c;
        const int w = threadIdx.x >> 5;
        uint32_t offset = 0;
        auto tensor = [&](int i, const void *p, uint32_t el, bool room) {
            if (p) {
                if (i == w) c.src = (const unsigned char *)p, c.bytes = a.width * el, c.offset = offset;
                if (w == 0) c.total += a.width * el;
            }
            if (room) offset += RPC * a.width * el;
        };
        tensor(0, a.y, sizeof(T), true);
        tensor(1, a.x, sizeof(TX), true);
        tensor(2, a.gate, sizeof(T), a.gate != nullptr);
        if (BACK) {
            tensor(3, a.dh, sizeof(T), true);
            tensor(4, a.dx_new, sizeof(TX), true);
        }
        return c;
    }
    // the group of rows from `row` into the stage `dst` of barrier `bar`
    static __device__ __forceinline__ void issue(const BlockNormArgs &a, const Copier &c, int row,
                                                 uint32_t dst, uint64_t *bar) {
        if (c.bytes == 0 || row >= a.rows) return;
        const uint32_t n = min((int)a.rows - row, RPC);
        if (c.total) mbar_arrive_expect_tx(bar, n * c.total);
        asm volatile(
            "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::
                "r"(dst + c.offset), "l"(c.src + (int64_t)row * c.bytes), "r"(n * c.bytes), "r"(smem_u32(bar))
            : "memory");
    }
    // this thread's elements of its row of the group, from the stage `tile` if STAGED
    __device__ __forceinline__ void read(const BlockNormArgs &a, int row, const unsigned char *tile) {
        const int t = threadIdx.x % TPR, side = threadIdx.x / TPR;
        const bool live = row < a.rows;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * TPR + t) * V;
            y[i].zero(), x[i].zero(), g[i].zero();
            if (BACK) dh[i].zero(), dx[i].zero();
            if (!live || c >= a.width) continue;
            if constexpr (STAGED) {
                const unsigned char *p = tile;
                const int at = side * a.width + c;
                const uint32_t row_group = (uint32_t)RPC * a.width;
                y[i].load_staged(p, at);
                p += row_group * sizeof(T);
                x[i].load_staged(p, at);
                p += row_group * sizeof(TX);
                if (a.gate) {
                    g[i].load_staged(p, at);
                    p += row_group * sizeof(T);
                }
                if (BACK) {
                    if (a.dh) dh[i].load_staged(p, at);
                    p += row_group * sizeof(T);
                    if (a.dx_new) dx[i].load_staged(p, at);
                }
            } else {
                const int64_t at = (int64_t)row * a.width + c;
                y[i].load((const T *)a.y + at);
                x[i].load((const TX *)a.x + at);
                if (a.gate) g[i].load((const T *)a.gate + at);
                if (BACK) {
                    if (a.dh) dh[i].load((const T *)a.dh + at);
                    if (a.dx_new) dx[i].load((const TX *)a.dx_new + at);
                }
            }
        }
    }
};

template <int V, int NV, int TPR, int NT, int CTAS, bool STAGED, typename TX, typename T>
__global__ void __launch_bounds__(NT, CTAS) block_norm_kernel(BlockNormArgs a) {
    using Rows = RowSource<V, NV, TPR, NT, false, STAGED, TX, T>;
    extern __shared__ __align__(128) unsigned char ring[];
    __shared__ float red[2][2][NT / 32];
    __shared__ uint64_t bars[kBlockNormStages];
    __shared__ volatile uint32_t abort;
    const int t = threadIdx.x % TPR, side = threadIdx.x / TPR;
    const int D = a.width;
    const bool gated = a.gate != nullptr;
    const float inv_d = 1.f / D;
    const auto copier = Rows::copier(a);
    const int first = blockIdx.x * Rows::RPC, step = gridDim.x * Rows::RPC;   // rows of a group
    const uint32_t bytes = STAGED ? Rows::stage_bytes(a) : 0u, ring_at = smem_u32(ring);
    if (STAGED) {
        if (threadIdx.x == 0) {
            for (int i = 0; i < kBlockNormStages; ++i) mbar_init(bars + i, 1);
            mbar_fence_init();
            abort = 0u;
        }
        __syncthreads();
        for (int i = 0; i < a.stages; ++i)
            if (first + (int64_t)i * step < a.rows)
                Rows::issue(a, copier, first + i * step, ring_at + i * bytes, bars + i);
    }
    Pack<V, T> wo[NV], wi[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        wo[i].zero(), wi[i].zero();
        if ((i * TPR + t) * V < D) {
            wo[i].load_shared((const T *)a.w_post + (i * TPR + t) * V);
            wi[i].load_shared((const T *)a.w_pre + (i * TPR + t) * V);
        }
    }
    int stage = 0, turn = 0;
    uint32_t parity = 0;
    for (int64_t base = first; base < a.rows; base += step, turn ^= 1) {
        Rows in;
        const int row = (int)base + side;
        const int64_t at = (int64_t)row * D;
        if (STAGED && !mbar_wait_abortable(bars + stage, parity, a.err, a.epoch, &abort)) return;
        in.read(a, row, ring + stage * bytes);
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j) ss = fmaf(in.y[i].get(j), in.y[i].get(j), ss);
        const float ry = rsqrtf(row_sum<TPR>(ss, red[turn][0]) * inv_d + a.eps) * a.scale;
        if (STAGED) {
            if (base + (int64_t)a.stages * step < a.rows)
                Rows::issue(a, copier, (int)base + a.stages * step, ring_at + stage * bytes, bars + stage);
            if (++stage == a.stages) stage = 0, parity ^= 1u;
        }
        float xn[NV][V];
        ss = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * TPR + t) * V;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float s = gated ? sigmoid(in.g[i].get(j)) : 1.f;
                xn[i][j] = fmaf(in.y[i].get(j) * ry * wo[i].get(j), s, in.x[i].get(j));
                ss = fmaf(xn[i][j], xn[i][j], ss);
            }
            if (row < a.rows && c < D) store<V>((TX *)a.x_new + at + c, xn[i]);
        }
        const float rx = rsqrtf(row_sum<TPR>(ss, red[turn][1]) * inv_d + a.eps);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * TPR + t) * V;
            float h[V];
#pragma unroll
            for (int j = 0; j < V; ++j) h[j] = xn[i][j] * rx * wi[i].get(j);
            if (row < a.rows && c < D) store<V>((T *)a.h + at + c, h);
        }
    }
}

// The sums of the weight gradients over a CTA's rows go to part[cta RPC + side][2][D].
template <int V, int NV, int TPR, int NT, int CTAS, bool STAGED, typename TX, typename T>
__global__ void __launch_bounds__(NT, CTAS) block_norm_backward_kernel(BlockNormArgs a) {
    using Rows = RowSource<V, NV, TPR, NT, true, STAGED, TX, T>;
    extern __shared__ __align__(128) unsigned char ring[];
    __shared__ float red[2][2][NT / 32];
    __shared__ float2 red2[2][NT / 32];
    __shared__ uint64_t bars[kBlockNormStages];
    __shared__ volatile uint32_t abort;
    const int t = threadIdx.x % TPR, side = threadIdx.x / TPR;
    const int D = a.width;
    const bool gated = a.gate != nullptr;
    const float inv_d = 1.f / D;
    const auto copier = Rows::copier(a);
    const int first = blockIdx.x * Rows::RPC, step = gridDim.x * Rows::RPC;   // rows of a group
    const uint32_t bytes = STAGED ? Rows::stage_bytes(a) : 0u, ring_at = smem_u32(ring);
    if (STAGED) {
        if (threadIdx.x == 0) {
            for (int i = 0; i < kBlockNormStages; ++i) mbar_init(bars + i, 1);
            mbar_fence_init();
            abort = 0u;
        }
        __syncthreads();
        for (int i = 0; i < a.stages; ++i)
            if (first + (int64_t)i * step < a.rows)
                Rows::issue(a, copier, first + i * step, ring_at + i * bytes, bars + i);
    }
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
    int stage = 0, turn = 0;
    uint32_t parity = 0;
    for (int64_t base = first; base < a.rows; base += step, turn ^= 1) {
        Rows in;
        const int row = (int)base + side;
        const int64_t at = (int64_t)row * D;
        if (STAGED && !mbar_wait_abortable(bars + stage, parity, a.err, a.epoch, &abort)) return;
        in.read(a, row, ring + stage * bytes);
        const bool live = row < a.rows;
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j) ss = fmaf(in.y[i].get(j), in.y[i].get(j), ss);
        const float ry = rsqrtf(row_sum<TPR>(ss, red[turn][0]) * inv_d + a.eps);
        if (STAGED) {
            if (base + (int64_t)a.stages * step < a.rows)
                Rows::issue(a, copier, (int)base + a.stages * step, ring_at + stage * bytes, bars + stage);
            if (++stage == a.stages) stage = 0, parity ^= 1u;
        }
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
        const float2 two = row_sum2<TPR>(sx, sg, red2[turn]);
        const float rx = rsqrtf(two.x * inv_d + a.eps), kx = rx * rx * rx * (two.y * inv_d);
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
            if (live && c < D) {
                store<V>((TX *)a.dx + at + c, dx);
                if (gated) store<V>((T *)a.dgate + at + c, dg);
            }
        }
        const float ky = ry * ry * ry * (row_sum<TPR>(sy, red[turn][1]) * inv_d);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * TPR + t) * V;
            float d[V];
#pragma unroll
            for (int j = 0; j < V; ++j) d[j] = fmaf(ry, gy[i][j], -ky * in.y[i].get(j));
            if (live && c < D) store<V>((T *)a.dy + at + c, d);
        }
    }
    float *part = a.part + ((int64_t)blockIdx.x * Rows::RPC + side) * 2 * D;
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

// Column sums of part[parts][2 D] in a fixed order: 32 columns and 32 groups of rows per CTA.
__global__ void __launch_bounds__(1024) block_norm_weights_kernel(const float *part, int parts,
                                                                  int D, float *dw_post,
                                                                  float *dw_pre) {
    __shared__ float red[32][33];
    const int col = blockIdx.x * 32 + (threadIdx.x & 31), group = threadIdx.x >> 5;
    float s = 0.f;
    if (col < 2 * D)
#pragma unroll 4
        for (int i = group; i < parts; i += 32) s += part[(int64_t)i * 2 * D + col];
    red[group][threadIdx.x & 31] = s;
    __syncthreads();
    if (group == 0 && col < 2 * D) {
        s = 0.f;
#pragma unroll
        for (int g = 0; g < 32; ++g) s += red[g][threadIdx.x];
        (col < D ? dw_post[col] : dw_pre[col - D]) = s;
    }
}

constexpr int kSMs = 148;
constexpr size_t kRingBytes = 200 * 1024;   // of an SM, shared by its CTAs

// Row groups of `rpc` rows over the SMs, `ctas` on each.
int64_t grid_of(int64_t rows, int rpc, int ctas) {
    const int64_t all = (rows + rpc - 1) / rpc;
    return all < ctas * kSMs ? all : ctas * kSMs;
}

template <int V, int NV, int TPR, int NT, int CTAS, bool BACK, bool STAGED, typename TX, typename T>
cudaError_t launch_s(const BlockNormArgs &a, size_t smem, cudaStream_t st) {
    constexpr int RPC = NT / TPR;
    const int64_t grid = grid_of(a.rows, RPC, CTAS);
    const auto kernel = [] {
        if constexpr (BACK) return block_norm_backward_kernel<V, NV, TPR, NT, CTAS, STAGED, TX, T>;
        else return block_norm_kernel<V, NV, TPR, NT, CTAS, STAGED, TX, T>;
    }();
    if (grid > 0) {
        if (STAGED) {
            const cudaError_t e = cudaFuncSetAttribute(
                kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)(kRingBytes / CTAS));
            if (e != cudaSuccess) return e;
        }
        kernel<<<(unsigned)grid, NT, smem, st>>>(a);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
        Profiler::mark(st);
    }
    if (!BACK) return cudaSuccess;
    block_norm_weights_kernel<<<(2 * a.width + 31) / 32, 1024, 0, st>>>(a.part, (int)grid * RPC, a.width,
                                                                       a.dw_post, a.dw_pre);
    const cudaError_t e = cudaGetLastError();
    Profiler::mark(st);
    return e;
}

// The ring takes as many stages as fit, two at least.
template <int V, int NV, int TPR, int NT, int CTAS, bool BACK, typename TX, typename T>
cudaError_t launch_t(BlockNormArgs a, cudaStream_t st) {
    if constexpr (V == 8) {
        const size_t stage = (size_t)(NT / TPR) * a.width *
                             ((BACK ? 2 : 1) * sizeof(TX) + ((BACK ? 2 : 1) + (a.gate ? 1 : 0)) * sizeof(T));
        const size_t fit = kRingBytes / CTAS / stage;
        a.stages = (int)(fit < (size_t)kBlockNormStages ? fit : (size_t)kBlockNormStages);
        if (a.stages >= 2)
            return launch_s<V, NV, TPR, NT, CTAS, BACK, true, TX, T>(a, a.stages * stage, st);
    }
    return launch_s<V, NV, TPR, NT, CTAS, BACK, false, TX, T>(a, 0, st);
}

// CTAs of FNT / BNT threads and as many to an SM as their registers allow, so that one CTA's
// barriers are hidden behind another's work.  Rows up to that many vectors take the next power
// of two of threads, wider ones a CTA of 512 threads with several vectors each.
constexpr int FNT = 512, FC = 2, BNT = 512, BC = 1;

template <int V, bool BACK, typename TX, typename T>
cudaError_t launch_v(const BlockNormArgs &a, cudaStream_t st) {
    constexpr int NT = BACK ? BNT : FNT, CTAS = BACK ? BC : FC;
    const int vecs = (a.width + V - 1) / V;
    if (vecs <= 32) return launch_t<V, 1, 32, NT, CTAS, BACK, TX, T>(a, st);
    if (vecs <= 64) return launch_t<V, 1, 64, NT, CTAS, BACK, TX, T>(a, st);
    if (vecs <= 128) return launch_t<V, 1, 128, NT, CTAS, BACK, TX, T>(a, st);
    if (vecs <= 256) return launch_t<V, 1, 256, NT, CTAS, BACK, TX, T>(a, st);
    if (vecs <= 512) return launch_t<V, 1, 512, NT, CTAS, BACK, TX, T>(a, st);
    if (vecs <= 1024) return launch_t<V, 2, 512, 512, 1, BACK, TX, T>(a, st);
    if constexpr (V == 8) {
        return launch_t<V, 4, 512, 512, 1, BACK, TX, T>(a, st);
    } else {
        if (vecs <= 4096) return launch_t<V, 8, 512, 512, 1, BACK, TX, T>(a, st);
        return launch_t<V, 32, 512, 512, 1, BACK, TX, T>(a, st);
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
    // rows side by side in a CTA, for one and for eight elements a vector: the larger number
    size_t most = 0;
    for (int v : {1, 8}) {
        const int vecs = (width + v - 1) / v;
        int tpr = 32;
        while (tpr < BNT && tpr < vecs) tpr *= 2;
        const size_t parts = (size_t)grid_of(rows, BNT / tpr, BC) * (BNT / tpr);
        if (parts > most) most = parts;
    }
    return most;
}

cudaError_t launch_block_norm(const BlockNormArgs &a, bool x_bf16, bool bf16, bool backward,
                              cudaStream_t st) {
    using bf = __nv_bfloat16;
    auto types = [&](auto back) {
        constexpr bool B = decltype(back)::value;
        const bool v = vectors(a);
        if (x_bf16) return v ? launch_v<8, B, bf, bf>(a, st) : launch_v<1, B, bf, bf>(a, st);
        if (bf16) return v ? launch_v<8, B, float, bf>(a, st) : launch_v<1, B, float, bf>(a, st);
        return v ? launch_v<8, B, float, float>(a, st) : launch_v<1, B, float, float>(a, st);
    };
    return backward ? types(std::true_type{}) : types(std::false_type{});
}

}  // namespace kda
