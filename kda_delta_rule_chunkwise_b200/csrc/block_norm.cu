// Block norm: what closes one block of a model and opens the next, in one pass.
//
//     n  = y rsqrt(mean y^2 + eps) w_post          norm after the block
//     x' = x + scale sigmoid(gate) n               gate, scaled residual sum
//     h  = x' rsqrt(mean x'^2 + eps) w_pre         norm before the next block
//
// Every input is read once and every output written once.  All arithmetic is fp32; h is taken from
// the unrounded x'.  Up to a width of 4096 a row's values stay in registers between the row sums; 8192
// rows of 4096, bf16: forward 63 us for 336 MB (5.3 TB/s, 82 % of a plain copy); backward 133 us for
// 537 MB (62 %), bound by the latency of its three row sums and by instruction issue (51 % of cycles).
// Wider rows, several vectors to a thread, do not all fit: the backward spills about 300 bytes a thread
// up to 8192 and 1.1 KB beyond, the forward some beyond 8192 (8192 rows of 5120 and of 8192, bf16: forward
// 100 and 106 us, 65 and 98 % of a plain copy's speed; backward 331 and 367 us, 31 and 45 %; 4096 rows of
// 16384: 135 us, 77 %, and 930 us, 18 %).
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

// Eight consecutive elements as loaded: 16 bytes of bf16 or 32 of fp32.  They stay packed in
// registers and are widened where they are used.
template <int V, typename T>
struct Pack {
    static_assert(V == 8, "vectors of eight");
    static constexpr int WORDS = V * (int)sizeof(T) / 4;
    uint32_t w[WORDS];
    __device__ __forceinline__ void take(int i, const uint4 &u) {
        w[4 * i] = u.x; w[4 * i + 1] = u.y; w[4 * i + 2] = u.z; w[4 * i + 3] = u.w;
    }
    __device__ __forceinline__ void load(const T *p) {
#pragma unroll
        for (int i = 0; i < WORDS / 4; ++i) take(i, __ldcs(reinterpret_cast<const uint4 *>(p) + i));
    }
    __device__ __forceinline__ void load_shared(const T *p) {   // weights: read by every row
#pragma unroll
        for (int i = 0; i < WORDS / 4; ++i) take(i, __ldg(reinterpret_cast<const uint4 *>(p) + i));
    }
    __device__ __forceinline__ void load_staged(const unsigned char *tile, int c) {
        const uint4 *p = reinterpret_cast<const uint4 *>(tile + (size_t)c * sizeof(T));
#pragma unroll
        for (int i = 0; i < WORDS / 4; ++i) take(i, p[i]);
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < WORDS; ++i) w[i] = 0u;
    }
    __device__ __forceinline__ float get(int j) const {
        if constexpr (sizeof(T) == 4) return __uint_as_float(w[j]);
        else return __uint_as_float((j & 1) ? w[j / 2] & 0xffff0000u : w[j / 2] << 16);
    }
};

template <int V, typename T>
__device__ __forceinline__ void store(T *p, const float (&x)[V]) {
    if constexpr (sizeof(T) == 2) {
        uint32_t u[V / 2];
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
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

constexpr double kLog2eExact = 1.44269504088896340736;
constexpr float kLog2e = (float)kLog2eExact, kLog2eLow = (float)(kLog2eExact - (double)kLog2e);

// r^2 mean of a norm's gradient r (z - u r^2 mean(z u)), factor by factor: r mean is of z's size, while r^2
// and r^3 alone leave the range of fp32 beside a small eps or with large rows (a row of zeros would be 0 inf).
__device__ __forceinline__ float mean_term(float mean, float r) { return mean * r * r; }

// The gate of logits of type T.  Beside bf16 values the fast exponential, whose error of 2^-24 |x| and two
// steps is far below a rounding to bf16.  fp32 gets 2^(-x log2 e) with the product's rounding error recovered by
// a fused multiply-add (Dekker's exact product) and log2 e in two terms: a few steps of 2^-24 for any x; and the
// fast quotient (two steps).  8192 x 4096 in fp32: forward 119 us, backward 217; with the fast exponential 112
// and 207, with expf and a rounded quotient 127 and 231.
template <typename T>
__device__ __forceinline__ float sigmoid(float x) {
    if constexpr (sizeof(T) == 2) return __fdividef(1.f, 1.f + __expf(-x));
    asm("max.NaN.f32 %0, %0, 0fC3160000;" : "+f"(x));   // to [-150, 150], where nothing is left to tell;
    asm("min.NaN.f32 %0, %0, 0f43160000;" : "+f"(x));   // a NaN stays
    const float t = x * -kLog2e, low = fmaf(x, -kLog2eLow, fmaf(x, -kLog2e, -t));
    float e;
    asm("ex2.approx.f32 %0, %1;" : "=f"(e) : "f"(t));
    return __fdividef(1.f, 1.f + e * fmaf(low, 0.6931471805599453f, 1.f));
}


// The inputs of the rows that a CTA works on: NT / TPR rows side by side, TPR threads and NV
// vectors of V elements each.  STAGED: they come through a ring of `stages` row groups in
// shared memory, each filled by one bulk copy per tensor (the rows of a group are contiguous),
// so that as many bytes are in flight as the ring holds; a stage is filled again as soon as the
// first barrier after its reading has passed, each tensor's copy issued by a warp of its own.
// Otherwise (rows too wide for the ring) each thread loads its own elements.
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
    // Waits, with a bound, for the groups from row `base` on that are on their way to the ring: a CTA that
    // gives up leaves only then.  `stage`, `parity`: of group `base`.
    static __device__ __forceinline__ void drain(const BlockNormArgs &a, int64_t base, int step, int stage,
                                                 uint32_t parity, uint64_t *bars) {
#pragma unroll 1
        for (int i = 0; i < a.stages && base + (int64_t)i * step < a.rows; ++i) {
            if (!mbar_wait(bars + stage, parity, a.err)) break;
            if (++stage == a.stages) stage = 0, parity ^= 1u;
        }
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
        if (STAGED) mbar_wait_abortable(bars + stage, parity, a.err, a.epoch, &abort);   // raises `abort`
        in.read(a, row, ring + stage * bytes);
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j) ss = fmaf(in.y[i].get(j), in.y[i].get(j), ss);
        const float ry = rsqrtf(row_sum<TPR>(ss, red[turn][0]) * inv_d + a.eps) * a.scale;
        if (STAGED) {
            if (abort) {   // the same for all threads between the row sums' barriers
                Rows::drain(a, base, step, stage, parity, bars);
                return;
            }
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
                const float s = gated ? sigmoid<T>(in.g[i].get(j)) : 1.f;
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
        if (STAGED) mbar_wait_abortable(bars + stage, parity, a.err, a.epoch, &abort);   // raises `abort`
        in.read(a, row, ring + stage * bytes);
        const bool live = row < a.rows;
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j) ss = fmaf(in.y[i].get(j), in.y[i].get(j), ss);
        const float ry = rsqrtf(row_sum<TPR>(ss, red[turn][0]) * inv_d + a.eps);
        if (STAGED) {
            if (abort) {   // the same for all threads between the row sums' barriers
                Rows::drain(a, base, step, stage, parity, bars);
                return;
            }
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
                s[i][j] = gated ? sigmoid<T>(in.g[i].get(j)) : 1.f;
                xn[i][j] = fmaf(in.y[i].get(j) * ry * wo[i].get(j), a.scale * s[i][j], in.x[i].get(j));
                sx = fmaf(xn[i][j], xn[i][j], sx);
                sg = fmaf(in.dh[i].get(j) * wi[i].get(j), xn[i][j], sg);
            }
        const float2 two = row_sum2<TPR>(sx, sg, red2[turn]);
        const float rx = rsqrtf(two.x * inv_d + a.eps), kx = mean_term(two.y * inv_d, rx);
        float gy[NV][V], sy = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * TPR + t) * V;
            float dx[V], dg[V];
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float h = in.dh[i].get(j), yn = in.y[i].get(j) * ry;
                dwi[i][j] = fmaf(h, xn[i][j] * rx, dwi[i][j]);
                dx[j] = fmaf(rx, fmaf(-kx, xn[i][j], h * wi[i].get(j)), in.dx[i].get(j));
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
        const float ky = mean_term(row_sum<TPR>(sy, red[turn][1]) * inv_d, ry);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * TPR + t) * V;
            float d[V];
#pragma unroll
            for (int j = 0; j < V; ++j) d[j] = ry * fmaf(-ky, in.y[i].get(j), gy[i][j]);
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

// Widths and addresses that are no multiple of 16 bytes: V = 1 or 2 elements at a time.  STASH: a row's
// values are kept in shared memory as fp32, each thread its own columns, so that global memory is read
// once and with all of a row's loads in flight; rows too wide for that are read again from the cache in
// each pass.  Everything is written in the last pass, each element by the thread that has read it, so
// outputs may lie on inputs here too.
template <int V, typename T>
__device__ __forceinline__ void fetch(float (&x)[V], const T *p) {
    if constexpr (V == 1) {
        x[0] = to_f32(*p);
    } else if constexpr (sizeof(T) == 2) {
        const uint32_t u = *reinterpret_cast<const uint32_t *>(p);
        x[0] = __uint_as_float(u << 16), x[1] = __uint_as_float(u & 0xffff0000u);
    } else {
        const float2 u = *reinterpret_cast<const float2 *>(p);
        x[0] = u.x, x[1] = u.y;
    }
}
template <int V, typename T>
__device__ __forceinline__ void put(T *p, const float (&x)[V]) {
    if constexpr (V == 1) *p = from_f32<T>(x[0]);
    else if constexpr (sizeof(T) == 2) *reinterpret_cast<__nv_bfloat162 *>(p) = __floats2bfloat162_rn(x[0], x[1]);
    else *reinterpret_cast<float2 *>(p) = make_float2(x[0], x[1]);
}

constexpr int kAnyThreads = 512, kAnyBackward = 3;   // CTAs per SM of the backward, if their sums fit

// fp32 values per row and column in shared memory: x', y, sigmoid(gate), and for the backward dh, dx and
// the sums of the two weights' gradients.
constexpr int any_floats(bool back, bool stash) { return (back ? 2 : 0) + (stash ? (back ? 5 : 3) : 0); }

template <int V, int TPR, bool BACK, bool STASH, typename TX, typename T>
__global__ void __launch_bounds__(kAnyThreads) block_norm_any_kernel(BlockNormArgs a) {
    constexpr int RPC = kAnyThreads / TPR;
    extern __shared__ __align__(16) float store_[];   // [RPC][any_floats][D], each thread its own columns
    __shared__ float red[2][2][kAnyThreads / 32];
    __shared__ float2 red2[2][kAnyThreads / 32];
    const int t = (threadIdx.x % TPR) * V, side = threadIdx.x / TPR, D = a.width;
    const float inv_d = 1.f / D;
    const T *wo = (const T *)a.w_post, *wi = (const T *)a.w_pre;
    float *dwo = store_ + side * any_floats(BACK, STASH) * D, *dwi = dwo + D;
    float *kx_ = dwo + (BACK ? 2 * D : 0), *ky_ = kx_ + D, *ks_ = ky_ + D, *kh_ = ks_ + D, *kd_ = kh_ + D;
    if (BACK)
        for (int c = t; c < D; c += TPR * V)
            for (int j = 0; j < V; ++j) dwo[c + j] = dwi[c + j] = 0.f;
    int turn = 0;
    for (int64_t base = (int64_t)blockIdx.x * RPC; base < a.rows; base += (int64_t)gridDim.x * RPC, turn ^= 1) {
        const int64_t row = base + side, at = row * D;
        const int end = row < a.rows ? D : 0;
        const TX *x = (const TX *)a.x + at, *dxn = a.dx_new ? (const TX *)a.dx_new + at : nullptr;
        const T *y = (const T *)a.y + at, *gate = a.gate ? (const T *)a.gate + at : nullptr;
        const T *dh = a.dh ? (const T *)a.dh + at : nullptr;
        // this thread's inputs at column c, as loaded: zeros for what is missing
        auto inputs = [&](int c, float (&xv)[V], float (&yv)[V], float (&s)[V], float (&h)[V], float (&d)[V]) {
            fetch<V>(yv, y + c);
            fetch<V>(xv, x + c);
            if (gate) fetch<V>(s, gate + c);
            if (BACK && dh) fetch<V>(h, dh + c);
            if (BACK && dxn) fetch<V>(d, dxn + c);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                s[j] = gate ? sigmoid<T>(s[j]) : 1.f;
                if (!(BACK && dh)) h[j] = 0.f;
                if (!(BACK && dxn)) d[j] = 0.f;
            }
        };
        float ss = 0.f;
#pragma unroll 4
        for (int c = t; c < end; c += TPR * V) {
            float xv[V], yv[V], s[V], h[V], d[V];
            if (STASH) {
                inputs(c, xv, yv, s, h, d);
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    kx_[c + j] = xv[j], ky_[c + j] = yv[j], ks_[c + j] = s[j];
                    if (BACK) kh_[c + j] = h[j], kd_[c + j] = d[j];
                }
            } else {
                fetch<V>(yv, y + c);
            }
#pragma unroll
            for (int j = 0; j < V; ++j) ss = fmaf(yv[j], yv[j], ss);
        }
        const float ry = rsqrtf(row_sum<TPR>(ss, red[turn][0]) * inv_d + a.eps);
        // x' (in place of x) and the rest at column c; FIRST: x' is not there yet
        auto joined = [&](auto first, int c, float (&xn)[V], float (&yv)[V], float (&s)[V], float (&h)[V],
                          float (&d)[V], float (&w)[V]) {
            constexpr bool FIRST = decltype(first)::value;
            fetch<V>(w, wo + c);
            if (STASH) {
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    xn[j] = kx_[c + j], yv[j] = ky_[c + j], s[j] = ks_[c + j];
                    h[j] = BACK ? kh_[c + j] : 0.f, d[j] = BACK ? kd_[c + j] : 0.f;
                }
            } else {
                inputs(c, xn, yv, s, h, d);
            }
            if (FIRST || !STASH)
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    xn[j] = fmaf(yv[j] * ry * w[j], a.scale * s[j], xn[j]);
                    if (STASH) kx_[c + j] = xn[j];
                }
        };
        using First = std::true_type;
        using Later = std::false_type;
        float sx = 0.f, sg = 0.f;
#pragma unroll 2
        for (int c = t; c < end; c += TPR * V) {
            float xn[V], yv[V], s[V], h[V], d[V], w[V], u[V];
            joined(First{}, c, xn, yv, s, h, d, w);
            if (BACK) fetch<V>(u, wi + c);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                sx = fmaf(xn[j], xn[j], sx);
                if (BACK) sg = fmaf(h[j] * u[j], xn[j], sg);
            }
        }
        if (!BACK) {
            const float rx = rsqrtf(row_sum<TPR>(sx, red[turn][1]) * inv_d + a.eps);
#pragma unroll 2
            for (int c = t; c < end; c += TPR * V) {
                float xn[V], yv[V], s[V], h[V], d[V], w[V], u[V];
                joined(Later{}, c, xn, yv, s, h, d, w);
                fetch<V>(u, wi + c);
                put<V>((TX *)a.x_new + at + c, xn);
#pragma unroll
                for (int j = 0; j < V; ++j) u[j] *= xn[j] * rx;
                put<V>((T *)a.h + at + c, u);
            }
            continue;
        }
        const float2 two = row_sum2<TPR>(sx, sg, red2[turn]);
        const float rx = rsqrtf(two.x * inv_d + a.eps), kx = mean_term(two.y * inv_d, rx);
        float sy = 0.f;
#pragma unroll 2
        for (int c = t; c < end; c += TPR * V) {
            float xn[V], yv[V], s[V], h[V], d[V], w[V], u[V];
            joined(Later{}, c, xn, yv, s, h, d, w);
            fetch<V>(u, wi + c);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float dx = fmaf(rx, fmaf(-kx, xn[j], h[j] * u[j]), d[j]), dn = a.scale * dx * s[j];
                dwi[c + j] = fmaf(h[j], xn[j] * rx, dwi[c + j]);
                dwo[c + j] = fmaf(dn, yv[j] * ry, dwo[c + j]);
                sy = fmaf(dn * w[j], yv[j], sy);
            }
        }
        const float ky = mean_term(row_sum<TPR>(sy, red[turn][1]) * inv_d, ry);
#pragma unroll 2
        for (int c = t; c < end; c += TPR * V) {
            float xn[V], yv[V], s[V], h[V], d[V], w[V], u[V];
            joined(Later{}, c, xn, yv, s, h, d, w);
            fetch<V>(u, wi + c);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                d[j] = fmaf(rx, fmaf(-kx, xn[j], h[j] * u[j]), d[j]);
                const float gy = a.scale * d[j] * s[j] * w[j];
                h[j] = gy * (1.f - s[j]) * (yv[j] * ry);
                yv[j] = ry * fmaf(-ky, yv[j], gy);
            }
            put<V>((TX *)a.dx + at + c, d);
            if (gate) put<V>((T *)a.dgate + at + c, h);
            put<V>((T *)a.dy + at + c, yv);
        }
    }
    if (BACK) {
        float *part = a.part + ((int64_t)blockIdx.x * RPC + side) * 2 * D;
        for (int c = t; c < D; c += TPR * V)
            for (int j = 0; j < V; ++j) {
                part[c + j] = dwo[c + j];
                part[D + c + j] = dwi[c + j];
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

// The weights' gradients from `parts` partial sums.
cudaError_t launch_weights(const BlockNormArgs &a, int parts, cudaStream_t st) {
    block_norm_weights_kernel<<<(2 * a.width + 31) / 32, 1024, 0, st>>>(a.part, parts, a.width, a.dw_post, a.dw_pre);
    const cudaError_t e = cudaGetLastError();
    Profiler::mark(st);
    return e;
}

template <int V, int TPR, bool BACK, bool STASH, typename TX, typename T>
cudaError_t launch_any_s(const BlockNormArgs &a, size_t smem, cudaStream_t st) {
    constexpr int RPC = kAnyThreads / TPR;
    const int64_t grid = grid_of(a.rows, RPC, BACK ? kAnyBackward : 4);
    const auto kernel = block_norm_any_kernel<V, TPR, BACK, STASH, TX, T>;
    if (grid > 0) {
        const cudaError_t set =
            cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (set != cudaSuccess) return set;
        kernel<<<(unsigned)grid, kAnyThreads, smem, st>>>(a);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
        Profiler::mark(st);
    }
    return BACK ? launch_weights(a, (int)grid * RPC, st) : cudaSuccess;
}
template <int V, int TPR, bool BACK, typename TX, typename T>
cudaError_t launch_any_t(const BlockNormArgs &a, cudaStream_t st) {
    const size_t row = (size_t)(kAnyThreads / TPR) * a.width * sizeof(float);
    if (row * any_floats(BACK, true) <= 220 * 1024)
        return launch_any_s<V, TPR, BACK, true, TX, T>(a, row * any_floats(BACK, true), st);
    return launch_any_s<V, TPR, BACK, false, TX, T>(a, row * any_floats(BACK, false), st);
}

// The next power of two of threads to a row, 32 to 512.
template <int V, bool BACK, typename TX, typename T>
cudaError_t launch_any(const BlockNormArgs &a, cudaStream_t st) {
    const int vecs = (a.width + V - 1) / V;
    if (vecs <= 32) return launch_any_t<V, 32, BACK, TX, T>(a, st);
    if (vecs <= 128) return launch_any_t<V, 128, BACK, TX, T>(a, st);
    return launch_any_t<V, 512, BACK, TX, T>(a, st);
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
    return BACK ? launch_weights(a, (int)grid * RPC, st) : cudaSuccess;
}

// The ring takes as many stages as fit; with one, the next rows come while the present ones are
// worked on, since a stage is free after the first barrier.
template <int V, int NV, int TPR, int NT, int CTAS, bool BACK, typename TX, typename T>
cudaError_t launch_t(BlockNormArgs a, cudaStream_t st) {
    {
        const size_t stage = (size_t)(NT / TPR) * a.width *
                             ((BACK ? 2 : 1) * sizeof(TX) + ((BACK ? 2 : 1) + (a.gate ? 1 : 0)) * sizeof(T));
        const size_t fit = kRingBytes / CTAS / stage;
        a.stages = (int)(fit < (size_t)kBlockNormStages ? fit : (size_t)kBlockNormStages);
        if (a.stages >= 1)
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
    return launch_t<V, 4, 512, 512, 1, BACK, TX, T>(a, st);
}

// Elements that every row and tensor lets be read at a time: 8 (the ring), 2 or 1.
int elements_at_once(const BlockNormArgs &a) {
    uintptr_t at = 0;
    for (const void *p : {a.x, a.y, a.gate, a.w_post, a.w_pre, a.dx_new, a.dh, (const void *)a.x_new,
                          (const void *)a.h, (const void *)a.dx, (const void *)a.dy, (const void *)a.dgate})
        at |= reinterpret_cast<uintptr_t>(p);
    if (a.width % 8 == 0 && (at & 15u) == 0) return 8;
    return a.width % 2 == 0 && (at & 7u) == 0 ? 2 : 1;
}

template <bool BACK, typename TX, typename T>
cudaError_t launch_types(const BlockNormArgs &a, cudaStream_t st) {
    switch (elements_at_once(a)) {
        case 8: return launch_v<8, BACK, TX, T>(a, st);
        case 2: return launch_any<2, BACK, TX, T>(a, st);
        default: return launch_any<1, BACK, TX, T>(a, st);
    }
}

}  // namespace

size_t block_norm_parts(int64_t rows, int width) {
    // rows side by side in a CTA of 512 threads, for each number of elements at once: the largest
    static_assert(BNT == kAnyThreads, "one CTA size for all paths");
    size_t most = 0;
    for (int v : {1, 2, 8}) {
        const int vecs = (width + v - 1) / v;
        int tpr = 32;
        while (tpr < BNT && tpr < vecs) tpr *= 2;
        const size_t parts = (size_t)grid_of(rows, BNT / tpr, v == 8 ? BC : kAnyBackward) * (BNT / tpr);
        if (parts > most) most = parts;
    }
    return most;
}

cudaError_t launch_block_norm(const BlockNormArgs &a, bool x_bf16, bool bf16, bool backward,
                              cudaStream_t st) {
    using bf = __nv_bfloat16;
    if (x_bf16) return backward ? launch_types<true, bf, bf>(a, st) : launch_types<false, bf, bf>(a, st);
    if (bf16) return backward ? launch_types<true, float, bf>(a, st) : launch_types<false, float, bf>(a, st);
    return backward ? launch_types<true, float, float>(a, st) : launch_types<false, float, float>(a, st);
}

}  // namespace kda
