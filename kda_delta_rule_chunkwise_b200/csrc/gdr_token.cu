// Gated delta rule, token by token in fp32: the decode step (one or a few tokens per
// request, either input type) and, by a kernel of its own below, the prefill of fp32 inputs.
//
// Per (request n, value head h) and token, with a = exp(g):
//     p = S^T k;  y = S^T q;  delta = beta (v - a p);  o = a y + (k.q) delta
//     S <- a S + k delta^T
// so one pass over the state gives both sums, and a second one updates it.
//
// One decode token is bound by HBM: each state (dk x dv fp32, 64 KiB at d = 128) is read
// and written once, everything else is about 1 KiB.  With L tokens the state stays in
// registers between them, so they cost one pass over it as well.  256 requests of 32 heads:
// 185 us for 1.08 GB (5.9 TB/s, 90 % of a plain copy); 48 requests of up to 5 tokens: 49 us
// for 204 MB, the tokens' barriers beside the pass.  Without the update: 103 us for 256 tokens.
//
// One CTA of 256 threads per (n, h, slice of DVS columns).  A thread keeps a
// (DK / RG) x 4 block of S in registers, loaded as coalesced 16-byte vectors.  The sums
// over channels are taken over a thread's rows, over the lanes of a warp that hold the
// same columns, and over the eight warps through shared memory, always in the same order.
// Inputs of the next token are loaded while this one is computed; buffers alternate and the next
// token's are filled between a token's two barriers, so that no third one is needed.
#include "gdr_common.cuh"
#include "gdr_launch.h"

namespace kda {
namespace gdr {

template <int DK, int DVS, typename Tin>
__global__ void __launch_bounds__(256) gdr_token_kernel(GdrTokenArgs a) {
    constexpr int NT = 256, CG = DVS / 4, RG = NT / CG, RPT = DK / RG, NW = NT / 32;
    static_assert(CG <= 32 && DK % RG == 0, "a warp covers whole rows");
    const int tid = threadIdx.x, cg = tid % CG, rg = tid / CG, warp = tid >> 5, lane = tid & 31;
    const int slices = a.dv / DVS;
    const int slice = blockIdx.x % slices, unit = blockIdx.x / slices;
    const int h = unit % a.H, n = unit / a.H, hk = h / (a.H / a.Hk);

    const int64_t first = (int64_t)n * a.T;   // row of the request's first token
    int len = (int)a.T;
    if (a.lens) len = min(max(a.lens[n], 0), len);
    int64_t entry = n;
    if (a.slots) {
        const int slot = a.slots[n];
        if (slot < 0 || slot >= a.P) {
            if (tid == 0 && h == 0 && slice == 0 && a.err) atomicOr(a.err, ERR_BAD_INDEX);
            return;
        }
        entry = slot;
    }
    if (len == 0 && (a.state_out == nullptr || a.state_out == a.state_in)) return;
    const int64_t soff = (entry * a.H + h) * DK * a.dv + slice * DVS;

    __shared__ float ks[2][DK], qs[2][DK], vs[2][DVS], gb[2][2];
    __shared__ float4 red_p[2][NW][CG], red_y[2][NW][CG];
    __shared__ float dl[2][DVS], kq[2];

    float4 s[RPT];
#pragma unroll
    for (int i = 0; i < RPT; ++i)
        s[i] = a.state_in ? __ldcs(reinterpret_cast<const float4 *>(
                                a.state_in + soff + (int64_t)(rg + i * RG) * a.dv) + cg)
                          : make_float4(0.f, 0.f, 0.f, 0.f);

    // one element of k, q or v per thread: DK + DK + DVS of them, DK of q by the upper half
    const Tin *q = (const Tin *)a.q, *k = (const Tin *)a.k, *v = (const Tin *)a.v;
    float in_k = 0.f, in_v = 0.f, in_g = 0.f;
    auto fetch = [&](int t) {
        const int64_t row = first + t;
        if (tid < DK) in_k = to_f32(k[(row * a.Hk + hk) * DK + tid]);
        else if (tid >= 128 && tid < 128 + DK) in_k = to_f32(q[(row * a.Hk + hk) * DK + tid - 128]);
        if (tid < DVS) in_v = to_f32(v[(row * a.H + h) * a.dv + slice * DVS + tid]);
        if (tid == 0) in_g = to_f32(((const Tin *)a.g)[row * a.H + h]);
        if (tid == 32) in_g = to_f32(((const Tin *)a.beta)[row * a.H + h]);
    };
    auto publish = [&](int b) {
        if (tid < DK) ks[b][tid] = in_k;
        else if (tid >= 128 && tid < 128 + DK) qs[b][tid - 128] = in_k;
        if (tid < DVS) vs[b][tid] = in_v;
        if (tid == 0) gb[b][0] = decay(in_g);
        if (tid == 32) gb[b][1] = in_g;
    };
    if (len > 0) {
        fetch(0);
        publish(0);
    }
    __syncthreads();
    for (int t = 0; t < len; ++t) {
        const int b = t & 1;
        if (t + 1 < len) fetch(t + 1);
        float4 p = make_float4(0.f, 0.f, 0.f, 0.f), y = p;
#pragma unroll
        for (int i = 0; i < RPT; ++i) {
            const float kr = ks[b][rg + i * RG], qr = qs[b][rg + i * RG];
            p.x = fmaf(s[i].x, kr, p.x); p.y = fmaf(s[i].y, kr, p.y);
            p.z = fmaf(s[i].z, kr, p.z); p.w = fmaf(s[i].w, kr, p.w);
            y.x = fmaf(s[i].x, qr, y.x); y.y = fmaf(s[i].y, qr, y.y);
            y.z = fmaf(s[i].z, qr, y.z); y.w = fmaf(s[i].w, qr, y.w);
        }
#pragma unroll
        for (int m = CG; m < 32; m <<= 1) {
            p.x += __shfl_xor_sync(0xffffffffu, p.x, m); p.y += __shfl_xor_sync(0xffffffffu, p.y, m);
            p.z += __shfl_xor_sync(0xffffffffu, p.z, m); p.w += __shfl_xor_sync(0xffffffffu, p.w, m);
            y.x += __shfl_xor_sync(0xffffffffu, y.x, m); y.y += __shfl_xor_sync(0xffffffffu, y.y, m);
            y.z += __shfl_xor_sync(0xffffffffu, y.z, m); y.w += __shfl_xor_sync(0xffffffffu, y.w, m);
        }
        if (lane < CG) {
            red_p[b][warp][lane] = p;
            red_y[b][warp][lane] = y;
        }
        if (warp == NW - 1) {
            float d = 0.f;
#pragma unroll
            for (int c = 0; c < DK; c += 32) d = fmaf(ks[b][c + lane], qs[b][c + lane], d);
#pragma unroll
            for (int m = 16; m > 0; m >>= 1) d += __shfl_xor_sync(0xffffffffu, d, m);
            if (lane == 0) kq[b] = d;
        }
        __syncthreads();
        // Only now have all warps updated the state of the token before, whose key lies where the next
        // token's goes; the barrier below stands between this and its reading.
        if (t + 1 < len) publish(b ^ 1);
        const float dec = gb[b][0];
        if (tid < DVS) {
            float pj = 0.f, yj = 0.f;
#pragma unroll
            for (int w = 0; w < NW; ++w) {
                pj += reinterpret_cast<const float *>(&red_p[b][w][0])[tid];
                yj += reinterpret_cast<const float *>(&red_y[b][w][0])[tid];
            }
            const float d = gb[b][1] * (vs[b][tid] - dec * pj);
            dl[b][tid] = d;
            ((Tin *)a.o)[((first + t) * a.H + h) * a.dv + slice * DVS + tid] =
                from_f32<Tin>(fmaf(kq[b], d, dec * yj));
        }
        __syncthreads();
        const float4 d4 = reinterpret_cast<const float4 *>(dl[b])[cg];
#pragma unroll
        for (int i = 0; i < RPT; ++i) {
            const float kr = ks[b][rg + i * RG];
            s[i].x = fmaf(kr, d4.x, dec * s[i].x); s[i].y = fmaf(kr, d4.y, dec * s[i].y);
            s[i].z = fmaf(kr, d4.z, dec * s[i].z); s[i].w = fmaf(kr, d4.w, dec * s[i].w);
        }
    }
    if (a.state_out) {
#pragma unroll
        for (int i = 0; i < RPT; ++i)
            __stcs(reinterpret_cast<float4 *>(a.state_out + soff + (int64_t)(rg + i * RG) * a.dv) + cg,
                   s[i]);
    }
}

// Prefill of fp32 inputs.  The same step, with nothing between the tokens but one warp: it keeps
// four columns of a state, each lane the rows lane + 32 i, and takes the eight sums over channels
// (S^T k and S^T q) in one halving exchange of nine shuffles.  No barrier and no shared memory;
// the inputs of the next four tokens are loaded while four are worked on.  What bounds it is the
// latency of a token's dependent steps, 0.24 us (256 tokens of 2 heads of 64: 62 us), so many narrow
// warps run side by side.
template <int DK>
__global__ void __launch_bounds__(128) gdr_token_prefill_kernel(GdrTokenArgs a) {
    constexpr int R = DK / 32, AHEAD = 4;
    const int lane = threadIdx.x & 31, groups = a.dv / 4;
    const int64_t w = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
    if (w >= (int64_t)a.N * a.H * groups) return;
    const int cg = (int)(w % groups), unit = (int)(w / groups);
    const int h = unit % a.H, n = unit / a.H, hk = h / (a.H / a.Hk);
    const Span span = sequence_span(a.cu_seqlens, n, a.T);
    const int64_t soff = ((int64_t)n * a.H + h) * DK * a.dv + cg * 4;
    const int mine = (lane >> 2) & 3;   // the column whose sums this lane ends up with

    float4 s[R];
#pragma unroll
    for (int i = 0; i < R; ++i)
        s[i] = a.state_in ? *reinterpret_cast<const float4 *>(a.state_in + soff + (int64_t)(lane + 32 * i) * a.dv)
                          : make_float4(0.f, 0.f, 0.f, 0.f);
    const float *q = (const float *)a.q + (span.row * a.Hk + hk) * DK + lane;
    const float *k = (const float *)a.k + (span.row * a.Hk + hk) * DK + lane;
    const float *v = (const float *)a.v + (span.row * a.H + h) * a.dv + cg * 4 + mine;
    const float *g = (const float *)a.g + span.row * a.H + h, *beta = (const float *)a.beta + span.row * a.H + h;
    float *o = (float *)a.o + (span.row * a.H + h) * a.dv + cg * 4 + mine;
    const int64_t kstride = (int64_t)a.Hk * DK, vstride = (int64_t)a.H * a.dv;

    struct Token {
        float k[R], q[R], v, g, b;
    };
    auto fetch = [&](Token (&t)[AHEAD], int from) {
#pragma unroll
        for (int j = 0; j < AHEAD; ++j) {
            const int64_t at = from + j;
            const bool live = at < span.len;   // a token of zeros changes nothing
#pragma unroll
            for (int i = 0; i < R; ++i) {
                t[j].k[i] = live ? __ldg(k + at * kstride + 32 * i) : 0.f;
                t[j].q[i] = live ? __ldg(q + at * kstride + 32 * i) : 0.f;
            }
            t[j].v = live ? __ldg(v + at * vstride) : 0.f;
            t[j].g = live ? __ldg(g + at * a.H) : 0.f;
            t[j].b = live ? __ldg(beta + at * a.H) : 0.f;
        }
    };
    Token now[AHEAD], next[AHEAD];
    fetch(next, 0);
    for (int t0 = 0; t0 < span.len; t0 += AHEAD) {
#pragma unroll
        for (int j = 0; j < AHEAD; ++j) now[j] = next[j];
        fetch(next, t0 + AHEAD);
        float kq[AHEAD], dec[AHEAD];   // k.q and the decays do not wait for the state
#pragma unroll
        for (int j = 0; j < AHEAD; ++j) {
            float x = 0.f;
#pragma unroll
            for (int i = 0; i < R; ++i) x = fmaf(now[j].k[i], now[j].q[i], x);
#pragma unroll
            for (int m = 16; m > 0; m >>= 1) x += __shfl_xor_sync(0xffffffffu, x, m);
            kq[j] = x;
            dec[j] = decay(now[j].g);
        }
#pragma unroll
        for (int j = 0; j < AHEAD; ++j) {
            // sums 0-3: S^T k of the four columns, 4-7: S^T q
            float x[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = 0.f;
#pragma unroll
            for (int i = 0; i < R; ++i) {
                const float kr = now[j].k[i], qr = now[j].q[i];
                x[0] = fmaf(s[i].x, kr, x[0]); x[1] = fmaf(s[i].y, kr, x[1]);
                x[2] = fmaf(s[i].z, kr, x[2]); x[3] = fmaf(s[i].w, kr, x[3]);
                x[4] = fmaf(s[i].x, qr, x[4]); x[5] = fmaf(s[i].y, qr, x[5]);
                x[6] = fmaf(s[i].z, qr, x[6]); x[7] = fmaf(s[i].w, qr, x[7]);
            }
            // each step halves the sums a lane has: bit 4 of the lane picks k or q, bits 3 and 2 the column
#pragma unroll
            for (int half = 4; half > 0; half >>= 1) {
                const int m = half * 4;
                const bool up = (lane & m) != 0;
#pragma unroll
                for (int i = 0; i < half; ++i) {
                    const float give = up ? x[i] : x[i + half], keep = up ? x[i + half] : x[i];
                    x[i] = keep + __shfl_xor_sync(0xffffffffu, give, m);
                }
            }
            float z = x[0];
            z += __shfl_xor_sync(0xffffffffu, z, 2);
            z += __shfl_xor_sync(0xffffffffu, z, 1);
            // lanes with bit 4 clear hold S^T k, the others S^T q
            const float d = now[j].b * (now[j].v - dec[j] * z);
            const float d0 = __shfl_sync(0xffffffffu, d, 0), d1 = __shfl_sync(0xffffffffu, d, 4);
            const float d2 = __shfl_sync(0xffffffffu, d, 8), d3 = __shfl_sync(0xffffffffu, d, 12);
            const float dm = mine & 2 ? (mine & 1 ? d3 : d2) : (mine & 1 ? d1 : d0);
            if ((lane & 19) == 16 && t0 + j < span.len) o[(t0 + j) * vstride] = fmaf(kq[j], dm, dec[j] * z);
#pragma unroll
            for (int i = 0; i < R; ++i) {
                const float kr = now[j].k[i];
                s[i].x = fmaf(kr, d0, dec[j] * s[i].x); s[i].y = fmaf(kr, d1, dec[j] * s[i].y);
                s[i].z = fmaf(kr, d2, dec[j] * s[i].z); s[i].w = fmaf(kr, d3, dec[j] * s[i].w);
            }
        }
    }
    if (a.state_out)
#pragma unroll
        for (int i = 0; i < R; ++i)
            *reinterpret_cast<float4 *>(a.state_out + soff + (int64_t)(lane + 32 * i) * a.dv) = s[i];
}

template <int DK, int DVS, typename Tin>
static cudaError_t launch_token_t(const GdrTokenArgs &a, cudaStream_t st) {
    const int64_t grid = (int64_t)a.N * a.H * (a.dv / DVS);
    gdr_token_kernel<DK, DVS, Tin><<<(unsigned)grid, 256, 0, st>>>(a);
    const cudaError_t e = cudaGetLastError();
    Profiler::mark(st);
    return e;
}

template <int DK, typename Tin>
static cudaError_t launch_token_d(const GdrTokenArgs &a, cudaStream_t st) {
    // few (request, head) units: narrow slices, so that more SMs read the states (32 heads of 128, times
    // between events around the launch: 1 request 9.9 us against 11.7 with whole states, 2 requests 10.0
    // against 10.7, 4 the same, 8 requests 13.2 against 12.1)
    const int64_t units = (int64_t)a.N * a.H;
    if (units * (a.dv / 32) <= 2 * 148) return launch_token_t<DK, 32, Tin>(a, st);
    return a.dv == 64 ? launch_token_t<DK, 64, Tin>(a, st) : launch_token_t<DK, 128, Tin>(a, st);
}

}  // namespace gdr

cudaError_t launch_gdr_token(const GdrTokenArgs &a, bool bf16, cudaStream_t st) {
    if (a.dk == 64)
        return bf16 ? gdr::launch_token_d<64, __nv_bfloat16>(a, st)
                    : gdr::launch_token_d<64, float>(a, st);
    return bf16 ? gdr::launch_token_d<128, __nv_bfloat16>(a, st)
                : gdr::launch_token_d<128, float>(a, st);
}

cudaError_t launch_gdr_token_prefill(const GdrTokenArgs &a, cudaStream_t st) {
    const int64_t warps = (int64_t)a.N * a.H * (a.dv / 4);
    const unsigned grid = (unsigned)((warps + 3) / 4);
    if (a.dk == 64) gdr::gdr_token_prefill_kernel<64><<<grid, 128, 0, st>>>(a);
    else gdr::gdr_token_prefill_kernel<128><<<grid, 128, 0, st>>>(a);
    const cudaError_t e = cudaGetLastError();
    Profiler::mark(st);
    return e;
}

}  // namespace kda
