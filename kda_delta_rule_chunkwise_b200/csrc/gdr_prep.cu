// Gated delta rule: the chunks' images, made once per chunk ahead of the chains.
//
// Per (32-token chunk, key head), by one warp:
//   K', Q'  rows of keys and queries as fp16 after a power-of-two scale per row that puts the row's
//           largest element in [1, 2) (exact but for elements below 2^-17 of it); ik, iq undo it
//   Q' K'^T and K' K'^T, blocks on and below the diagonal
// and for each value head of the group, with G the running sum of g (64 bits: the decay between far
// rows is a difference of long sums), D[r][s] = exp(G_r - G_s):
//   P       D[r][s] (q'_r . k'_s), s <= r
//   X       (I + A)^-1, A[r][s] = D[r][s] (k_r . k_s) b, s < r; b = beta_s (forward: N = X (V - Gamma
//           K S), U = beta N) or b = beta_r (adjoint: E = X^T dU, dR = beta E)
//   scalars of HeadImage
// The inverse in fp32: the two 16x16 diagonal blocks by forward substitution (one column per lane,
// both blocks at once), the block below them as -X22 A21 X11 in split products.
//
// A warp keeps its tiles in shared memory (26 KiB, 34 KiB with both inverses), builds an image there
// and sends it off with one bulk store; rows come in by coalesced asynchronous copies.  What bounds it is
// latency at eight warps per SM with few chunks (8192 tokens, 16 key and 32 value heads: 55 us for
// 0.21 GB read and written), the bytes with many (65536 tokens of 32 and 32 heads: 2.8 GB in 502 us).
//
// X fits fp16 where g <= 0 and 0 <= b |k|^2 <= 2 (b = beta): off the diagonal X[r][s] is
// -D[r][s] k_r^T (prod over s < j < r of I - b_j k_j k_j^T) k_s times b_s (b_r for the adjoint), and no
// factor of the product is longer than 1, so |X[r][s]| <= b |k_r| |k_s| < 2^14.  The same holds for A.
// With the 1/32 that is taken beyond 2 each of the at most 30 factors is at most 1 + 1/32 long: 2.6 times that.
#include "gdr_common.cuh"
#include "gdr_launch.h"

namespace kda {
namespace gdr {

struct PrepArgs {
    const __nv_bfloat16 *q, *k, *g, *beta;
    const int32_t *cu;
    int64_t T;
    int Hk, H, splits;   // CTAs per (sequence, key head)
    unsigned char *keys, *forward, *adjoint;
};

template <bool ADJ>
constexpr int prep_warps() { return ADJ ? 6 : 8; }   // as many as their tiles fit
// The diagonal blocks of A while they are inverted stand where P of the image will: 2 x 16 rows.
constexpr int kAP = 20;   // fp32 row pitch
static_assert(2 * 16 * kAP * 4 <= kChunk * HeadImage<false>::XP, "A fits the place of P");
// The forward's image; the backward's recomputation has no use for P.
template <bool ADJ>
constexpr int forward_bytes() { return ADJ ? HeadImage<false>::P : HeadImage<false>::BYTES; }
template <int DK, bool ADJ>
constexpr int prep_warp_bytes() {
    return KeyImage<DK>::BYTES + forward_bytes<ADJ>() + (ADJ ? HeadImage<true>::BYTES : 0);
}

// 32 rows of D bf16 elements into a padded tile, zeros from row `valid` on: coalesced copies.
template <int D>
__device__ __forceinline__ void copy_rows(uint32_t tile, int pitch, const __nv_bfloat16 *base, int64_t stride,
                                          int valid) {
    constexpr int LPR = D / 8, RPI = 32 / LPR;
    const int lane = threadIdx.x & 31, c = lane % LPR;
#pragma unroll 4
    for (int r = lane / LPR; r < kChunk; r += RPI) {
        const bool ok = r < valid;
        const int n = ok ? 16 : 0;   // the rest of the 16 bytes is filled with zeros
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(tile + r * pitch + c * 16),
                     "l"(base + (ok ? r * stride : 0) + c * 8), "r"(n)
                     : "memory");
    }
}
// In place: lane r scales row r of a bf16 tile into fp16; returns 2^-e.
template <int D>
__device__ __forceinline__ float scale_row(uint32_t tile, int pitch) {
    tile += (threadIdx.x & 31) * pitch;
    uint32_t w[D / 8][4];
    __nv_bfloat162 m = __floats2bfloat162_rn(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < D / 8; ++i)
        asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(w[i][0]), "=r"(w[i][1]), "=r"(w[i][2]), "=r"(w[i][3])
                     : "r"(tile + i * 16)
                     : "memory");
#pragma unroll
    for (int i = 0; i < D / 8; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) m = __hmax2(m, __habs2(reinterpret_cast<const __nv_bfloat162 &>(w[i][j])));
    const float top = fmaxf(__low2float(m), __high2float(m));
    const int e = min(max((int)(__float_as_uint(top) >> 23), 1), 253);
    const float sc = __uint_as_float((uint32_t)(254 - e) << 23);
#pragma unroll
    for (int i = 0; i < D / 8; ++i) {
        uint32_t h[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            h[j] = pack_half(__uint_as_float(w[i][j] << 16) * sc, __uint_as_float(w[i][j] & 0xffff0000u) * sc);
        asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(tile + i * 16), "r"(h[0]), "r"(h[1]),
                     "r"(h[2]), "r"(h[3])
                     : "memory");
    }
    return __uint_as_float((uint32_t)e << 23);
}

// X into an image (HeadImage's XH, XL) from K' K'^T (times D and the row scales already) and b:
// A = acc times b_s (forward) or b_r (adjoint).
template <bool ADJ>
__device__ __forceinline__ void invert(unsigned char *image, float *scratch, const float (&kk)[6][4], float b) {
    using HI = HeadImage<ADJ>;
    const int lane = threadIdx.x & 31, r0 = lane >> 2, c0 = 2 * (lane & 3);
    const uint32_t xh = smem_u32(image) + HI::XH, xl = smem_u32(image) + HI::XL;
    float br[4], bs[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) br[i] = ADJ ? __shfl_sync(0xffffffffu, b, r0 + 8 * i) : 1.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) bs[j] = ADJ ? 1.f : __shfl_sync(0xffffffffu, b, c0 + 8 * (j >> 1) + (j & 1));
    // diagonal blocks to the scratch; A21 as fp16 hi + lo where X21 will stand.  The block above the
    // diagonal is never read.
#pragma unroll
    for (int i = 0; i < 6; ++i)
#pragma unroll
        for (int x = 0; x < 4; x += 2) {
            const int ri = (i < 2 ? 0 : 2) + (x >> 1), cj = (i < 2 ? i : i - 2) * 2;
            const float a0 = kk[i][x] * br[ri] * bs[cj], a1 = kk[i][x + 1] * br[ri] * bs[cj + 1];
            const int r = r0 + (x >> 1) * 8;   // within the row block
            if (i == 2 || i == 3) {
                uint32_t hi, lo;
                split_half(a0, a1, hi, lo);
                const int at = (16 + r) * HI::XP + ((i - 2) * 8 + c0) * 2;
                *reinterpret_cast<uint32_t *>(image + HI::XH + at) = hi;
                *reinterpret_cast<uint32_t *>(image + HI::XL + at) = lo;
            } else {
                *reinterpret_cast<float2 *>(scratch + (i < 2 ? 0 : 16 * kAP) + r * kAP + (i & 1) * 8 + c0) =
                    make_float2(a0, a1);
            }
        }
    __syncwarp();
    {   // column lane % 16 of (I + A)^-1 of diagonal block lane / 16
        const float *A = scratch + (lane >> 4) * 16 * kAP;
        unsigned char *to = image + HI::XH + (lane >> 4) * (16 * HI::XP + 32) + (lane & 15) * 2;
        float x[16];
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            float a0 = r == (lane & 15) ? 1.f : 0.f, a1 = 0.f;
            const float4 *row = reinterpret_cast<const float4 *>(A + r * kAP);
#pragma unroll
            for (int s4 = 0; s4 < (r + 3) / 4; ++s4) {
                const float4 w = row[s4];
                if (4 * s4 + 0 < r) a0 = fmaf(-w.x, x[4 * s4 + 0], a0);
                if (4 * s4 + 1 < r) a1 = fmaf(-w.y, x[4 * s4 + 1], a1);
                if (4 * s4 + 2 < r) a0 = fmaf(-w.z, x[4 * s4 + 2], a0);
                if (4 * s4 + 3 < r) a1 = fmaf(-w.w, x[4 * s4 + 3], a1);
            }
            x[r] = a0 + a1;
        }
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            const __half h = __float2half_rn(x[r]);
            *reinterpret_cast<__half *>(to + r * HI::XP) = h;
            *reinterpret_cast<__half *>(to + (HI::XL - HI::XH) + r * HI::XP) =
                __float2half_rn(x[r] - __half2float(h));
        }
    }
    __syncwarp();
    // X21 = -(X22 A21) X11
    const int am = (16 + (lane & 15)) * HI::XP + (lane >> 4) * 16;   // rows 16.., as [m][k]
    const int bt = (lane & 15) * HI::XP + (lane >> 4) * 16;          // as [k][n], transposed
    uint32_t ah[4], al[4], bh[4], bl[4];
    ldsm4(ah, xh + am + 32);
    ldsm4(al, xl + am + 32);
    ldsm4_t(bh, xh + bt + 16 * HI::XP);
    ldsm4_t(bl, xl + bt + 16 * HI::XP);
    float m[2][4];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
#pragma unroll
        for (int x = 0; x < 4; ++x) m[t][x] = 0.f;
        mma16816(m[t], ah, bh[2 * t], bh[2 * t + 1]);
        mma16816(m[t], al, bh[2 * t], bh[2 * t + 1]);
        mma16816(m[t], ah, bl[2 * t], bl[2 * t + 1]);
    }
    split_half(m[0][0], m[0][1], ah[0], al[0]);
    split_half(m[0][2], m[0][3], ah[1], al[1]);
    split_half(m[1][0], m[1][1], ah[2], al[2]);
    split_half(m[1][2], m[1][3], ah[3], al[3]);
    ldsm4_t(bh, xh + bt);
    ldsm4_t(bl, xl + bt);
    __syncwarp();   // A21 has been read
#pragma unroll
    for (int t = 0; t < 2; ++t) {
#pragma unroll
        for (int x = 0; x < 4; ++x) m[t][x] = 0.f;
        mma16816(m[t], ah, bh[2 * t], bh[2 * t + 1]);
        mma16816(m[t], al, bh[2 * t], bh[2 * t + 1]);
        mma16816(m[t], ah, bl[2 * t], bl[2 * t + 1]);
#pragma unroll
        for (int x = 0; x < 4; x += 2) {
            uint32_t hi, lo;
            split_half(-m[t][x], -m[t][x + 1], hi, lo);
            const int at = (16 + r0 + (x >> 1) * 8) * HI::XP + (8 * t + c0) * 2;
            *reinterpret_cast<uint32_t *>(image + HI::XH + at) = hi;
            *reinterpret_cast<uint32_t *>(image + HI::XL + at) = lo;
        }
    }
}

// The rest of a value head's image: scalars, and P (hi, and lo for the adjoint).
template <bool ADJ>
__device__ __forceinline__ void fill_image(unsigned char *image, const float (&qk)[6][4], const float (&D)[6][4],
                                           float ik, float iq, float into, float out, float b, bool want_p) {
    using HI = HeadImage<ADJ>;
    const int lane = threadIdx.x & 31, r0 = lane >> 2, c0 = 2 * (lane & 3);
    float *at = reinterpret_cast<float *>(image + HI::S) + lane;
    at[HI::IK * kChunk] = ik;
    at[HI::CK * kChunk] = into * ik;
    at[HI::OK * kChunk] = ADJ ? out * ik : out * ik * b;
    at[HI::BETA * kChunk] = b;
    at[HI::IQ * kChunk] = iq;
    at[HI::CQ * kChunk] = into * iq;
    at[HI::MISC * kChunk] = __shfl_sync(0xffffffffu, into, 31);
    at[HI::BK * kChunk] = ik * b;
    if (want_p)
#pragma unroll
        for (int i = 0; i < 6; ++i)
#pragma unroll
            for (int x = 0; x < 4; x += 2) {
                const int r = (i < 2 ? 0 : 16) + r0 + (x >> 1) * 8, s = (i < 2 ? i : i - 2) * 8 + c0;
                uint32_t hi, lo;
                split_half(qk[i][x] * D[i][x], qk[i][x + 1] * D[i][x + 1], hi, lo);
                *reinterpret_cast<uint32_t *>(image + HI::P + r * HI::XP + s * 2) = hi;
                if (ADJ) *reinterpret_cast<uint32_t *>(image + HI::PL + r * HI::XP + s * 2) = lo;
            }
}

// ADJ: the adjoint's images as well as the forward's.
template <int DK, bool ADJ>
__global__ void __launch_bounds__(prep_warps<ADJ>() * 32, 1) gdr_prep_kernel(PrepArgs a) {
    using KI = KeyImage<DK>;
    extern __shared__ __align__(128) unsigned char smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    unsigned char *keys = smem + warp * prep_warp_bytes<DK, ADJ>();
    unsigned char *fwd = keys + KI::BYTES, *adj = fwd + forward_bytes<ADJ>();
    // where P will stand: the adjoint's, where there is one (the forward's image then ends before P)
    float *scratch = reinterpret_cast<float *>(ADJ ? adj + HeadImage<true>::P : fwd + HeadImage<false>::P);
    const uint32_t kt = smem_u32(keys) + KI::K, qt = smem_u32(keys) + KI::Q;

    const int split = blockIdx.x % a.splits, pair = blockIdx.x / a.splits;
    const int hk = pair % a.Hk, n = pair / a.Hk, group = a.H / a.Hk;
    const Span span = sequence_span(a.cu, n, a.T);
    const int chunks = (span.len + kChunk - 1) / kChunk;
    const int r0 = lane >> 2, c0 = 2 * (lane & 3);
    for (int c = split * prep_warps<ADJ>() + warp; c < chunks; c += a.splits * prep_warps<ADJ>()) {
        const int valid = min(kChunk, span.len - c * kChunk);
        const int64_t row = span.row + (int64_t)c * kChunk + lane, slot = first_chunk(span, n) + c;
        const bool live = lane < valid;
        if (lane == 0) bulk_store_wait_read();   // the images before have left shared memory
        __syncwarp();
        const int64_t koff = ((row - lane) * a.Hk + hk) * DK, stride = (int64_t)a.Hk * DK;
        copy_rows<DK>(kt, KI::KP, a.k + koff, stride, valid);
        copy_rows<DK>(qt, KI::KP, a.q + koff, stride, valid);
        asm volatile("cp.async.wait_all;" ::: "memory");
        __syncwarp();
        const float ik = scale_row<DK>(kt, KI::KP);
        const float iq = scale_row<DK>(qt, KI::KP);
        fence_proxy_async_shared();
        __syncwarp();
        if (lane == 0) {
            bulk_store(a.keys + (slot * a.Hk + hk) * KI::BYTES, kt, KI::BYTES);
            bulk_store_commit();
        }
        float kk[6][4], qk[6][4];
        gram_lower<DK>(qk, qt, kt, KI::KP);
        gram_lower<DK>(kk, kt, kt, KI::KP);
        {   // k_r . k_s in true units
            float ir[4], is[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) ir[i] = __shfl_sync(0xffffffffu, ik, r0 + 8 * i);
#pragma unroll
            for (int j = 0; j < 8; ++j) is[j] = __shfl_sync(0xffffffffu, ik, c0 + 8 * (j >> 1) + (j & 1));
#pragma unroll
            for (int i = 0; i < 6; ++i)
#pragma unroll
                for (int x = 0; x < 4; ++x)
                    kk[i][x] *= ir[(i < 2 ? 0 : 2) + (x >> 1)] * is[(i < 2 ? i : i - 2) * 2 + (x & 1)];
        }
#pragma unroll 1
        for (int hg = 0; hg < group; ++hg) {
            const int h = hk * group + hg;
            float g = 0.f, b = 0.f;
            if (live) {
                g = log_decay(__bfloat162float(a.g[row * a.H + h]));
                b = __bfloat162float(a.beta[row * a.H + h]);
            }
            double G = (double)g;
#pragma unroll
            for (int m = 1; m < 32; m <<= 1) {
                const double o = __shfl_up_sync(0xffffffffu, G, m);
                if (lane >= m) G += o;
            }
            const double Gend = __shfl_sync(0xffffffffu, G, 31);
            const float into = decay((float)G), out = decay((float)(Gend - G));
            // D for this lane's rows lane/4 + 8i and columns 2(lane%4) + 8j + {0, 1}: exponents of
            // two as a high and a low part, so that far sums cancel exactly
            float D[6][4], dk[6][4];
            {
                const double G2 = G * 1.4426950408889634074;
                const float g_hi = (float)G2, g_lo = (float)(G2 - (double)g_hi);
                float hr[4], lr[4], hs[8], ls[8];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    hr[i] = __shfl_sync(0xffffffffu, g_hi, r0 + 8 * i);
                    lr[i] = __shfl_sync(0xffffffffu, g_lo, r0 + 8 * i);
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    hs[j] = __shfl_sync(0xffffffffu, g_hi, c0 + 8 * (j >> 1) + (j & 1));
                    ls[j] = __shfl_sync(0xffffffffu, g_lo, c0 + 8 * (j >> 1) + (j & 1));
                }
#pragma unroll
                for (int t = 0; t < 6; ++t)
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const int i = (t < 2 ? 0 : 2) + (x >> 1), j = (t < 2 ? t : t - 2) * 2 + (x & 1);
                        const int r = r0 + 8 * i, s = c0 + 8 * (j >> 1) + (j & 1);
                        D[t][x] = s <= r ? exp2_approx((hr[i] - hs[j]) + (lr[i] - ls[j])) : 0.f;
                        dk[t][x] = D[t][x] * kk[t][x];
                    }
            }
            if (lane == 0) bulk_store_wait_read();   // the head before has left shared memory
            __syncwarp();
            invert<false>(fwd, scratch, dk, b);
            fill_image<false>(fwd, qk, D, ik, iq, into, out, b, !ADJ);
            __syncwarp();
            if (ADJ) {
                invert<true>(adj, scratch, dk, b);
                fill_image<true>(adj, qk, D, ik, iq, into, out, b, true);
            }
            fence_proxy_async_shared();
            __syncwarp();
            if (lane == 0) {
                const int64_t at = slot * a.H + h;
                bulk_store(a.forward + at * HeadImage<false>::BYTES, smem_u32(fwd), forward_bytes<ADJ>());
                if (ADJ) bulk_store(a.adjoint + at * HeadImage<true>::BYTES, smem_u32(adj), HeadImage<true>::BYTES);
                bulk_store_commit();
            }
        }
    }
    if (lane == 0) bulk_store_wait();
}

// The sequences from the longest to the shortest, ties by index, so that the longest chains start
// first.  One CTA; beyond kOrderMost sequences their order is kept.
constexpr int kOrderMost = 4096;
__global__ void __launch_bounds__(1024) gdr_order_kernel(const int32_t *cu, int64_t T, int N, int32_t *order) {
    __shared__ int len[kOrderMost];
    if (N > kOrderMost) {
        for (int i = threadIdx.x; i < N; i += blockDim.x) order[i] = i;
        return;
    }
    // offsets clamped and raised to the largest before them, 32 sequences at a time
    if (threadIdx.x < 32) {
        int top = 0;
        for (int i0 = 0; i0 <= N; i0 += 32) {
            const int i = i0 + threadIdx.x;
            const int64_t c = i <= N ? cu[i] : 0;
            int x = max(top, (int)(c < 0 ? 0 : (c > T ? T : c)));
#pragma unroll
            for (int m = 1; m < 32; m <<= 1) {
                const int o = __shfl_up_sync(0xffffffffu, x, m);
                if ((int)threadIdx.x >= m) x = max(x, o);
            }
            const int before = __shfl_up_sync(0xffffffffu, x, 1);
            if (i >= 1 && i <= N) len[i - 1] = x - (threadIdx.x == 0 ? top : before);
            top = __shfl_sync(0xffffffffu, x, 31);
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < N; i += blockDim.x) {
        const int mine = len[i];
        int place = 0;
        for (int j = 0; j < N; ++j) place += len[j] > mine || (len[j] == mine && j < i);
        order[place] = i;
    }
}

template <int DK, bool ADJ>
static cudaError_t launch_prep_t(const PrepArgs &a, int64_t pairs, cudaStream_t st) {
    constexpr int bytes = prep_warps<ADJ>() * prep_warp_bytes<DK, ADJ>();
    static_assert(bytes <= 227 * 1024, "shared memory of a CTA");
    const auto kernel = gdr_prep_kernel<DK, ADJ>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    kernel<<<(unsigned)(pairs * a.splits), prep_warps<ADJ>() * 32, bytes, st>>>(a);
    e = cudaGetLastError();
    Profiler::mark(st);
    return e;
}

}  // namespace gdr

static size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }

size_t gdr_image_bytes(int64_t rows, int N, int Hk, int H, int dk, bool adjoint) {
    const size_t slots = (size_t)gdr::chunk_slots(rows, N);
    const size_t key = dk == 64 ? gdr::KeyImage<64>::BYTES : gdr::KeyImage<128>::BYTES;
    return up256(slots * Hk * key) + up256(slots * H * gdr::HeadImage<false>::BYTES) + up256((size_t)N * 4) +
           (adjoint ? up256(slots * H * gdr::HeadImage<true>::BYTES) : 0);
}

GdrImages gdr_images(void *space, const GdrArgs &a, bool adjoint) {
    const size_t slots = (size_t)gdr::chunk_slots(a.rows, a.N);
    const size_t key = a.dk == 64 ? gdr::KeyImage<64>::BYTES : gdr::KeyImage<128>::BYTES;
    GdrImages m;
    m.keys = static_cast<unsigned char *>(space);
    m.forward = m.keys + up256(slots * a.Hk * key);
    unsigned char *order = m.forward + up256(slots * a.H * gdr::HeadImage<false>::BYTES);
    m.order = a.cu_seqlens && a.N > 1 ? reinterpret_cast<int32_t *>(order) : nullptr;
    m.adjoint = adjoint ? order + up256((size_t)a.N * 4) : nullptr;
    return m;
}

cudaError_t launch_gdr_prep(const GdrArgs &p, const GdrImages &m, cudaStream_t st) {
    using bf = __nv_bfloat16;
    const int64_t pairs = (int64_t)p.N * p.Hk;
    // CTAs per (sequence, key head): enough for a few rounds over the SMs, at most one per six chunks of
    // the longest sequence there can be
    const int64_t most = (p.T + 6 * gdr::kChunk - 1) / (6 * gdr::kChunk);
    int64_t splits = (148 * 8 + pairs - 1) / pairs;
    splits = splits < most ? splits : most;
    if (splits < 1) splits = 1;
    if (m.order) {
        gdr::gdr_order_kernel<<<1, 1024, 0, st>>>(p.cu_seqlens, p.T, p.N, m.order);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
        Profiler::mark(st);
    }
    gdr::PrepArgs a{(const bf *)p.q, (const bf *)p.k, (const bf *)p.g, (const bf *)p.beta, p.cu_seqlens,
                    p.T, p.Hk, p.H, (int)splits, m.keys, m.forward, m.adjoint};
    if (m.adjoint)
        return p.dk == 64 ? gdr::launch_prep_t<64, true>(a, pairs, st) : gdr::launch_prep_t<128, true>(a, pairs, st);
    return p.dk == 64 ? gdr::launch_prep_t<64, false>(a, pairs, st) : gdr::launch_prep_t<128, false>(a, pairs, st);
}

}  // namespace kda
