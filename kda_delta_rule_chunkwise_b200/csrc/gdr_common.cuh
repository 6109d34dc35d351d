// Device helpers shared by the gated-delta-rule kernels: warp matrix products,
// the two-term fp16 split of fp32 operands, sequence bounds, and the work of a
// producer warp (one chunk's scaled keys and queries, their Gram products and
// the unit-lower-triangular inverse).
#pragma once

#include "kda_common.cuh"

#include <cuda_fp16.h>

namespace kda {
namespace gdr {

constexpr int kChunk = 32;          // tokens per chunk of the chained kernels
constexpr int kScratch = 2 * 16 * 20;   // floats of a producer's scratch
constexpr float kMinLogDecay = -100.f;

// ---------------------------------------------------------------- warp products
// D += A B with A 16x16 (row-major fragment) and B 16x8, fp16 operands, fp32 sums.
// Not volatile: the compiler may interleave independent products.
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void stsm4_t(uint32_t addr, uint32_t a, uint32_t b, uint32_t c,
                                        uint32_t d) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(addr),
                 "r"(a), "r"(b), "r"(c), "r"(d)
                 : "memory");
}

// One row from global to shared memory by an asynchronous bulk copy (both addresses and
// the size are multiples of 16 bytes); its bytes complete the mbarrier's phase.
__device__ __forceinline__ void bulk_row(uint32_t dst, const void *src, uint32_t bytes,
                                         uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::
            "r"(dst), "l"(src), "r"(bytes), "r"(smem_u32(bar))
        : "memory");
}
// Orders this thread's earlier shared-memory accesses before later bulk copies into it.
__device__ __forceinline__ void fence_proxy_async_shared() {
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// ---------------------------------------------------------------- operand split
// An fp32 operand x enters a product as fp16 hi + lo of x * 2^e, with e chosen
// per row so that the row's largest value lies in [2^14, 2^15): 22 bits below
// that maximum (2^-23 relative), independent of the operand's magnitude.  The
// power of two is exact and is taken out of the fp32 result again.
__device__ __forceinline__ uint32_t pack_half(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return reinterpret_cast<const uint32_t &>(h);
}
__device__ __forceinline__ void split_half(float a, float b, uint32_t &hi, uint32_t &lo) {
    const __half2 h = __floats2half2_rn(a, b);
    const float2 f = __half22float2(h);
    hi = reinterpret_cast<const uint32_t &>(h);
    lo = pack_half(a - f.x, b - f.y);
}
// 2^e and 2^-e for a row whose largest magnitude is m (m = 0 and huge m clamp).
__device__ __forceinline__ float row_scale(float m, float &inv) {
    int e = (int)((__float_as_uint(m) >> 23) & 255u);
    e = min(max(e, 16), 253);
    inv = __uint_as_float((uint32_t)(e - 14) << 23);
    return __uint_as_float((uint32_t)(268 - e) << 23);
}
__device__ __forceinline__ float quad_max(float m) {
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
    return fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
}

// The largest of a warp's values (m: this lane's), for its part of a stored block: two slots,
// one for each half of the channels (both written where one warp has them all).
__device__ __forceinline__ void store_top(float *dst, float m, int halves, int part) {
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
    const int lane = threadIdx.x & 31;
    if (halves == 2 ? lane == 0 : lane < 2) dst[halves == 2 ? part : lane] = m;
}

// Wait of a whole warp with the library's bounds: every lane takes the same way.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, uint32_t *err,
                                          uint32_t epoch, volatile uint32_t *abort) {
    const bool ok = mbar_wait_abortable(bar, parity, err, epoch, abort);
    return __all_sync(0xffffffffu, ok);
}

// ---------------------------------------------------------------- sequences
// First row and length of sequence n: offsets clamped to [0, T] and raised to the
// largest offset before them, so that no offset leads outside the tensors.
struct Span {
    int64_t row;
    int len;
};
__device__ __forceinline__ Span sequence_span(const int32_t *cu, int n, int64_t T) {
    if (cu == nullptr) return {(int64_t)n * T, (int)T};
    int lo = 0;
    for (int i = threadIdx.x & 31; i <= n; i += 32) {
        const int64_t x = cu[i];
        lo = max(lo, (int)(x < 0 ? 0 : (x > T ? T : x)));
    }
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) lo = max(lo, __shfl_xor_sync(0xffffffffu, lo, m));
    const int64_t x = cu[n + 1];
    const int hi = max(lo, (int)(x < 0 ? 0 : (x > T ? T : x)));
    return {lo, hi - lo};
}
// First 64-token block of a sequence in the backward's per-block arrays: distinct
// for all sequences, since a sequence of len rows from `row` has at most
// (row + len) / 64 - row / 64 + 1 blocks.
__device__ __forceinline__ int64_t first_block(const Span &s, int n) { return s.row / 64 + n; }

// ---------------------------------------------------------------- a chunk in shared memory
// Byte offsets inside one stage.  Rows are padded by 16 bytes, so the eight rows
// of an ldmatrix lie in different banks.
template <int DK, int W, bool PLO>
struct Stage {
    static constexpr int KP = DK * 2 + 16;       // keys, queries: fp16 [32][DK]
    static constexpr int XP = kChunk * 2 + 16;   // 32 x 32 fp16 matrices
    static constexpr int VP = W * 2 + 16;        // values (or output gradients): bf16 [32][W]
    static constexpr int K = 0;
    static constexpr int Q = K + kChunk * KP;
    static constexpr int XH = Q + kChunk * KP;
    static constexpr int XL = XH + kChunk * XP;
    static constexpr int P = XL + kChunk * XP;
    static constexpr int PL = P + kChunk * XP;   // low part of P (adjoint only)
    static constexpr int V = PL + (PLO ? kChunk * XP : 0);
    static constexpr int S = V + kChunk * VP;    // per-row scalars, 8 x 32 fp32
    static constexpr int BYTES = S + 8 * kChunk * 4;
    // rows of the scalar block
    enum { IK = 0, CK = 1, OK = 2, BETA = 3, IQ = 4, CQ = 5, MISC = 6 };
};

// In place: lane r scales row r of a bf16 tile by the power of two that puts its largest element in
// [1, 2) and stores it as fp16 (exact but for elements below 2^-17 of the row's largest);
// rows from `valid` on become zeros.  Returns 2^-e.  Padded rows: the lanes' 16-byte
// pieces lie in different banks.
template <int D>
__device__ __forceinline__ float scale_row(uint32_t tile, int pitch, bool valid) {
    const int lane = threadIdx.x & 31;
    tile += lane * pitch;
    __nv_bfloat162 m = __floats2bfloat162_rn(0.f, 0.f);
#pragma unroll 4
    for (int c = 0; c < D * 2; c += 16) {
        uint32_t w[4];
        asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                     : "r"(tile + c)
                     : "memory");
#pragma unroll
        for (int j = 0; j < 4; ++j)
            m = __hmax2(m, __habs2(reinterpret_cast<const __nv_bfloat162 &>(w[j])));
    }
    const float top = fmaxf(__low2float(m), __high2float(m));
    int e = (int)(__float_as_uint(top) >> 23);
    e = valid ? min(max(e, 1), 253) : 1;
    const float sc = __uint_as_float((uint32_t)(254 - e) << 23);
#pragma unroll 4
    for (int c = 0; c < D * 2; c += 16) {
        uint32_t w[4], h[4];
        asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                     : "r"(tile + c)
                     : "memory");
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            h[j] = pack_half(__uint_as_float(w[j] << 16) * sc,
                             __uint_as_float(w[j] & 0xffff0000u) * sc);
            if (!valid) h[j] = 0u;
        }
        asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(tile + c), "r"(h[0]), "r"(h[1]),
                     "r"(h[2]), "r"(h[3])
                     : "memory");
    }
    return __uint_as_float((uint32_t)e << 23);
}

__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Lower triangle (16x16 blocks on and below the diagonal) of K K^T, and of Q K^T if
// WANT_Q, for scaled [32][D] tiles: accumulator tiles (row block, column tile) = (0,0)
// (0,1) (1,0..3).
template <int D, bool WANT_Q>
__device__ __forceinline__ void gram_lower(float (&kk)[6][4], float (&qk)[6][4], uint32_t k,
                                           uint32_t q, int pitch) {
    const int lane = threadIdx.x & 31;
    const int am = (lane & 15) * pitch + (lane >> 4) * 16;
    const int bn = ((lane & 7) + ((lane >> 4) & 1) * 8) * pitch + ((lane >> 3) & 1) * 16;
#pragma unroll
    for (int i = 0; i < 6; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) kk[i][j] = qk[i][j] = 0.f;
#pragma unroll 2
    for (int c = 0; c < D * 2; c += 32) {
        uint32_t a0[4], a1[4], b0[4], b1[4];
        ldsm4(b0, k + bn + c);
        ldsm4(b1, k + bn + 16 * pitch + c);
        ldsm4(a0, k + am + c);
        ldsm4(a1, k + am + 16 * pitch + c);
        mma16816(kk[0], a0, b0[0], b0[1]);
        mma16816(kk[1], a0, b0[2], b0[3]);
        mma16816(kk[2], a1, b0[0], b0[1]);
        mma16816(kk[3], a1, b0[2], b0[3]);
        mma16816(kk[4], a1, b1[0], b1[1]);
        mma16816(kk[5], a1, b1[2], b1[3]);
        if (WANT_Q) {
            ldsm4(a0, q + am + c);
            ldsm4(a1, q + am + 16 * pitch + c);
            mma16816(qk[0], a0, b0[0], b0[1]);
            mma16816(qk[1], a0, b0[2], b0[3]);
            mma16816(qk[2], a1, b0[0], b0[1]);
            mma16816(qk[3], a1, b0[2], b0[3]);
            mma16816(qk[4], a1, b1[0], b1[1]);
            mma16816(qk[5], a1, b1[2], b1[3]);
        }
    }
}

// One chunk's inputs for the chain, made by one warp:
//   K' , Q'   keys and queries scaled per row (inverse scales ik, iq)
//   X         (I + A)^-1, A[r][s] = D[r][s] (k_r . k_s) b, s < r, as fp16 hi + lo;
//             b = beta_s (forward: N = X (V - Gamma K S), U = beta N) or
//             b = beta_r (adjoint:  E = X^T dU, dR = beta E);
//             D[r][s] = exp(G_r - G_s), G the running sum of the log-decays
//   P         D[r][s] (q'_r . k'_s), s <= r, in the scaled units, fp16 (hi + lo)
//   scalars   ik, Gamma ik, exp(G_end - G) ik, beta, iq, Gamma iq; MISC[0] = exp(G_end)
// The inverse: the two 16x16 diagonal blocks by forward substitution in fp32 (one column
// per lane, both blocks at once), the block below them as -X22 A21 X11 in split products.
//
// The warp copies the chunk's rows into the (free) stage, lane r row r, and scales keys
// and queries in place.
struct ChunkSource {   // one (sequence, head): pointers to its first row
    const __nv_bfloat16 *k, *q, *v, *g, *beta;
    int64_t kstride, vstride, gstride;
    int len;
};

template <int DK, int W, bool ADJ, bool WANT_Q>
__device__ __forceinline__ bool produce_chunk(const ChunkSource &c, int t, unsigned char *stage,
                                              float *scratch, uint64_t *landed, uint32_t parity,
                                              uint32_t *err, uint32_t epoch,
                                              volatile uint32_t *abort) {
    using L = Stage<DK, W, ADJ>;
    const int lane = threadIdx.x & 31, valid = min(kChunk, c.len - t);
    const uint32_t sb = smem_u32(stage);
    float *scal = reinterpret_cast<float *>(stage + L::S);

    fence_proxy_async_shared();
    if (lane == 0)
        mbar_arrive_expect_tx(landed, (uint32_t)(valid * (DK * 2 * (WANT_Q ? 2 : 1) + W * 2)));
    __syncwarp();
    float g = 0.f, bt = 0.f;
    if (lane < valid) {
        const int64_t row = t + lane;
        bulk_row(sb + L::K + lane * L::KP, c.k + row * c.kstride, DK * 2, landed);
        if (WANT_Q) bulk_row(sb + L::Q + lane * L::KP, c.q + row * c.kstride, DK * 2, landed);
        bulk_row(sb + L::V + lane * L::VP, c.v + row * c.vstride, W * 2, landed);
        g = fmaxf(__bfloat162float(c.g[row * c.gstride]), kMinLogDecay);
        bt = __bfloat162float(c.beta[row * c.gstride]);
    } else {
        for (int i = 0; i < W * 2; i += 16)
            *reinterpret_cast<uint4 *>(stage + L::V + lane * L::VP + i) = make_uint4(0, 0, 0, 0);
    }
    // running sum in 64 bits: the decay between far rows is a difference of long sums
    double G = (double)g;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
        const double o = __shfl_up_sync(0xffffffffu, G, m);
        if (lane >= m) G += o;
    }
    const double Gend = __shfl_sync(0xffffffffu, G, 31);
    const float into = expf((float)G), out = expf((float)(Gend - G));

    // this lane's rows lane/4 + 8i and columns 2(lane%4) + 8j + {0, 1} of a 32 x 32 matrix:
    // the 16x16 blocks on and below the diagonal as six m16n8 tiles, tile t of row block
    // (t > 1) and columns 8 (t or t - 2)
    constexpr int AP = 20;   // fp32 row pitch of a diagonal block of A in the scratch
    const int r0 = lane >> 2, c0 = 2 * (lane & 3);
    float D[6][4];
    {
        // exponents of two, as a high and a low part: far sums cancel exactly
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
            }
    }
    if (!warp_wait(landed, parity, err, epoch, abort)) return false;
    float inv[2];
#pragma unroll 1
    for (int i = 0; i < (WANT_Q ? 2 : 1); ++i) {
        const float x = scale_row<DK>(sb + (i ? L::Q : L::K), L::KP, lane < valid);
        inv[0] = i ? inv[0] : x;
        inv[1] = x;
    }
    __syncwarp();
    const float ik = inv[0];
    scal[L::IK * kChunk + lane] = ik;
    scal[L::CK * kChunk + lane] = into * ik;
    scal[L::OK * kChunk + lane] = out * ik;
    scal[L::BETA * kChunk + lane] = bt;
    if (WANT_Q) {
        scal[L::IQ * kChunk + lane] = inv[1];
        scal[L::CQ * kChunk + lane] = into * inv[1];
    }
    if (lane == 31) scal[L::MISC * kChunk] = into;

    float acc[6][4], qk[6][4];
    gram_lower<DK, WANT_Q>(acc, qk, sb + L::K, sb + L::Q, L::KP);
    {
        const float wr_ = ADJ ? ik * bt : ik, ws_ = ADJ ? ik : ik * bt;
        float wr[4], ws[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) wr[i] = __shfl_sync(0xffffffffu, wr_, r0 + 8 * i);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            ws[j] = __shfl_sync(0xffffffffu, ws_, c0 + 8 * (j >> 1) + (j & 1));
#pragma unroll
        for (int t = 0; t < 6; ++t)
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const int i = (t < 2 ? 0 : 2) + (x >> 1), j = (t < 2 ? t : t - 2) * 2 + (x & 1);
                acc[t][x] *= D[t][x] * wr[i] * ws[j];
            }
    }
    // diagonal blocks to the scratch; A21 as fp16 hi + lo where X21 will stand
#pragma unroll
    for (int t = 0; t < 6; ++t)
#pragma unroll
        for (int x = 0; x < 4; x += 2) {
            const int r = r0 + (x >> 1) * 8;   // within the row block
            if (t == 2 || t == 3) {
                uint32_t hi, lo;
                split_half(acc[t][x], acc[t][x + 1], hi, lo);
                const int at = (16 + r) * L::XP + ((t - 2) * 8 + c0) * 2;
                *reinterpret_cast<uint32_t *>(stage + L::XH + at) = hi;
                *reinterpret_cast<uint32_t *>(stage + L::XL + at) = lo;
            } else {
                const int s = (t & 1) * 8 + c0;
                *reinterpret_cast<float2 *>(scratch + (t < 2 ? 0 : 16 * AP) + r * AP + s) =
                    make_float2(acc[t][x], acc[t][x + 1]);
            }
        }
    if (WANT_Q) {
#pragma unroll
        for (int t = 0; t < 6; ++t)
#pragma unroll
            for (int x = 0; x < 4; x += 2) {
                const int r = (t < 2 ? 0 : 16) + r0 + (x >> 1) * 8;
                const int s = (t < 2 ? t : t - 2) * 8 + c0;
                uint32_t hi, lo;
                split_half(qk[t][x] * D[t][x], qk[t][x + 1] * D[t][x + 1], hi, lo);
                *reinterpret_cast<uint32_t *>(stage + L::P + r * L::XP + s * 2) = hi;
                if (ADJ) *reinterpret_cast<uint32_t *>(stage + L::PL + r * L::XP + s * 2) = lo;
            }
    }
    __syncwarp();
    {   // column lane % 16 of (I + A)^-1 of diagonal block lane / 16
        const float *A = scratch + (lane >> 4) * 16 * AP;
        unsigned char *xh = stage + L::XH + (lane >> 4) * (16 * L::XP + 32) + (lane & 15) * 2;
        float x[16];
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            float a0 = r == (lane & 15) ? 1.f : 0.f, a1 = 0.f;
            const float4 *row = reinterpret_cast<const float4 *>(A + r * AP);
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
            *reinterpret_cast<__half *>(xh + r * L::XP) = h;
            *reinterpret_cast<__half *>(xh + (L::XL - L::XH) + r * L::XP) =
                __float2half_rn(x[r] - __half2float(h));
        }
    }
    __syncwarp();
    {   // X21 = -(X22 A21) X11
        const uint32_t xh = sb + L::XH, xl = sb + L::XL;
        const int am = (16 + (lane & 15)) * L::XP + (lane >> 4) * 16;   // rows 16.., as [m][k]
        const int bt = (lane & 15) * L::XP + (lane >> 4) * 16;          // as [k][n], transposed
        uint32_t ah[4], al[4], bh[4], bl[4];
        ldsm4(ah, xh + am + 32);
        ldsm4(al, xl + am + 32);
        ldsm4_t(bh, xh + bt + 16 * L::XP);
        ldsm4_t(bl, xl + bt + 16 * L::XP);
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
                const int at = (16 + r0 + (x >> 1) * 8) * L::XP + (8 * t + c0) * 2;
                *reinterpret_cast<uint32_t *>(stage + L::XH + at) = hi;
                *reinterpret_cast<uint32_t *>(stage + L::XL + at) = lo;
            }
        }
    }
    __syncwarp();
    return true;
}

}  // namespace gdr
}  // namespace kda
