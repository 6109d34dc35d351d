// Device helpers shared by the gated-delta-rule kernels: warp matrix products,
// the two-term fp16 split of fp32 operands, sequence bounds, and the work of a
// producer warp (one chunk's scaled keys and queries, their Gram products and
// the unit-lower-triangular inverse).
#pragma once

#include "kda_common.cuh"
#include "kda_launch.h"
#include "kda_tma.h"

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

// One box of 32 rows (tokens) of one head, through a tensor map over [rows, heads, D] passed as a
// __grid_constant__ parameter; its bytes complete the mbarrier's phase.  No multicast.
__device__ __forceinline__ void tma_rows(uint32_t dst, const CUtensorMap *map, int channel, int head,
                                         int row, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(channel), "r"(head), "r"(row), "r"(smem_u32(bar))
        : "memory");
}
// Orders this thread's earlier shared-memory accesses before later bulk copies of it.
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

// Zero the tokens from `valid` on in four transposed 8x8 bf16 fragments: the first two hold tokens t
// and t + 1 of this lane, the others t + 8 and t + 9.
__device__ __forceinline__ void clear_rows(uint32_t (&v)[4], int t, int valid) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int first = t + (i >> 1) * 8;
        if (first >= valid) v[i] = 0u;
        else if (first + 1 >= valid) v[i] &= 0xffffu;
    }
}

// Wait of a whole warp with the library's bounds: every lane takes the same way.  The bounded
// loop stays out of line: the warps of these kernels run different code side by side, and what
// they run together has to fit the instruction cache (see Pipe).
static __device__ __noinline__ bool warp_wait_long(uint64_t *bar, uint32_t parity, uint32_t *err,
                                            uint32_t epoch, volatile uint32_t *abort) {
    const bool ok = mbar_wait_abortable(bar, parity, err, epoch, abort);
    return __all_sync(0xffffffffu, ok);
}
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, uint32_t *err,
                                          uint32_t epoch, volatile uint32_t *abort) {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    return warp_wait_long(bar, parity, err, epoch, abort);
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
// Byte offsets inside one stage.  Rows are padded by 16 bytes, so the eight rows of an
// ldmatrix lie in different banks.  The values, which differ between the slices of a head, come
// last.
template <int DK, int W, bool PLO>
struct Stage {
    static constexpr int KP = DK * 2 + 16;       // keys, queries: fp16 [32][DK]
    static constexpr int XP = kChunk * 2 + 16;   // 32 x 32 fp16 matrices
    static constexpr int PANEL = W < 64 ? W : 64;   // columns of a tile of the values
    static constexpr int K = 0;
    static constexpr int XH = K + kChunk * KP;
    static constexpr int XL = XH + kChunk * XP;
    static constexpr int S = XL + kChunk * XP;   // per-row scalars, 8 x 32 fp32
    static constexpr int P = S + 8 * kChunk * 4;
    static constexpr int PL = P + kChunk * XP;   // low part of P (adjoint only)
    static constexpr int Q = PL + (PLO ? kChunk * XP : 0);
    static constexpr int SHARED_END = Q + kChunk * KP;
    static constexpr int V = (SHARED_END + 1023) / 1024 * 1024;
    static constexpr int VBYTES = kChunk * W * 2;
    static constexpr int BYTES = (V + VBYTES + 1023) / 1024 * 1024;
    // 16-byte piece c of row r of the values (or output gradients), bf16 as the TMA writes them:
    // panels of 64 columns with the 128-byte swizzle, or one plain panel of 32
    static __device__ __forceinline__ int v_at(int r, int c) {
        return V + (W < 64 ? r * 64 + c * 16 : (c >> 3) * 4096 + r * 128 + (((c & 7) ^ (r & 7)) << 4));
    }
    // rows of the scalar block
    enum { IK = 0, CK = 1, OK = 2, BETA = 3, IQ = 4, CQ = 5, MISC = 6 };
};

// Lane r scales row r of a raw tile by the power of two that puts its largest element in [1, 2)
// and stores it as fp16 (exact but for elements below 2^-17 of the row's largest); rows from
// `valid` on become zeros.  Returns 2^-e.  The raw tile is bf16 in panels of 64 channels with
// the 128-byte swizzle, the result has padded rows: either way the lanes' 16-byte pieces lie in
// different banks.
template <int D>
__device__ __forceinline__ float scale_row(uint32_t raw, uint32_t tile, int pitch, bool valid) {
    const int lane = threadIdx.x & 31;
    raw += lane * 128;
    tile += lane * pitch;
    const uint32_t turn = (lane & 7) << 4;
    __nv_bfloat162 m = __floats2bfloat162_rn(0.f, 0.f);
#pragma unroll 1
    for (int p = 0; p < D / 64; ++p)
#pragma unroll 4
        for (int c = 0; c < 128; c += 16) {
            uint32_t w[4];
            asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                         : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                         : "r"(raw + p * 4096 + (c ^ turn))
                         : "memory");
#pragma unroll
            for (int j = 0; j < 4; ++j)
                m = __hmax2(m, __habs2(reinterpret_cast<const __nv_bfloat162 &>(w[j])));
        }
    const float top = fmaxf(__low2float(m), __high2float(m));
    int e = (int)(__float_as_uint(top) >> 23);
    e = valid ? min(max(e, 1), 253) : 1;
    const float sc = __uint_as_float((uint32_t)(254 - e) << 23);
#pragma unroll 1
    for (int p = 0; p < D / 64; ++p)
#pragma unroll 4
        for (int c = 0; c < 128; c += 16) {
            uint32_t w[4], h[4];
            asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                         : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                         : "r"(raw + p * 4096 + (c ^ turn))
                         : "memory");
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                h[j] = pack_half(__uint_as_float(w[j] << 16) * sc,
                                 __uint_as_float(w[j] & 0xffff0000u) * sc);
                if (!valid) h[j] = 0u;
            }
            asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(tile + p * 128 + c), "r"(h[0]),
                         "r"(h[1]), "r"(h[2]), "r"(h[3])
                         : "memory");
        }
    return __uint_as_float((uint32_t)e << 23);
}

__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Lower triangle (16x16 blocks on and below the diagonal) of M N^T for scaled [32][D] tiles:
// accumulator tiles (row block, column tile) = (0,0) (0,1) (1,0..3).
template <int D>
__device__ __forceinline__ void gram_lower(float (&acc)[6][4], uint32_t m, uint32_t n, int pitch) {
    const int lane = threadIdx.x & 31;
    m += (lane & 15) * pitch + (lane >> 4) * 16;
    n += ((lane & 7) + ((lane >> 4) & 1) * 8) * pitch + ((lane >> 3) & 1) * 16;
#pragma unroll
    for (int i = 0; i < 6; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = 0.f;
#pragma unroll 2
    for (int c = 0; c < D * 2; c += 32) {
        uint32_t a0[4], a1[4], b0[4], b1[4];
        ldsm4(b0, n + c);
        ldsm4(b1, n + 16 * pitch + c);
        ldsm4(a0, m + c);
        ldsm4(a1, m + 16 * pitch + c);
        mma16816(acc[0], a0, b0[0], b0[1]);
        mma16816(acc[1], a0, b0[2], b0[3]);
        mma16816(acc[2], a1, b0[0], b0[1]);
        mma16816(acc[3], a1, b0[2], b0[3]);
        mma16816(acc[4], a1, b1[0], b1[1]);
        mma16816(acc[5], a1, b1[2], b1[3]);
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
// A team of TW warps makes a chunk; with two warps the second one has the queries and P.  The
// chunk's keys and queries come by TMA into the team's raw tiles while the chunk before is worked
// on.
struct alignas(64) Maps {   // tensor maps over the whole tensors
    CUtensorMap k, q, v;
};
struct ChunkSource {   // one (sequence, head)
    const Maps *maps;
    const __nv_bfloat16 *g, *beta;   // at its first row
    int row, kh, vh, column;         // first row; key and value head; first value column
    int64_t gstride;
    int len;
};

template <int TW>
__device__ __forceinline__ void team_sync(int id) {
    if (TW == 1) __syncwarp();
    else asm volatile("bar.sync %0, %1;" ::"r"(id), "n"(TW * 32) : "memory");
}

template <int W>
__device__ __forceinline__ void fetch_values(const ChunkSource &c, int t, uint32_t dst, uint64_t *bar) {
    constexpr int PANEL = W < 64 ? W : 64;
#pragma unroll
    for (int p = 0; p < W; p += PANEL)
        tma_rows(dst + p * kChunk * 2, &c.maps->v, c.column + p, c.vh, c.row + t, bar);
}

// A producer warp's view of the chunk that comes next.
struct NextChunk {
    float g, beta;   // of row `lane`
};
// Start the copies of the chunk at row t: keys by role 0, queries by role 1 (or both by a lone
// warp).  The raw tiles are free: every lane of the team has read them.
template <int DK, bool WANT_Q, int TW>
__device__ __forceinline__ void fetch_chunk(const ChunkSource &c, int t, uint32_t raw, uint64_t *landed,
                                            int role, NextChunk &next) {
    const int lane = threadIdx.x & 31;
    const bool keys = TW == 1 || role == 0, queries = WANT_Q && (TW == 1 || role == 1);
    if (lane == 0) {
        mbar_arrive_expect_tx(landed, kChunk * DK * 2 * ((keys ? 1 : 0) + (queries ? 1 : 0)));
#pragma unroll
        for (int p = 0; p < DK / 64; ++p) {
            if (keys) tma_rows(raw + p * 4096, &c.maps->k, p * 64, c.kh, c.row + t, landed);
            if (queries) tma_rows(raw + (DK / 64 + p) * 4096, &c.maps->q, p * 64, c.kh, c.row + t, landed);
        }
    }
    next.g = next.beta = 0.f;
    if (lane < c.len - t) {
        next.g = fmaxf(__bfloat162float(c.g[(t + lane) * c.gstride]), kMinLogDecay);
        next.beta = __bfloat162float(c.beta[(t + lane) * c.gstride]);
    }
}

// `before_stage` waits for the stage to be free; `scaled` runs when this warp's part of the scaled
// keys and queries is in the stage and the raw tiles are free.  False if a wait ran out (the
// team's warps all come back).
template <int DK, int W, bool ADJ, bool WANT_Q, int TW, typename Free, typename Scaled>
__device__ __forceinline__ bool produce_chunk(const ChunkSource &c, int t, unsigned char *stage,
                                              uint32_t raw, float *scratch, uint64_t *landed,
                                              uint32_t parity, int role, int team_bar, NextChunk now,
                                              uint32_t *err, uint32_t epoch, volatile uint32_t *abort,
                                              Free before_stage, Scaled scaled) {
    using L = Stage<DK, W, ADJ>;
    const int lane = threadIdx.x & 31, valid = min(kChunk, c.len - t);
    const bool keys = TW == 1 || role == 0, queries = WANT_Q && (TW == 1 || role == 1);
    const uint32_t sb = smem_u32(stage);
    float *scal = reinterpret_cast<float *>(stage + L::S);
    const float g = now.g, bt = now.beta;
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
    const bool landed_ok = warp_wait(landed, parity, err, epoch, abort);
    const bool ok = before_stage() && landed_ok;
    // keys (pass 0) and queries (pass 1), whichever this warp has
    const int first = keys ? 0 : 1, last = queries ? 1 : 0;
    float ik = 1.f;
#pragma unroll 1
    for (int pass = first; pass <= last; ++pass) {
        const float inv = scale_row<DK>(raw + pass * kChunk * DK * 2, sb + (pass ? L::Q : L::K), L::KP,
                                        lane < valid);
        float *at = scal + lane;
        at[(pass ? L::IQ : L::IK) * kChunk] = inv;
        at[(pass ? L::CQ : L::CK) * kChunk] = into * inv;
        if (pass == 0) {
            ik = inv;
            at[L::OK * kChunk] = out * inv;
            at[L::BETA * kChunk] = bt;
            if (lane == 31) scal[L::MISC * kChunk] = into;
        }
    }
    fence_proxy_async_shared();   // before the copies of these tiles, and into the raw ones
    team_sync<TW>(team_bar);      // both warps come here whether the waits ran out or not
    if (!ok || *abort) return false;
    scaled();

    float acc[6][4];
#pragma unroll 1
    for (int pass = last; pass >= first; --pass) {
        gram_lower<DK>(acc, sb + (pass ? L::Q : L::K), sb + L::K, L::KP);
        if (pass == 0) break;
#pragma unroll
        for (int i = 0; i < 6; ++i)
#pragma unroll
            for (int x = 0; x < 4; x += 2) {
                const int r = (i < 2 ? 0 : 16) + r0 + (x >> 1) * 8;
                const int s = (i < 2 ? i : i - 2) * 8 + c0;
                uint32_t hi, lo;
                split_half(acc[i][x] * D[i][x], acc[i][x + 1] * D[i][x + 1], hi, lo);
                *reinterpret_cast<uint32_t *>(stage + L::P + r * L::XP + s * 2) = hi;
                if (ADJ) *reinterpret_cast<uint32_t *>(stage + L::PL + r * L::XP + s * 2) = lo;
            }
    }
    if (!keys) {
        __syncwarp();
        return true;
    }
    {
        const float wr_ = ADJ ? ik * bt : ik, ws_ = ADJ ? ik : ik * bt;
        float wr[4], ws[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) wr[i] = __shfl_sync(0xffffffffu, wr_, r0 + 8 * i);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            ws[j] = __shfl_sync(0xffffffffu, ws_, c0 + 8 * (j >> 1) + (j & 1));
#pragma unroll
        for (int i = 0; i < 6; ++i)
#pragma unroll
            for (int x = 0; x < 4; ++x)
                acc[i][x] *= D[i][x] * wr[(i < 2 ? 0 : 2) + (x >> 1)] * ws[(i < 2 ? i : i - 2) * 2 + (x & 1)];
    }
    // diagonal blocks to the scratch; A21 as fp16 hi + lo where X21 will stand
#pragma unroll
    for (int i = 0; i < 6; ++i)
#pragma unroll
        for (int x = 0; x < 4; x += 2) {
            const int r = r0 + (x >> 1) * 8;   // within the row block
            if (i == 2 || i == 3) {
                uint32_t hi, lo;
                split_half(acc[i][x], acc[i][x + 1], hi, lo);
                const int at = (16 + r) * L::XP + ((i - 2) * 8 + c0) * 2;
                *reinterpret_cast<uint32_t *>(stage + L::XH + at) = hi;
                *reinterpret_cast<uint32_t *>(stage + L::XL + at) = lo;
            } else {
                const int s = (i & 1) * 8 + c0;
                *reinterpret_cast<float2 *>(scratch + (i < 2 ? 0 : 16 * AP) + r * AP + s) =
                    make_float2(acc[i][x], acc[i][x + 1]);
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

// ---------------------------------------------------------------- clusters
__device__ __forceinline__ uint32_t map_to_cta(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
__device__ __forceinline__ void mbar_arrive_cluster(uint64_t *bar, uint32_t rank) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(
                     map_to_cta(smem_u32(bar), rank))
                 : "memory");
}
__device__ __forceinline__ void cluster_arrive() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// `bytes` of this CTA's shared memory to the same place in another CTA of the cluster; they
// complete that CTA's copy of the barrier.
__device__ __forceinline__ void bulk_to_cta(uint32_t addr, uint32_t bytes, uint64_t *bar, uint32_t rank) {
    asm volatile(
        "cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
            map_to_cta(addr, rank)),
        "r"(addr), "r"(bytes), "r"(map_to_cta(smem_u32(bar), rank))
        : "memory");
}

// ---------------------------------------------------------------- the chain kernels' pipeline
// NCW groups of 16 value columns per CTA, KS warps per group (each with dk / KS channels), and
// the CTAs of a head's CL slices as one cluster.  Chunks go through a ring of ST stages; chunk i
// is made by CTA i % CL of the cluster, which copies everything but the values to the other CTAs,
// so that a head's keys, queries and inverses are worked on once and not once per slice.
//
// Barriers of a stage: `landed` (the raw tiles of the team that makes it), `full` (everything is
// there), `empty` (the chain warps of all CTAs are through with it; used in the producing CTA), and
// for CL > 1 `vempty` (this CTA's are: the value loader waits for it and tells the producing CTA).
template <int DK, int NCW, int KS, int CL, bool ADJ, bool WANT_Q, int XF>
struct Pipe {
    static constexpr int W = NCW * 16;
    using L = Stage<DK, W, ADJ>;
    // stages, and a team for each that this CTA makes: a chunk takes a lone warp about three times
    // as long as the chain
    static constexpr int ST = NCW == 8 && ADJ ? 3 : 4, NT = ST / CL;
    static constexpr int TW = CL > 1 && WANT_Q ? 2 : 1;
    static constexpr int CHAIN = NCW * KS, WARPS = CHAIN + NT * TW + (CL > 1 ? 1 : 0);
    // what the other CTAs get: keys; inverses and scalars; P and queries
    static constexpr int SHARED = WANT_Q ? L::SHARED_END : L::P;
    static constexpr int RAWB = kChunk * DK * 2 * (WANT_Q ? 2 : 1);
    static constexpr int OP = 48;                         // row pitch of a 32 x 16 output tile
    static constexpr int RAW = ST * L::BYTES;
    static constexpr int SCRATCH = RAW + NT * RAWB;
    static constexpr int OUT = SCRATCH + NT * kScratch * 4;
    static constexpr int SWAP = OUT + NCW * kChunk * OP;
    static constexpr int BARS = SWAP + (KS == 2 ? NCW * 2 * 2 * XF * 32 * 4 : 0);
    static constexpr int BYTES = BARS + (4 * ST + 2 * NCW) * 8 + 16;
    static_assert(ST % CL == 0 && BYTES <= 227 * 1024, "stages and shared memory");

    unsigned char *smem;
    uint64_t *full, *empty, *landed, *vempty, *swapped;
    volatile uint32_t *abort;
    uint32_t *err;
    uint32_t epoch, rank;

    __device__ __forceinline__ Pipe(unsigned char *s, uint32_t *e, uint32_t ep, int slice)
        : smem(s), err(e), epoch(ep), rank(slice) {
        full = reinterpret_cast<uint64_t *>(smem + BARS);
        empty = full + ST, landed = empty + ST, vempty = landed + ST, swapped = vempty + ST;
        abort = reinterpret_cast<volatile uint32_t *>(swapped + 2 * NCW);
        if (threadIdx.x == 0) {
            for (int i = 0; i < ST; ++i) {
                mbar_init(full + i, 1 + TW);   // the values' copy, and each warp of the team
                mbar_init(empty + i, CL == 1 ? CHAIN : CL);
                mbar_init(landed + i, TW);
                mbar_init(vempty + i, CHAIN);
            }
            for (int i = 0; i < 2 * NCW; ++i) mbar_init(swapped + i, 1);
            mbar_fence_init();
            *abort = 0u;
        }
        __syncthreads();
        if (CL > 1) {
            cluster_arrive();
            cluster_wait();
        }
    }
    __device__ __forceinline__ bool wait(uint64_t *bar, uint32_t parity) const {
        return warp_wait(bar, parity, err, epoch, abort);
    }
    __device__ __forceinline__ unsigned char *stage(int i) const { return smem + i * L::BYTES; }

    // bytes [from, to) of stage s to the other CTAs (one thread, after a proxy fence of the writers)
    __device__ __forceinline__ void share(int s, int from, int to) const {
#pragma unroll 1
        for (uint32_t r = 1; r < CL; ++r)
            bulk_to_cta(smem_u32(stage(s)) + from, to - from, full + s, (rank + r) % CL);
    }

    // The part of a warp that is not a chain warp.  REVERSE: chunk i of the order is the i-th
    // from the sequence's end.
    template <bool REVERSE>
    __device__ __forceinline__ void produce(const ChunkSource &src, int chunks) const {
        const int lane = threadIdx.x & 31, w = (threadIdx.x >> 5) - CHAIN;
        auto row = [&](int i) { return (REVERSE ? chunks - 1 - i : i) * kChunk; };
        if (w == NT * TW) {   // value loader (CL > 1)
            for (int i = 0, s = 0, use = 0; i < chunks; ++i) {
                if (use > 0) {
                    if (!wait(vempty + s, (use - 1) & 1)) return;
                    // for this CTA's chain warps: their own arrival at cluster scope would wait
                    // for their stores to global memory (1800 cycles a chunk)
                    if (lane == 0) mbar_arrive_cluster(empty + s, s % CL);
                }
                if (lane == 0) {
                    mbar_arrive_expect_tx(full + s, L::VBYTES);
                    fetch_values<W>(src, row(i), smem_u32(stage(s)) + L::V, full + s);
                    if (s % CL != (int)rank) {   // for the team of the producing CTA
                        mbar_arrive_expect_tx(full + s, SHARED);
                        if (TW > 1) mbar_arrive(full + s);
                    }
                }
                __syncwarp();
                if (++s == ST) s = 0, ++use;
            }
            return;
        }
        const int team = w / TW, role = w % TW, s = (int)rank + CL * team;
        const uint32_t raw = smem_u32(smem + RAW + team * RAWB);
        float *scratch = reinterpret_cast<float *>(smem + SCRATCH) + team * kScratch;
        NextChunk next;
        if (s < chunks) fetch_chunk<DK, WANT_Q, TW>(src, row(s), raw, landed + s, role, next);
        for (int i = s, use = 0; i < chunks; i += ST, ++use) {
            const NextChunk now = next;
            const bool ok = produce_chunk<DK, W, ADJ, WANT_Q, TW>(
                src, row(i), stage(s), raw, scratch, landed + s, use & 1, role, 1 + team, now, err, epoch,
                abort,
                [&] {
                    const bool free = use == 0 || wait(empty + s, (use - 1) & 1);
                    if (CL == 1 && free && role == 0 && lane == 0) {
                        mbar_arrive_expect_tx(full + s, L::VBYTES);
                        fetch_values<W>(src, row(i), smem_u32(stage(s)) + L::V, full + s);
                    }
                    return free;
                },
                [&] {
                    if (i + ST < chunks)
                        fetch_chunk<DK, WANT_Q, TW>(src, row(i + ST), raw, landed + s, role, next);
                    if (CL > 1 && lane == 0) {
                        if (role == 0) share(s, L::K, L::XH);
                        if (WANT_Q && role == TW - 1) share(s, L::Q, L::SHARED_END);
                    }
                });
            if (!ok) return;
            if (CL > 1) fence_proxy_async_shared();
            __syncwarp();
            if (lane == 0) {
                if (CL > 1) {
                    if (role == 0) share(s, L::XH, L::P);
                    if (WANT_Q && role == TW - 1) share(s, L::P, L::Q);
                }
                mbar_arrive(full + s);
            }
        }
    }
    // A chain warp is through with stage s.
    __device__ __forceinline__ void release(int s) const {
        __syncwarp();
        if ((threadIdx.x & 31) == 0) mbar_arrive(CL == 1 ? empty + s : vempty + s);
    }
    // No CTA of a cluster leaves while another may write to its shared memory.
    __device__ __forceinline__ void finish() const {
        if (CL > 1) {
            __syncwarp();
            cluster_arrive();
            cluster_wait();
        }
    }
};

// Launch of a chain kernel over `rows` rows: `cluster` consecutive CTAs of `cols` columns each are
// one head's slices.  v: the values, or the output gradients in their place.
template <typename Args>
inline cudaError_t launch_pipe(void (*kernel)(const Maps, const Args), const Args &a, const void *k, const void *q,
                               const void *v, int64_t rows, int dk, int cols, int64_t ctas, int threads,
                               int smem, int cluster, cudaStream_t st) {
    Maps maps = {};
    if (rows > 0) {   // with no rows nothing is loaded
        const bool narrow = cols < 64;
        if (!make_rows_heads_tmap(&maps.k, k, rows, a.Hk, dk, 64, kChunk, CU_TENSOR_MAP_SWIZZLE_128B) ||
            !make_rows_heads_tmap(&maps.q, q, rows, a.Hk, dk, 64, kChunk, CU_TENSOR_MAP_SWIZZLE_128B) ||
            !make_rows_heads_tmap(&maps.v, v, rows, a.H, a.dv, narrow ? cols : 64, kChunk,
                                  narrow ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B))
            return cudaErrorInvalidValue;
    }
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = st;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = (unsigned)cluster;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = cluster > 1 ? 1 : 0;
    e = cudaLaunchKernelEx(&cfg, kernel, maps, a);
    if (e == cudaSuccess) e = cudaGetLastError();
    Profiler::mark(st);
    return e;
}

}  // namespace gdr
}  // namespace kda
