// Gated delta rule, chunked, bf16: prefill, and the forward recomputation of the backward.
//
//     S_t = a_t (I - beta_t k_t k_t^T) S_{t-1} + beta_t k_t v_t^T,  a_t = exp(g_t),  o_t = S_t^T q_t
//
// A chunk of C = 32 tokens with G_r the running sum of g inside it, Gamma = exp(G),
// D[r][s] = exp(G_r - G_s):
//
//     N = X (V - Gamma K S),   X = (I + A)^-1,  A[r][s] = D[r][s] (k_r . k_s) beta_s, s < r
//     O = Gamma Q S + P (beta N),               P[r][s] = D[r][s] (q_r . k_s),        s <= r
//     S' = Gamma_C S + sum_s exp(G_C - G_s) k_s (beta N)_s^T
//
// With one decay per token and head every factor that exp makes is at most 1 (for g <= 0)
// and multiplies a whole row, so no operand is rescaled by a reciprocal.
//
// The value columns of S are independent of one another.  One warp keeps 16 of them as
// S^T [16 x dk] in its accumulator registers; the products K S, X (..) and K^T (..) of the
// transposed form take their left operand from the previous product's accumulators in
// place (an m16n8 accumulator pair is an m16k16 operand), so the chain over chunks never
// leaves the warp: no shared memory, no barrier between its products.  The right operands
// (K, Q, X, P) are the same for all columns; four to six producer warps make them in shared
// memory, each a chunk of its own, ahead of the chain.
//
// Precision: S, V - Gamma K S and beta N enter the products as fp16 hi + lo of the row
// scaled by a power of two (22 bits), K and Q are exact in fp16 after a power-of-two scale
// per row, so the state keeps fp32 accuracy (the final state is an fp32 output).  What
// only o depends on (S and beta N in its two products, P) is rounded once to fp16, 2^-12,
// below o's own rounding to bf16.
#include "gdr_common.cuh"
#include "gdr_launch.h"

namespace kda {
namespace gdr {

struct ChainArgs {
    const __nv_bfloat16 *q, *k, *v, *g, *beta;
    const float *state_in;
    const int32_t *cu;
    int64_t T, rows;
    int Hk, H, dv;
    __nv_bfloat16 *o;       // prefill
    float *state_out;       // prefill
    float *n_out;           // recomputation: N [rows, H, dv]
    float *blocks;          // recomputation: state before each 64-token block [.., H, dk, dv]
    float *tops;            // recomputation: largest |state| of each block's parts [.., H, dv/16, 2]
    int32_t *owners;        // recomputation: the sequence of each block
    uint32_t *err;
    uint32_t epoch;
};

// What a chain warp needs to finish a chunk's outputs, kept in registers so that with KS = 2
// they are finished inside the next chunk, while the two halves' warps wait for each other.
template <int KS>
struct ChunkOut {
    static constexpr int NTILE = 4 / KS, T0 = KS == 2 ? 16 : 32;   // token tiles; tokens of a warp
    uint32_t u[2][4], p[KS == 2 ? 2 : 3][4];
    float oq[NTILE][4], i0, i1;
    float2 cq[NTILE], iq[NTILE];

    // O = Gamma Q S + P U, both in the scaled units of Q'; rounded and written through `tile`.
    __device__ __forceinline__ void write(unsigned char *tile, int pitch, __nv_bfloat16 *dst,
                                          int64_t stride, int part, int valid) const {
        const int lane = threadIdx.x & 31;
        const int nrow = (lane & 7) + (lane >> 4) * 8, ncol = ((lane >> 3) & 1) * 16;
        float ou[NTILE][4];
#pragma unroll
        for (int t = 0; t < NTILE; ++t)
#pragma unroll
            for (int x = 0; x < 4; ++x) ou[t][x] = 0.f;
        // P is zero above the diagonal
        if (KS == 2) {
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) {   // part 0 has zeros for its second step
                mma16816(ou[0], u[ks], p[ks][0], p[ks][1]);
                mma16816(ou[1], u[ks], p[ks][2], p[ks][3]);
            }
        } else {
            mma16816(ou[0], u[0], p[0][0], p[0][1]);
            mma16816(ou[1], u[0], p[0][2], p[0][3]);
            mma16816(ou[NTILE - 2], u[0], p[1][0], p[1][1]);
            mma16816(ou[NTILE - 1], u[0], p[1][2], p[1][3]);
            mma16816(ou[NTILE - 2], u[1], p[KS == 2 ? 1 : 2][0], p[KS == 2 ? 1 : 2][1]);
            mma16816(ou[NTILE - 1], u[1], p[KS == 2 ? 1 : 2][2], p[KS == 2 ? 1 : 2][3]);
        }
        uint32_t pk[NTILE][2];
#pragma unroll
        for (int t = 0; t < NTILE; ++t) {
            const __nv_bfloat162 w0 = __floats2bfloat162_rn(cq[t].x * oq[t][0] + iq[t].x * (i0 * ou[t][0]),
                                                            cq[t].y * oq[t][1] + iq[t].y * (i0 * ou[t][1]));
            const __nv_bfloat162 w1 = __floats2bfloat162_rn(cq[t].x * oq[t][2] + iq[t].x * (i1 * ou[t][2]),
                                                            cq[t].y * oq[t][3] + iq[t].y * (i1 * ou[t][3]));
            pk[t][0] = reinterpret_cast<const uint32_t &>(w0);
            pk[t][1] = reinterpret_cast<const uint32_t &>(w1);
        }
        const int t0 = part * 16;   // 0 with KS = 1
        __syncwarp();               // the rows written before have been read out of the tile
#pragma unroll
        for (int t = 0; t < NTILE; t += 2)
            stsm4_t(smem_u32(tile) + (t0 + 8 * t + nrow) * pitch + ncol, pk[t][0], pk[t][1], pk[t + 1][0],
                    pk[t + 1][1]);
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 2 / KS; ++i) {
            const int tok = t0 + i * 16 + (lane >> 1);
            const uint4 w = *reinterpret_cast<const uint4 *>(tile + tok * pitch + (lane & 1) * 16);
            if (tok < valid) *reinterpret_cast<uint4 *>(dst + tok * stride + (lane & 1) * 8) = w;
        }
    }
};

// With KS = 2 the two warps of a column group add their partial K S (and Q S) through shared
// memory, compute N twice, and update their own halves of S: half the products per warp on the
// chain, for one exchange.
template <int DK, int NCW, int KS, int CL, bool REC>
__global__ void __launch_bounds__((Pipe<DK, NCW, KS, CL, false, !REC, 24>::WARPS * 32), 1)
    gdr_chain_kernel(const __grid_constant__ Maps maps, const __grid_constant__ ChainArgs a) {
    using M = Pipe<DK, NCW, KS, CL, false, !REC, 24>;
    using L = typename M::L;
    constexpr int W = M::W, NC = DK / 8 / KS, NK = DK / 16 / KS, XF = 24;
    extern __shared__ __align__(1024) unsigned char smem[];

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int slices = a.dv / W;
    const int slice = blockIdx.x % slices, unit = blockIdx.x / slices;
    const int h = unit % a.H, n = unit / a.H, hk = h / (a.H / a.Hk);
    const Span span = sequence_span(a.cu, n, a.T);
    const int chunks = (span.len + kChunk - 1) / kChunk;
    if (REC && h == 0 && slice == 0)
        for (int i = threadIdx.x; 2 * i < chunks; i += blockDim.x)
            a.owners[first_block(span, n) + i] = n;
    const M pipe(smem, a.err, a.epoch, CL == 1 ? 0 : slice);

    if (warp >= M::CHAIN) {
        const ChunkSource src{&maps, a.g + span.row * a.H + h, a.beta + span.row * a.H + h,
                              (int)span.row, hk, h, slice * W, a.H, span.len};
        pipe.template produce<false>(src, chunks);
        pipe.finish();
        return;
    }

    // ---- chain: columns j0 .. j0 + 15 of this head's state, channels c0 .. c0 + dk/KS - 1
    const int group = warp / KS, part = warp % KS;
    const int j0 = slice * W + group * 16, jr = lane >> 2, tc = 2 * (lane & 3);
    const int c0 = part * (DK / KS);
    float s[NC][4];   // S^T: (column jr, channel c0 + 8i + tc), +1, (column jr + 8, ..)
    const int64_t state_off = ((int64_t)n * a.H + h) * DK * a.dv + (int64_t)(c0 + tc) * a.dv + j0 + jr;
    float sm0 = 0.f, sm1 = 0.f;   // this lane's largest |S| of its two columns
    {
        const float *in = a.state_in ? a.state_in + state_off : nullptr;
#pragma unroll
        for (int i = 0; i < NC; ++i) {
#pragma unroll
            for (int x = 0; x < 4; ++x)
                s[i][x] = in ? in[(int64_t)(8 * i + (x & 1)) * a.dv + (x >> 1) * 8] : 0.f;
            sm0 = fmaxf(sm0, fmaxf(fabsf(s[i][0]), fabsf(s[i][1])));
            sm1 = fmaxf(sm1, fmaxf(fabsf(s[i][2]), fabsf(s[i][3])));
        }
    }
    // per-lane parts of the ldmatrix addresses
    const int nrow = (lane & 7) + (lane >> 4) * 8, ncol = ((lane >> 3) & 1) * 16;   // [n][k] tiles
    const int trow = lane & 15, tcol = (lane >> 4) * 16;                            // [k][n] tiles
    unsigned char *out_tile = smem + M::OUT + group * kChunk * M::OP;
    const int64_t vstride = (int64_t)a.H * a.dv;
    ChunkOut<KS> out;
    bool ok = true;

    for (int ci = 0; ci < chunks; ++ci) {
        const int st = ci % M::ST;
        unsigned char *stage = pipe.stage(st);
        const uint32_t sb = smem_u32(stage);
        const float *scal = reinterpret_cast<const float *>(stage + L::S);
        const int64_t row = span.row + (int64_t)ci * kChunk;
        const int valid = span.len - ci * kChunk;

        // row scales of S
        float is0, is1;
        const float fs0 = row_scale(quad_max(sm0), is0), fs1 = row_scale(quad_max(sm1), is1);
        if (REC && (ci & 1) == 0) {
            const int64_t blk = (first_block(span, n) + ci / 2) * a.H + h;
            float *dst = a.blocks + blk * DK * a.dv + (int64_t)(c0 + tc) * a.dv + j0 + jr;
#pragma unroll
            for (int i = 0; i < NC; ++i)
#pragma unroll
                for (int x = 0; x < 4; ++x)
                    dst[(int64_t)(8 * i + (x & 1)) * a.dv + (x >> 1) * 8] = s[i][x];
            store_top(a.tops + (blk * (a.dv / 16) + j0 / 16) * 2, fmaxf(sm0, sm1), KS, part);
        }
        ok = pipe.wait(pipe.full + st, (ci / M::ST) & 1);
        if (!ok) break;

        // Y^T = S^T K'^T (two terms of S) and S^T Q'^T (the high term)
        float y[4][4], oq[4][4];
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int x = 0; x < 4; ++x) y[t][x] = oq[t][x] = 0.f;
#pragma unroll
        for (int kk = 0; kk < NK; ++kk) {
            uint32_t hi[4], lo[4], b0[4], b1[4];
            split_half(s[2 * kk][0] * fs0, s[2 * kk][1] * fs0, hi[0], lo[0]);
            split_half(s[2 * kk][2] * fs1, s[2 * kk][3] * fs1, hi[1], lo[1]);
            split_half(s[2 * kk + 1][0] * fs0, s[2 * kk + 1][1] * fs0, hi[2], lo[2]);
            split_half(s[2 * kk + 1][2] * fs1, s[2 * kk + 1][3] * fs1, hi[3], lo[3]);
            ldsm4(b0, sb + L::K + nrow * L::KP + ncol + c0 * 2 + kk * 32);
            ldsm4(b1, sb + L::K + (nrow + 16) * L::KP + ncol + c0 * 2 + kk * 32);
            mma16816(y[0], hi, b0[0], b0[1]);
            mma16816(y[1], hi, b0[2], b0[3]);
            mma16816(y[2], hi, b1[0], b1[1]);
            mma16816(y[3], hi, b1[2], b1[3]);
            mma16816(y[0], lo, b0[0], b0[1]);
            mma16816(y[1], lo, b0[2], b0[3]);
            mma16816(y[2], lo, b1[0], b1[1]);
            mma16816(y[3], lo, b1[2], b1[3]);
            if (!REC) {
                ldsm4(b0, sb + L::Q + nrow * L::KP + ncol + c0 * 2 + kk * 32);
                ldsm4(b1, sb + L::Q + (nrow + 16) * L::KP + ncol + c0 * 2 + kk * 32);
                mma16816(oq[0], hi, b0[0], b0[1]);
                mma16816(oq[1], hi, b0[2], b0[3]);
                mma16816(oq[2], hi, b1[0], b1[1]);
                mma16816(oq[3], hi, b1[2], b1[3]);
            }
        }
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            y[t][0] *= is0; y[t][1] *= is0; y[t][2] *= is1; y[t][3] *= is1;
            oq[t][0] *= is0; oq[t][1] *= is0; oq[t][2] *= is1; oq[t][3] *= is1;
        }
        if (KS == 2) {
            // add the other half's sums; of Q S each warp keeps 16 of the tokens.  Buffers
            // alternate: the other warp has read the ones of two chunks before by now.
            float4 *mine = reinterpret_cast<float4 *>(smem + M::SWAP) +
                           (((group * 2 + (ci & 1)) * 2 + part) * XF / 4) * 32 + lane;
            const float4 *other = mine + (part ? -1 : 1) * (XF / 4) * 32;
#pragma unroll
            for (int t = 0; t < 4; ++t) mine[t * 32] = make_float4(y[t][0], y[t][1], y[t][2], y[t][3]);
            if (!REC) {
#pragma unroll
                for (int t = 0; t < 2; ++t)
                    mine[(4 + t) * 32] = part ? make_float4(oq[t][0], oq[t][1], oq[t][2], oq[t][3])
                                              : make_float4(oq[t + 2][0], oq[t + 2][1],
                                                            oq[t + 2][2], oq[t + 2][3]);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(pipe.swapped + group * 2 + (part ^ 1));
            if (!REC && ci > 0)   // the chunk before, all of whose 32 rows are valid
                out.write(out_tile, M::OP, a.o + ((row - kChunk) * a.H + h) * a.dv + j0, vstride, part, kChunk);
            ok = pipe.wait(pipe.swapped + group * 2 + part, ci & 1);
            if (!ok) break;
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const float4 o = other[t * 32];
                y[t][0] += o.x; y[t][1] += o.y; y[t][2] += o.z; y[t][3] += o.w;
            }
            if (!REC) {
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    const float4 o = other[(4 + t) * 32];
#pragma unroll
                    for (int x = 0; x < 4; ++x) oq[t][x] = part ? oq[t + 2][x] : oq[t][x];
                    oq[t][0] += o.x; oq[t][1] += o.y; oq[t][2] += o.z; oq[t][3] += o.w;
                }
            }
        }
        // R = V - Gamma K S, this lane's tokens 8t + tc + {0, 1}
        float r[4][4], m0 = 0.f, m1 = 0.f;
#pragma unroll
        for (int t = 0; t < 4; t += 2) {
            uint32_t v[4];
            ldsm4_t(v, sb + L::v_at(8 * t + nrow, group * 2 + ((lane >> 3) & 1)));
            if (valid < kChunk) clear_rows(v, 8 * t + tc, valid);   // the rows behind the sequence's end
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const float2 c = *reinterpret_cast<const float2 *>(scal + L::CK * kChunk +
                                                                   8 * (t + u) + tc);
                r[t + u][0] = __uint_as_float(v[2 * u] << 16) - c.x * y[t + u][0];
                r[t + u][1] = __uint_as_float(v[2 * u] & 0xffff0000u) - c.y * y[t + u][1];
                r[t + u][2] = __uint_as_float(v[2 * u + 1] << 16) - c.x * y[t + u][2];
                r[t + u][3] = __uint_as_float(v[2 * u + 1] & 0xffff0000u) - c.y * y[t + u][3];
                m0 = fmaxf(m0, fmaxf(fabsf(r[t + u][0]), fabsf(r[t + u][1])));
                m1 = fmaxf(m1, fmaxf(fabsf(r[t + u][2]), fabsf(r[t + u][3])));
            }
        }
        // N^T = R^T X^T: three of the four products of the split operands
        float nn[4][4], nl[4][4];
        {
            float ir0, ir1;
            const float fr0 = row_scale(quad_max(m0), ir0), fr1 = row_scale(quad_max(m1), ir1);
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int x = 0; x < 4; ++x) nn[t][x] = nl[t][x] = 0.f;
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) {
                uint32_t hi[4], lo[4];
                split_half(r[2 * ks][0] * fr0, r[2 * ks][1] * fr0, hi[0], lo[0]);
                split_half(r[2 * ks][2] * fr1, r[2 * ks][3] * fr1, hi[1], lo[1]);
                split_half(r[2 * ks + 1][0] * fr0, r[2 * ks + 1][1] * fr0, hi[2], lo[2]);
                split_half(r[2 * ks + 1][2] * fr1, r[2 * ks + 1][3] * fr1, hi[3], lo[3]);
#pragma unroll
                for (int half = ks; half < 2; ++half) {   // X is zero above the diagonal
                    uint32_t xh[4], xl[4];
                    ldsm4(xh, sb + L::XH + (16 * half + nrow) * L::XP + ncol + ks * 32);
                    ldsm4(xl, sb + L::XL + (16 * half + nrow) * L::XP + ncol + ks * 32);
                    mma16816(nn[2 * half], hi, xh[0], xh[1]);
                    mma16816(nn[2 * half + 1], hi, xh[2], xh[3]);
                    mma16816(nl[2 * half], lo, xh[0], xh[1]);
                    mma16816(nl[2 * half + 1], lo, xh[2], xh[3]);
                    mma16816(nl[2 * half], hi, xl[0], xl[1]);
                    mma16816(nl[2 * half + 1], hi, xl[2], xl[3]);
                }
            }
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                nn[t][0] = (nn[t][0] + nl[t][0]) * ir0;
                nn[t][1] = (nn[t][1] + nl[t][1]) * ir0;
                nn[t][2] = (nn[t][2] + nl[t][2]) * ir1;
                nn[t][3] = (nn[t][3] + nl[t][3]) * ir1;
            }
        }
        if (REC) {
            float *dst = a.n_out + (row * a.H + h) * a.dv + j0 + jr;
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const int tok = 8 * t + tc + (x & 1);
                    if (tok < valid && (KS == 1 || t / 2 == part)) dst[tok * vstride + (x >> 1) * 8] = nn[t][x];
                }
        }
        // U = beta N in the scaled units of K', and with the decay to the chunk's end
        float m2 = 0.f, m3 = 0.f;
        m0 = m1 = 0.f;
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const float2 b = *reinterpret_cast<const float2 *>(scal + L::BETA * kChunk + 8 * t + tc);
            const float2 e = *reinterpret_cast<const float2 *>(scal + L::OK * kChunk + 8 * t + tc);
            const float2 k = *reinterpret_cast<const float2 *>(scal + L::IK * kChunk + 8 * t + tc);
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const float u = nn[t][x] * ((x & 1) ? b.y : b.x);
                r[t][x] = u * ((x & 1) ? e.y : e.x);
                nn[t][x] = u * ((x & 1) ? k.y : k.x);
            }
            m0 = fmaxf(m0, fmaxf(fabsf(r[t][0]), fabsf(r[t][1])));
            m1 = fmaxf(m1, fmaxf(fabsf(r[t][2]), fabsf(r[t][3])));
            m2 = fmaxf(m2, fmaxf(fabsf(nn[t][0]), fabsf(nn[t][1])));
            m3 = fmaxf(m3, fmaxf(fabsf(nn[t][2]), fabsf(nn[t][3])));
        }
        // S' = Gamma_C S + (decayed U)^T K'
        {
            float iu0, iu1;
            const float fu0 = row_scale(quad_max(m0), iu0), fu1 = row_scale(quad_max(m1), iu1);
            const float gend = scal[L::MISC * kChunk];
            uint32_t hi[2][4], lo[2][4];
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) {
                split_half(r[2 * ks][0] * fu0, r[2 * ks][1] * fu0, hi[ks][0], lo[ks][0]);
                split_half(r[2 * ks][2] * fu1, r[2 * ks][3] * fu1, hi[ks][1], lo[ks][1]);
                split_half(r[2 * ks + 1][0] * fu0, r[2 * ks + 1][1] * fu0, hi[ks][2], lo[ks][2]);
                split_half(r[2 * ks + 1][2] * fu1, r[2 * ks + 1][3] * fu1, hi[ks][3], lo[ks][3]);
            }
            sm0 = sm1 = 0.f;
#pragma unroll
            for (int i = 0; i < NC; i += 4) {
                float acc[4][4];
#pragma unroll
                for (int t = 0; t < 4; ++t)
#pragma unroll
                    for (int x = 0; x < 4; ++x) acc[t][x] = 0.f;
#pragma unroll
                for (int ks = 0; ks < 2; ++ks) {
                    uint32_t b0[4], b1[4];
                    ldsm4_t(b0, sb + L::K + (16 * ks + trow) * L::KP + tcol + c0 * 2 + i * 16);
                    ldsm4_t(b1, sb + L::K + (16 * ks + trow) * L::KP + tcol + c0 * 2 + i * 16 + 32);
                    mma16816(acc[0], hi[ks], b0[0], b0[1]);
                    mma16816(acc[1], hi[ks], b0[2], b0[3]);
                    mma16816(acc[2], hi[ks], b1[0], b1[1]);
                    mma16816(acc[3], hi[ks], b1[2], b1[3]);
                    mma16816(acc[0], lo[ks], b0[0], b0[1]);
                    mma16816(acc[1], lo[ks], b0[2], b0[3]);
                    mma16816(acc[2], lo[ks], b1[0], b1[1]);
                    mma16816(acc[3], lo[ks], b1[2], b1[3]);
                }
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    s[i + t][0] = fmaf(gend, s[i + t][0], iu0 * acc[t][0]);
                    s[i + t][1] = fmaf(gend, s[i + t][1], iu0 * acc[t][1]);
                    s[i + t][2] = fmaf(gend, s[i + t][2], iu1 * acc[t][2]);
                    s[i + t][3] = fmaf(gend, s[i + t][3], iu1 * acc[t][3]);
                    sm0 = fmaxf(sm0, fmaxf(fabsf(s[i + t][0]), fabsf(s[i + t][1])));
                    sm1 = fmaxf(sm1, fmaxf(fabsf(s[i + t][2]), fabsf(s[i + t][3])));
                }
            }
        }
        if (!REC) {
            const float fu0 = row_scale(quad_max(m2), out.i0), fu1 = row_scale(quad_max(m3), out.i1);
            const int t0 = KS == 2 ? part * 16 : 0;
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) {
                out.u[ks][0] = pack_half(nn[2 * ks][0] * fu0, nn[2 * ks][1] * fu0);
                out.u[ks][1] = pack_half(nn[2 * ks][2] * fu1, nn[2 * ks][3] * fu1);
                out.u[ks][2] = pack_half(nn[2 * ks + 1][0] * fu0, nn[2 * ks + 1][1] * fu0);
                out.u[ks][3] = pack_half(nn[2 * ks + 1][2] * fu1, nn[2 * ks + 1][3] * fu1);
            }
            const uint32_t pb = sb + L::P + nrow * L::XP + ncol;
            if constexpr (KS == 2) {
                ldsm4(out.p[0], pb + t0 * L::XP);
                if (part) {
                    ldsm4(out.p[1], pb + t0 * L::XP + 32);
                } else {
#pragma unroll
                    for (int x = 0; x < 4; ++x) out.p[1][x] = 0u;
                }
            } else {
                ldsm4(out.p[0], pb);
                ldsm4(out.p[1], pb + 16 * L::XP);
                ldsm4(out.p[2], pb + 16 * L::XP + 32);
            }
#pragma unroll
            for (int t = 0; t < 4 / KS; ++t) {
                out.cq[t] = *reinterpret_cast<const float2 *>(scal + L::CQ * kChunk + t0 + 8 * t + tc);
                out.iq[t] = *reinterpret_cast<const float2 *>(scal + L::IQ * kChunk + t0 + 8 * t + tc);
#pragma unroll
                for (int x = 0; x < 4; ++x) out.oq[t][x] = oq[t][x];
            }
            if (KS == 1 || ci + 1 == chunks)
                out.write(out_tile, M::OP, a.o + (row * a.H + h) * a.dv + j0, vstride, part, valid);
        }
        pipe.release(st);
    }
    if (ok && a.state_out) {
        float *dst = a.state_out + state_off;
#pragma unroll
        for (int i = 0; i < NC; ++i)
#pragma unroll
            for (int x = 0; x < 4; ++x)
                dst[(int64_t)(8 * i + (x & 1)) * a.dv + (x >> 1) * 8] = s[i][x];
    }
    pipe.finish();
}

template <int DK, int NCW, int KS, int CL, bool REC>
static cudaError_t launch_chain_t(const ChainArgs &a, int64_t units, cudaStream_t st) {
    using M = Pipe<DK, NCW, KS, CL, false, !REC, 24>;
    return launch_pipe(gdr_chain_kernel<DK, NCW, KS, CL, REC>, a, a.k, a.q, a.v, a.rows, DK, M::W,
                       units * CL, M::WARPS * 32, M::BYTES, CL, st);
}

// Columns per CTA and warps per column group.  The chain's rate is set by its warps'
// matrix instructions (8 cycles each per SM quarter), so with few (sequence, head) units
// the work is spread over as many SMs and warps as there are; with many, one CTA takes all
// columns, so that the producers' work is done once per chunk without a cluster.
template <int DK, bool REC>
static cudaError_t launch_chain_d(const ChainArgs &a, int64_t units, cudaStream_t st) {
    if (a.dv == 128) {
        if (units * 4 <= 128) return launch_chain_t<DK, 2, 2, 4, REC>(a, units, st);
        if (units * 2 <= 148) return launch_chain_t<DK, 4, 1, 2, REC>(a, units, st);
        return launch_chain_t<DK, 8, 1, 1, REC>(a, units, st);
    }
    if (units * 2 <= 148) return launch_chain_t<DK, 2, 2, 2, REC>(a, units, st);
    return launch_chain_t<DK, 4, 1, 1, REC>(a, units, st);
}

}  // namespace gdr

cudaError_t launch_gdr_prefill(const GdrArgs &p, cudaStream_t st) {
    using bf = __nv_bfloat16;
    gdr::ChainArgs a{(const bf *)p.q, (const bf *)p.k, (const bf *)p.v, (const bf *)p.g,
                     (const bf *)p.beta, p.state_in, p.cu_seqlens, p.T, p.rows, p.Hk, p.H, p.dv,
                     (bf *)p.o, p.state_out, nullptr, nullptr, nullptr, nullptr, p.err, p.epoch};
    const int64_t units = (int64_t)p.N * p.H;
    return p.dk == 64 ? gdr::launch_chain_d<64, false>(a, units, st)
                      : gdr::launch_chain_d<128, false>(a, units, st);
}

cudaError_t launch_gdr_recompute(const GdrArgs &p, const GdrBackwardSpace &w, cudaStream_t st) {
    using bf = __nv_bfloat16;
    gdr::ChainArgs a{(const bf *)p.q, (const bf *)p.k, (const bf *)p.v, (const bf *)p.g,
                     (const bf *)p.beta, p.state_in, p.cu_seqlens, p.T, p.rows, p.Hk, p.H, p.dv,
                     nullptr, nullptr, w.n, w.s_blocks, w.s_tops, w.owners, p.err, p.epoch};
    const int64_t units = (int64_t)p.N * p.H;
    return p.dk == 64 ? gdr::launch_chain_d<64, true>(a, units, st)
                      : gdr::launch_chain_d<128, true>(a, units, st);
}

}  // namespace kda
