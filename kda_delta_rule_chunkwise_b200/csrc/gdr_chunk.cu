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
// (K, Q, X, P) are the same for all columns; gdr_prep_kernel makes them, all chunks at once.
//
// Precision: S, V - Gamma K S and beta N enter the products as fp16 hi + lo of the row
// scaled by a power of two (22 bits), K and Q are exact in fp16 after a power-of-two scale
// per row, so the state keeps fp32 accuracy (the final state is an fp32 output).  What
// only o depends on (S and beta N in its two products, P) is rounded once to fp16, 2^-12,
// below o's own rounding to bf16.
//
// What bounds it: with few heads the latency of a chunk's dependent steps, 2500 cycles of which the
// matrix instructions are 800 (354 us for 8192 tokens of 32 heads, dk = dv = 128, beside 55 us for
// the chunks; the operator's bytes would take 32 us); with many the matrix pipe and the shared memory
// that feeds it, each half busy with the two warps per SM quarter that the registers allow (641 us
// for 16 packed prompts of 30011 tokens together; the operator's bytes would take 106 us).
#include "gdr_common.cuh"
#include "gdr_launch.h"

namespace kda {
namespace gdr {

struct ChainArgs {
    ChainInput in;
    const float *state_in;
    __nv_bfloat16 *o;       // prefill
    float *state_out;       // prefill
    float *n_out;           // recomputation: N [rows, H, dv]
    unsigned char *blocks;  // recomputation: state before each 64-token block [.., H] (store_block)
    float *scales;          // recomputation: their inverse scales [.., H, dv/16, 2]
    int32_t *owners;        // recomputation: the sequence of each block
};

// What finishes a chunk's outputs of a column group: O = Gamma Q S + P U, both in the scaled units
// of Q', rounded and written through `tile`.
struct ChunkOut {
    uint32_t u[2][4], p[3][4];   // U^T (16 columns x 32 tokens); P's blocks (0,0) (1,0) (1,1)
    float oq[4][4], i0, i1;
    float2 cq[4], iq[4];

    // U^T times ik, fp16 after a power-of-two scale per column
    __device__ __forceinline__ void pack_u(const float (&x)[4][4]) {
        float m0 = 0.f, m1 = 0.f;
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            m0 = fmaxf(m0, fmaxf(fabsf(x[t][0]), fabsf(x[t][1])));
            m1 = fmaxf(m1, fmaxf(fabsf(x[t][2]), fabsf(x[t][3])));
        }
        const float f0 = row_scale(quad_max(m0), i0), f1 = row_scale(quad_max(m1), i1);
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
            u[ks][0] = pack_half(x[2 * ks][0] * f0, x[2 * ks][1] * f0);
            u[ks][1] = pack_half(x[2 * ks][2] * f1, x[2 * ks][3] * f1);
            u[ks][2] = pack_half(x[2 * ks + 1][0] * f0, x[2 * ks + 1][1] * f0);
            u[ks][3] = pack_half(x[2 * ks + 1][2] * f1, x[2 * ks + 1][3] * f1);
        }
    }
    // P and the row scalars of the chunk in a stage
    template <typename L>
    __device__ __forceinline__ void read_stage(uint32_t sb, const float *scal) {
        const int lane = threadIdx.x & 31, tc = 2 * (lane & 3);
        const uint32_t pb = sb + L::P + ((lane & 7) + (lane >> 4) * 8) * L::XP + ((lane >> 3) & 1) * 16;
        ldsm4(p[0], pb);
        ldsm4(p[1], pb + 16 * L::XP);
        ldsm4(p[2], pb + 16 * L::XP + 32);
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            cq[t] = *reinterpret_cast<const float2 *>(scal + L::CQ * kChunk + 8 * t + tc);
            iq[t] = *reinterpret_cast<const float2 *>(scal + L::IQ * kChunk + 8 * t + tc);
        }
    }
    __device__ __forceinline__ void write(unsigned char *tile, int pitch, __nv_bfloat16 *dst,
                                          int64_t stride, int valid) const {
        const int lane = threadIdx.x & 31;
        const int nrow = (lane & 7) + (lane >> 4) * 8, ncol = ((lane >> 3) & 1) * 16;
        float ou[4][4];
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int x = 0; x < 4; ++x) ou[t][x] = 0.f;
        mma16816(ou[0], u[0], p[0][0], p[0][1]);
        mma16816(ou[1], u[0], p[0][2], p[0][3]);
        mma16816(ou[2], u[0], p[1][0], p[1][1]);
        mma16816(ou[3], u[0], p[1][2], p[1][3]);
        mma16816(ou[2], u[1], p[2][0], p[2][1]);
        mma16816(ou[3], u[1], p[2][2], p[2][3]);
        __syncwarp();   // the rows written before have been read out of the tile
#pragma unroll
        for (int t = 0; t < 4; t += 2) {
            uint32_t pk[2][2];
#pragma unroll
            for (int v = 0; v < 2; ++v) {
                const int i = t + v;
                const __nv_bfloat162 w0 = __floats2bfloat162_rn(cq[i].x * oq[i][0] + iq[i].x * (i0 * ou[i][0]),
                                                                cq[i].y * oq[i][1] + iq[i].y * (i0 * ou[i][1]));
                const __nv_bfloat162 w1 = __floats2bfloat162_rn(cq[i].x * oq[i][2] + iq[i].x * (i1 * ou[i][2]),
                                                                cq[i].y * oq[i][3] + iq[i].y * (i1 * ou[i][3]));
                pk[v][0] = reinterpret_cast<const uint32_t &>(w0);
                pk[v][1] = reinterpret_cast<const uint32_t &>(w1);
            }
            stsm4_t(smem_u32(tile) + (8 * t + nrow) * pitch + ncol, pk[0][0], pk[0][1], pk[1][0], pk[1][1]);
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int tok = i * 16 + (lane >> 1);
            const uint4 w = *reinterpret_cast<const uint4 *>(tile + tok * pitch + (lane & 1) * 16);
            if (tok < valid) *reinterpret_cast<uint4 *>(dst + tok * stride + (lane & 1) * 8) = w;
        }
    }
};
// The hand-over of a chunk from a group's two chain warps to its output warp (KS = 2): per lane the
// two partial Q S (4 float4 each) and U^T (4 float4, each warp writes its half of the tokens).
constexpr int kHandU = 2 * 4 * 512, kHandBytes = kHandU + 4 * 512;
template <int KS, bool REC>
constexpr int hand_bytes() { return KS == 2 && !REC ? kHandBytes : 0; }

// With KS = 2 the two warps of a column group add their partial K S through shared memory, compute
// N twice, and update their own halves of S: half the products per warp on the chain, for one
// exchange; and the outputs are left to an output warp per group.
template <int DK, int NCW, int KS, bool REC>
__global__ void __launch_bounds__((Pipe<DK, NCW, KS, false, !REC, hand_bytes<KS, REC>()>::WARPS * 32), 1)
    gdr_chain_kernel(const __grid_constant__ CUtensorMap vmap, const __grid_constant__ ChainArgs args) {
    using M = Pipe<DK, NCW, KS, false, !REC, hand_bytes<KS, REC>()>;
    using L = typename M::L;
    constexpr int W = M::W, NC = DK / 8 / KS, NK = DK / 16 / KS;
    extern __shared__ __align__(1024) unsigned char smem[];
    const ChainInput &a = args.in;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int slices = a.dv / W;
    const int slice = blockIdx.x % slices, unit = blockIdx.x / slices;
    const int h = unit % a.H, n = a.order ? a.order[unit / a.H] : unit / a.H, hk = h / (a.H / a.Hk);
    const Span span = sequence_span(a.cu, n, a.T);
    const int chunks = (span.len + kChunk - 1) / kChunk;
    if (REC && h == 0 && slice == 0)
        for (int i = threadIdx.x; 2 * i < chunks; i += blockDim.x)
            args.owners[first_block(span, n) + i] = n;
    const M pipe(smem, a.err, a.epoch);

    if (M::OW > 0 && warp > M::CHAIN) {
        // ---- output warp of a column group
        const int group = warp - M::CHAIN - 1;
        unsigned char *tile = smem + M::OUT + group * kChunk * M::OP;
        ChunkOut out;
        for (int ci = 0; ci < chunks; ++ci) {
            const int st = ci % M::ST;
            const uint32_t turn = (ci / M::ST) & 1;
            if (!pipe.wait(pipe.full + st, turn)) break;
            out.template read_stage<L>(smem_u32(pipe.stage(st)),
                                       reinterpret_cast<const float *>(pipe.stage(st) + L::S));
            if (!pipe.wait(pipe.handed + group * M::ST + st, turn)) break;
            const float4 *hand = reinterpret_cast<const float4 *>(pipe.hand(group, st)) + lane;
            float u[4][4];
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const float4 x = hand[t * 32], y = hand[(4 + t) * 32], w = hand[(8 + t) * 32];
                out.oq[t][0] = x.x + y.x; out.oq[t][1] = x.y + y.y;
                out.oq[t][2] = x.z + y.z; out.oq[t][3] = x.w + y.w;
                u[t][0] = w.x; u[t][1] = w.y; u[t][2] = w.z; u[t][3] = w.w;
            }
            out.pack_u(u);
            const int64_t row = span.row + (int64_t)ci * kChunk;
            out.write(tile, M::OP, args.o + (row * a.H + h) * a.dv + slice * W + group * 16,
                      (int64_t)a.H * a.dv, span.len - ci * kChunk);
            pipe.release(st);   // P has been used
        }
        return;
    }
    if (warp >= M::CHAIN) {
        pipe.template load<false>(a, &vmap, span, n, h, hk, slice * W, chunks);
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
        const float *in = args.state_in ? args.state_in + state_off : nullptr;
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
    unsigned char *out_tile = smem + M::OUT + warp * kChunk * M::OP;
    const int64_t vstride = (int64_t)a.H * a.dv;
    ChunkOut out;   // KS = 1: this warp writes the outputs itself
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
            store_block<NC>(args.blocks + blk * DK * block_row(a.dv), args.scales + (blk * (a.dv / 16) + j0 / 16) * 2,
                            s, fmaxf(sm0, sm1), KS, part, c0, j0, a.dv, out_tile);
        }
        ok = pipe.wait(pipe.full + st, (ci / M::ST) & 1);
        if (!ok) break;

        // Y^T = S^T K'^T (two terms of S) and S^T Q'^T (the high term)
        float y[4][4], oq[4][4];
        uint32_t high[NK][4];   // S's high terms, for Q S
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int x = 0; x < 4; ++x) y[t][x] = oq[t][x] = 0.f;
        auto add_qs = [&](int kk) {
            uint32_t b0[4], b1[4];
            ldsm4(b0, sb + L::Q + nrow * L::KP + ncol + c0 * 2 + kk * 32);
            ldsm4(b1, sb + L::Q + (nrow + 16) * L::KP + ncol + c0 * 2 + kk * 32);
            mma16816(oq[0], high[kk], b0[0], b0[1]);
            mma16816(oq[1], high[kk], b0[2], b0[3]);
            mma16816(oq[2], high[kk], b1[0], b1[1]);
            mma16816(oq[3], high[kk], b1[2], b1[3]);
        };
#pragma unroll
        for (int kk = 0; kk < NK; ++kk) {
            uint32_t(&hi)[4] = high[kk], lo[4], b0[4], b1[4];
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
            if (!REC && KS == 1) add_qs(kk);
        }
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            y[t][0] *= is0; y[t][1] *= is0; y[t][2] *= is1; y[t][3] *= is1;
        }
        float4 *hand = KS == 2 && !REC ? reinterpret_cast<float4 *>(pipe.hand(group, st)) + lane : nullptr;
        if (KS == 2) {
            // add the other half's sums.  Buffers alternate: the other warp has read the ones of
            // two chunks before by now.
            float4 *mine = reinterpret_cast<float4 *>(smem + M::SWAP) +
                           (((group * 2 + (ci & 1)) * 2 + part) * 4) * 32 + lane;
#pragma unroll
            for (int t = 0; t < 4; ++t) mine[t * 32] = make_float4(y[t][0], y[t][1], y[t][2], y[t][3]);
            __syncwarp();
            if (lane == 0) mbar_arrive(pipe.swapped + group);
        }
        // what does not depend on the other half, while it is on its way: this half's Q S, for the output
        // warp, and the operands of what follows
        if (!REC && KS == 2)
#pragma unroll
            for (int kk = 0; kk < NK; ++kk) add_qs(kk);
        if (!REC)
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                oq[t][0] *= is0; oq[t][1] *= is0; oq[t][2] *= is1; oq[t][3] *= is1;
                if (KS == 2) hand[(part * 4 + t) * 32] = make_float4(oq[t][0], oq[t][1], oq[t][2], oq[t][3]);
            }
        uint32_t v[2][4], xh[3][4], xl[3][4];   // values; blocks (0,0) (1,0) (1,1) of X
        float2 ck[4];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            ldsm4_t(v[t], sb + L::v_at(16 * t + nrow, group * 2 + ((lane >> 3) & 1)));
            if (valid < kChunk) clear_rows(v[t], 16 * t + tc, valid);   // rows behind the sequence's end
        }
#pragma unroll
        for (int t = 0; t < 4; ++t) ck[t] = *reinterpret_cast<const float2 *>(scal + L::CK * kChunk + 8 * t + tc);
        {
            const uint32_t at = sb + nrow * L::XP + ncol;
            ldsm4(xh[0], at + L::XH);
            ldsm4(xl[0], at + L::XL);
            ldsm4(xh[1], at + L::XH + 16 * L::XP);
            ldsm4(xl[1], at + L::XL + 16 * L::XP);
            ldsm4(xh[2], at + L::XH + 16 * L::XP + 32);
            ldsm4(xl[2], at + L::XL + 16 * L::XP + 32);
        }
        if (KS == 2) {
            ok = pipe.wait(pipe.swapped + group, ci & 1);
            if (!ok) break;
            const float4 *other = reinterpret_cast<const float4 *>(smem + M::SWAP) +
                                  (((group * 2 + (ci & 1)) * 2 + (part ^ 1)) * 4) * 32 + lane;
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const float4 o = other[t * 32];
                y[t][0] += o.x; y[t][1] += o.y; y[t][2] += o.z; y[t][3] += o.w;
            }
        }
        // R = V - Gamma K S, this lane's tokens 8t + tc + {0, 1}
        float r[4][4], m0 = 0.f, m1 = 0.f;
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const uint32_t v0 = v[t >> 1][2 * (t & 1)], v1 = v[t >> 1][2 * (t & 1) + 1];
            r[t][0] = __uint_as_float(v0 << 16) - ck[t].x * y[t][0];
            r[t][1] = __uint_as_float(v0 & 0xffff0000u) - ck[t].y * y[t][1];
            r[t][2] = __uint_as_float(v1 << 16) - ck[t].x * y[t][2];
            r[t][3] = __uint_as_float(v1 & 0xffff0000u) - ck[t].y * y[t][3];
            m0 = fmaxf(m0, fmaxf(fabsf(r[t][0]), fabsf(r[t][1])));
            m1 = fmaxf(m1, fmaxf(fabsf(r[t][2]), fabsf(r[t][3])));
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
                    const uint32_t(&h4)[4] = xh[half + ks], (&l4)[4] = xl[half + ks];
                    mma16816(nn[2 * half], hi, h4[0], h4[1]);
                    mma16816(nn[2 * half + 1], hi, h4[2], h4[3]);
                    mma16816(nl[2 * half], lo, h4[0], h4[1]);
                    mma16816(nl[2 * half + 1], lo, h4[2], h4[3]);
                    mma16816(nl[2 * half], hi, l4[0], l4[1]);
                    mma16816(nl[2 * half + 1], hi, l4[2], l4[3]);
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
            float *dst = args.n_out + (row * a.H + h) * a.dv + j0 + jr;
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const int tok = 8 * t + tc + (x & 1);
                    if (tok < valid && (KS == 1 || t / 2 == part)) dst[tok * vstride + (x >> 1) * 8] = nn[t][x];
                }
        }
        // U = beta N in the scaled units of K', and with the decay to the chunk's end
        m0 = m1 = 0.f;
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const float2 e = *reinterpret_cast<const float2 *>(scal + L::OK * kChunk + 8 * t + tc);
#pragma unroll
            for (int x = 0; x < 4; ++x) r[t][x] = nn[t][x] * ((x & 1) ? e.y : e.x);
            m0 = fmaxf(m0, fmaxf(fabsf(r[t][0]), fabsf(r[t][1])));
            m1 = fmaxf(m1, fmaxf(fabsf(r[t][2]), fabsf(r[t][3])));
        }
        if (!REC)
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const float2 k = *reinterpret_cast<const float2 *>(scal + L::BK * kChunk + 8 * t + tc);
#pragma unroll
                for (int x = 0; x < 4; ++x) nn[t][x] *= (x & 1) ? k.y : k.x;
                if (KS == 2 && t / 2 == part)
                    hand[(8 + t) * 32] = make_float4(nn[t][0], nn[t][1], nn[t][2], nn[t][3]);
            }
        if (KS == 2 && !REC) {   // the output warp may go on
            __syncwarp();
            if (lane == 0) mbar_arrive(pipe.handed + group * M::ST + st);
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
        if (!REC && KS == 1) {
            out.pack_u(nn);
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int x = 0; x < 4; ++x) out.oq[t][x] = oq[t][x];
            out.template read_stage<L>(sb, scal);
            out.write(out_tile, M::OP, args.o + (row * a.H + h) * a.dv + j0, vstride, valid);
        }
        pipe.release(st);
    }
    if (ok && args.state_out) {
        float *dst = args.state_out + state_off;
#pragma unroll
        for (int i = 0; i < NC; ++i)
#pragma unroll
            for (int x = 0; x < 4; ++x)
                dst[(int64_t)(8 * i + (x & 1)) * a.dv + (x >> 1) * 8] = s[i][x];
    }
}

template <int DK, int NCW, int KS, bool REC>
static cudaError_t launch_chain_t(const ChainArgs &a, const void *v, int64_t rows, int64_t units, cudaStream_t st) {
    using M = Pipe<DK, NCW, KS, false, !REC, hand_bytes<KS, REC>()>;
    return launch_chain_kernel(gdr_chain_kernel<DK, NCW, KS, REC>, a, v, rows, M::W, units, M::WARPS * 32, M::BYTES,
                               st);
}

template <int DK, bool REC>
static cudaError_t launch_chain_d(const ChainArgs &a, const void *v, int64_t rows, int64_t units, cudaStream_t st) {
    switch (chain_variant(units, a.in.dv, a.in.cu != nullptr)) {
        case 22: return launch_chain_t<DK, 2, 2, REC>(a, v, rows, units, st);
        case 41: return launch_chain_t<DK, 4, 1, REC>(a, v, rows, units, st);
        default: return launch_chain_t<DK, 8, 1, REC>(a, v, rows, units, st);
    }
}

}  // namespace gdr

cudaError_t launch_gdr_prefill(const GdrArgs &p, void *workspace, cudaStream_t st) {
    const GdrImages m = gdr_images(workspace, p, false);
    const cudaError_t e = launch_gdr_prep(p, m, st);
    if (e != cudaSuccess) return e;
    gdr::ChainArgs a{{m.keys, m.forward, p.cu_seqlens, m.order, p.T, p.Hk, p.H, p.dv, p.err, p.epoch},
                     p.state_in, (__nv_bfloat16 *)p.o, p.state_out};
    const int64_t units = (int64_t)p.N * p.H;
    return p.dk == 64 ? gdr::launch_chain_d<64, false>(a, p.v, p.rows, units, st)
                      : gdr::launch_chain_d<128, false>(a, p.v, p.rows, units, st);
}

cudaError_t launch_gdr_recompute(const GdrArgs &p, const GdrImages &m, const GdrBackwardSpace &w, cudaStream_t st) {
    gdr::ChainArgs a{{m.keys, m.forward, p.cu_seqlens, m.order, p.T, p.Hk, p.H, p.dv, p.err, p.epoch},
                     p.state_in, nullptr, nullptr, w.n, w.s_blocks, w.s_scales, w.owners};
    const int64_t units = (int64_t)p.N * p.H;
    return p.dk == 64 ? gdr::launch_chain_d<64, true>(a, p.v, p.rows, units, st)
                      : gdr::launch_chain_d<128, true>(a, p.v, p.rows, units, st);
}

}  // namespace kda
