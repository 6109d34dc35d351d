// Gated delta rule, backward, bf16 (notation of gdr_chunk.cu).
//
// With Z = dL/dS behind a chunk, E = X^T dU for X = (I + A)^-1, A[r][s] = beta_r D[r][s] (k_r . k_s):
//
//     dU = P^T dO + exp(G_C - G) K Z
//     E  = X^T dU,   dV = dR = beta E
//     Z' = Gamma_C Z + (Gamma Q)^T dO - (Gamma K)^T dR                      (before the chunk)
//
// which has the shape of the forward chain and runs like it: one warp keeps 16 value columns of Z
// in registers and walks the chunks backward (gdr_adjoint_kernel).  N = U / beta and E are formed
// without a division (each by an inverse with beta on its own side), so beta = 0 needs no case.
//
// What is left is local to a block of 64 tokens, given the state S before it and Z behind it
// (gdr_grads_kernel), with M1 = dO N^T, M2 = E N^T, dP = D beta_s M1, dA = -beta_r beta_s D M2:
//
//     dQ = Gamma dO S^T + dP K
//     dK = -Gamma beta E S^T + dA K  +  exp(G_C - G) beta N Z^T + dP^T Q + dA^T K
//     dbeta_r = E_r . N_r
//     dg_t = sum_{r >= t} (row - column sums of W) + sum_{r >= t} Gamma_r (q_r . (dO S^T)_r - beta_r k_r . (E S^T)_r)
//          + sum_{s < t} exp(G_C - G_s) beta_s k_s . (N Z^T)_s + Gamma_C <S, Z>,
//            W = dP o (Q K^T) + dA o (K K^T), strictly lower
//
// The last line holds no difference of large sums: the parts of k . dk that a plain reverse sum
// would first add and then take away again are left out of it.
//
// The adjoint chain keeps fp32 accuracy like the forward one (dstate_in is fp32).  The block
// kernel's products take fp16 operands scaled by a power of two per tile (2^-11 each, 29 binary
// orders below the tile's largest value), below the rounding of its bf16 outputs.
//
// At 8192 tokens of 32 heads (dk = dv = 128): chunks 70 us, the forward's chain 360, the adjoint's
// 479 (latency of a chunk's steps, like the forward's), the blocks' gradients 401 (shared-memory reads
// of the operands and the loads between barriers); the operator's bytes would take 53 us.
#include "gdr_common.cuh"
#include "gdr_launch.h"
#include "gdr_token_backward.h"

#include <type_traits>

namespace kda {
namespace gdr {

struct AdjointArgs {
    ChainInput in;
    const float *dstate_out;
    __nv_bfloat16 *dv_out;
    float *dstate_in;
    float *e_out;
    unsigned char *blocks;
    float *scales;
};

// Warps, stages and the two halves of KS = 2 as in gdr_chain_kernel; chunks from last to first.
template <int DK, int NCW, int KS>
__global__ void __launch_bounds__((Pipe<DK, NCW, KS, true, true, 0>::WARPS * 32), 1)
    gdr_adjoint_kernel(const __grid_constant__ CUtensorMap vmap, const __grid_constant__ AdjointArgs args) {
    using M = Pipe<DK, NCW, KS, true, true, 0>;
    using L = typename M::L;
    constexpr int W = M::W, NC = DK / 8 / KS, NK = DK / 16 / KS, XF = 16;
    extern __shared__ __align__(1024) unsigned char smem[];
    const ChainInput &a = args.in;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int slices = a.dv / W;
    const int slice = blockIdx.x % slices, unit = blockIdx.x / slices;
    const int h = unit % a.H, n = a.order ? a.order[unit / a.H] : unit / a.H, hk = h / (a.H / a.Hk);
    const Span span = sequence_span(a.cu, n, a.T);
    const int chunks = (span.len + kChunk - 1) / kChunk;
    const M pipe(smem, a.err, a.epoch);

    if (warp >= M::CHAIN) {
        pipe.template load<true>(a, &vmap, span, n, h, hk, slice * W, chunks);
        return;
    }

    const int group = warp / KS, part = warp % KS;
    const int j0 = slice * W + group * 16, jr = lane >> 2, tc = 2 * (lane & 3);
    const int c0 = part * (DK / KS);
    float z[NC][4];   // Z^T, laid out like the forward's S^T
    float zm0 = 0.f, zm1 = 0.f;   // this lane's largest |Z| of its two columns
    const int64_t state_off = ((int64_t)n * a.H + h) * DK * a.dv + (int64_t)(c0 + tc) * a.dv + j0 + jr;
    {
        const float *in = args.dstate_out ? args.dstate_out + state_off : nullptr;
#pragma unroll
        for (int i = 0; i < NC; ++i) {
#pragma unroll
            for (int x = 0; x < 4; ++x)
                z[i][x] = in ? in[(int64_t)(8 * i + (x & 1)) * a.dv + (x >> 1) * 8] : 0.f;
            zm0 = fmaxf(zm0, fmaxf(fabsf(z[i][0]), fabsf(z[i][1])));
            zm1 = fmaxf(zm1, fmaxf(fabsf(z[i][2]), fabsf(z[i][3])));
        }
    }
    const int nrow = (lane & 7) + (lane >> 4) * 8, ncol = ((lane >> 3) & 1) * 16;
    const int trow = lane & 15, tcol = (lane >> 4) * 16;
    unsigned char *out_tile = smem + M::OUT + warp * kChunk * M::OP;
    const int64_t vstride = (int64_t)a.H * a.dv;
    bool ok = true;
    uint32_t pk[4][2];   // a chunk's dV in bf16; with KS = 2 written inside the next chunk
    auto write_dv = [&](int64_t row, int valid) {   // this warp's 16 tokens with KS = 2, else all 32
        const int t0 = KS == 2 ? part * 16 : 0;
        __syncwarp();
#pragma unroll
        for (int t = 0; t < 4; t += 2)
            if (KS == 1 || t / 2 == part)
                stsm4_t(smem_u32(out_tile) + (8 * t + nrow) * M::OP + ncol, pk[t][0], pk[t][1],
                        pk[t + 1][0], pk[t + 1][1]);
        __syncwarp();
        __nv_bfloat16 *dst = args.dv_out + (row * a.H + h) * a.dv + j0;
#pragma unroll
        for (int i = 0; i < 2 / KS; ++i) {
            const int tok = t0 + i * 16 + (lane >> 1);
            const uint4 w = *reinterpret_cast<const uint4 *>(out_tile + tok * M::OP + (lane & 1) * 16);
            if (tok < valid) *reinterpret_cast<uint4 *>(dst + tok * vstride + (lane & 1) * 8) = w;
        }
    };

    for (int it = 0; it < chunks; ++it) {
        const int ci = chunks - 1 - it, st = it % M::ST;
        unsigned char *stage = pipe.stage(st);
        const uint32_t sb = smem_u32(stage);
        const float *scal = reinterpret_cast<const float *>(stage + L::S);
        const int64_t row = span.row + (int64_t)ci * kChunk;
        const int valid = span.len - ci * kChunk;
        const bool block_end = (ci & 1) == 1 || it == 0;
        const int64_t blk = (first_block(span, n) + ci / 2) * a.H + h;

        float m0, m1, iz0, iz1;
        const float fz0 = row_scale(quad_max(zm0), iz0), fz1 = row_scale(quad_max(zm1), iz1);
        if (block_end)
            store_block<NC>(args.blocks + blk * DK * block_row(a.dv), args.scales + (blk * (a.dv / 16) + j0 / 16) * 2,
                            z, fmaxf(zm0, zm1), KS, part, c0, j0, a.dv, smem + M::OUT + warp * kChunk * M::OP);

        ok = pipe.wait(pipe.full + st, (it / M::ST) & 1);
        if (!ok) break;

        // Z^T K'^T, two terms of Z
        float y[4][4];
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int x = 0; x < 4; ++x) y[t][x] = 0.f;
#pragma unroll
        for (int kk = 0; kk < NK; ++kk) {
            uint32_t hi[4], lo[4], b0[4], b1[4];
            split_half(z[2 * kk][0] * fz0, z[2 * kk][1] * fz0, hi[0], lo[0]);
            split_half(z[2 * kk][2] * fz1, z[2 * kk][3] * fz1, hi[1], lo[1]);
            split_half(z[2 * kk + 1][0] * fz0, z[2 * kk + 1][1] * fz0, hi[2], lo[2]);
            split_half(z[2 * kk + 1][2] * fz1, z[2 * kk + 1][3] * fz1, hi[3], lo[3]);
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
        }
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            y[t][0] *= iz0; y[t][1] *= iz0; y[t][2] *= iz1; y[t][3] *= iz1;
        }
        if (KS == 2) {
            float4 *mine = reinterpret_cast<float4 *>(smem + M::SWAP) +
                           (((group * 2 + (it & 1)) * 2 + part) * XF / 4) * 32 + lane;
#pragma unroll
            for (int t = 0; t < 4; ++t) mine[t * 32] = make_float4(y[t][0], y[t][1], y[t][2], y[t][3]);
            __syncwarp();
            if (lane == 0) mbar_arrive(pipe.swapped + group);
            if (it > 0) write_dv(row + kChunk, valid - kChunk);   // the chunk after this one
        }
        // What does not depend on the other half, while its sums are on their way: dO^T in the scaled
        // units of Q' (exact: powers of two), P'^T dO, and Z <- Gamma_C Z + (Gamma dO)^T Q'.
        float pu[4][4];
        {
            float o[4][4];
            m0 = m1 = 0.f;
#pragma unroll
            for (int t = 0; t < 4; t += 2) {
                uint32_t v[4];
                ldsm4_t(v, sb + L::v_at(8 * t + nrow, group * 2 + ((lane >> 3) & 1)));
                if (valid < kChunk) clear_rows(v, 8 * t + tc, valid);   // the rows behind the sequence's end
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const float2 iq = *reinterpret_cast<const float2 *>(scal + L::IQ * kChunk + 8 * (t + u) + tc);
                    o[t + u][0] = __uint_as_float(v[2 * u] << 16) * iq.x;
                    o[t + u][1] = __uint_as_float(v[2 * u] & 0xffff0000u) * iq.y;
                    o[t + u][2] = __uint_as_float(v[2 * u + 1] << 16) * iq.x;
                    o[t + u][3] = __uint_as_float(v[2 * u + 1] & 0xffff0000u) * iq.y;
                    m0 = fmaxf(m0, fmaxf(fabsf(o[t + u][0]), fabsf(o[t + u][1])));
                    m1 = fmaxf(m1, fmaxf(fabsf(o[t + u][2]), fabsf(o[t + u][3])));
                }
            }
            float io0, io1;
            const float fo0 = row_scale(quad_max(m0), io0), fo1 = row_scale(quad_max(m1), io1);
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int x = 0; x < 4; ++x) pu[t][x] = 0.f;
            m0 = m1 = 0.f;
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) {
                const uint32_t u[4] = {
                    pack_half(o[2 * ks][0] * fo0, o[2 * ks][1] * fo0),
                    pack_half(o[2 * ks][2] * fo1, o[2 * ks][3] * fo1),
                    pack_half(o[2 * ks + 1][0] * fo0, o[2 * ks + 1][1] * fo0),
                    pack_half(o[2 * ks + 1][2] * fo1, o[2 * ks + 1][3] * fo1)};
#pragma unroll
                for (int half = 0; half <= ks; ++half) {   // P is zero above the diagonal
                    uint32_t bh[4], bl[4];
                    ldsm4_t(bh, sb + L::P + (16 * ks + trow) * L::XP + tcol + half * 32);
                    ldsm4_t(bl, sb + L::PL + (16 * ks + trow) * L::XP + tcol + half * 32);
                    mma16816(pu[2 * half], u, bh[0], bh[1]);
                    mma16816(pu[2 * half + 1], u, bh[2], bh[3]);
                    mma16816(pu[2 * half], u, bl[0], bl[1]);
                    mma16816(pu[2 * half + 1], u, bl[2], bl[3]);
                }
#pragma unroll
                for (int t = 2 * ks; t < 2 * ks + 2; ++t) {   // Gamma dO (iq is a power of two)
                    const float2 cq = *reinterpret_cast<const float2 *>(scal + L::CQ * kChunk + 8 * t + tc);
                    const float2 iq = *reinterpret_cast<const float2 *>(scal + L::IQ * kChunk + 8 * t + tc);
                    const float gx = __fdividef(cq.x, iq.x), gy = __fdividef(cq.y, iq.y);
                    o[t][0] *= gx; o[t][1] *= gy; o[t][2] *= gx; o[t][3] *= gy;
                    m0 = fmaxf(m0, fmaxf(fabsf(o[t][0]), fabsf(o[t][1])));
                    m1 = fmaxf(m1, fmaxf(fabsf(o[t][2]), fabsf(o[t][3])));
                }
            }
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                pu[t][0] *= io0; pu[t][1] *= io0; pu[t][2] *= io1; pu[t][3] *= io1;
            }
            float iu0, iu1;
            const float fu0 = row_scale(quad_max(m0), iu0), fu1 = row_scale(quad_max(m1), iu1);
            const float gend = scal[L::MISC * kChunk];
            uint32_t oh[2][4], ol[2][4];
#pragma unroll
            for (int ks = 0; ks < 2; ++ks)
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const int t = 2 * ks + (x >> 1), c = (x & 1) * 2;
                    const float f = (x & 1) ? fu1 : fu0;
                    split_half(o[t][c] * f, o[t][c + 1] * f, oh[ks][x], ol[ks][x]);
                }
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
                    ldsm4_t(b0, sb + L::Q + (16 * ks + trow) * L::KP + tcol + c0 * 2 + i * 16);
                    ldsm4_t(b1, sb + L::Q + (16 * ks + trow) * L::KP + tcol + c0 * 2 + i * 16 + 32);
                    mma16816(acc[0], oh[ks], b0[0], b0[1]);
                    mma16816(acc[1], oh[ks], b0[2], b0[3]);
                    mma16816(acc[2], oh[ks], b1[0], b1[1]);
                    mma16816(acc[3], oh[ks], b1[2], b1[3]);
                    mma16816(acc[0], ol[ks], b0[0], b0[1]);
                    mma16816(acc[1], ol[ks], b0[2], b0[3]);
                    mma16816(acc[2], ol[ks], b1[0], b1[1]);
                    mma16816(acc[3], ol[ks], b1[2], b1[3]);
                }
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    z[i + t][0] = fmaf(gend, z[i + t][0], iu0 * acc[t][0]);
                    z[i + t][1] = fmaf(gend, z[i + t][1], iu0 * acc[t][1]);
                    z[i + t][2] = fmaf(gend, z[i + t][2], iu1 * acc[t][2]);
                    z[i + t][3] = fmaf(gend, z[i + t][3], iu1 * acc[t][3]);
                }
            }
        }
        if (KS == 2) {
            ok = pipe.wait(pipe.swapped + group, it & 1);
            if (!ok) break;
            const float4 *other = reinterpret_cast<const float4 *>(smem + M::SWAP) +
                                  (((group * 2 + (it & 1)) * 2 + (part ^ 1)) * XF / 4) * 32 + lane;
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const float4 x = other[t * 32];
                y[t][0] += x.x; y[t][1] += x.y; y[t][2] += x.z; y[t][3] += x.w;
            }
        }
        // dU = ik P'^T dO + exp(G_C - G) ik K' Z
        float e[4][4];
        {
            m0 = m1 = 0.f;
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const float2 ik = *reinterpret_cast<const float2 *>(scal + L::IK * kChunk + 8 * t + tc);
                const float2 ok2 = *reinterpret_cast<const float2 *>(scal + L::OK * kChunk + 8 * t + tc);
                y[t][0] = ik.x * pu[t][0] + ok2.x * y[t][0];
                y[t][1] = ik.y * pu[t][1] + ok2.y * y[t][1];
                y[t][2] = ik.x * pu[t][2] + ok2.x * y[t][2];
                y[t][3] = ik.y * pu[t][3] + ok2.y * y[t][3];
                m0 = fmaxf(m0, fmaxf(fabsf(y[t][0]), fabsf(y[t][1])));
                m1 = fmaxf(m1, fmaxf(fabsf(y[t][2]), fabsf(y[t][3])));
            }
            // E^T = dU^T X
            float iu0, iu1, el[4][4];
            const float fu0 = row_scale(quad_max(m0), iu0), fu1 = row_scale(quad_max(m1), iu1);
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int x = 0; x < 4; ++x) e[t][x] = el[t][x] = 0.f;
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) {
                uint32_t hi[4], lo[4];
                split_half(y[2 * ks][0] * fu0, y[2 * ks][1] * fu0, hi[0], lo[0]);
                split_half(y[2 * ks][2] * fu1, y[2 * ks][3] * fu1, hi[1], lo[1]);
                split_half(y[2 * ks + 1][0] * fu0, y[2 * ks + 1][1] * fu0, hi[2], lo[2]);
                split_half(y[2 * ks + 1][2] * fu1, y[2 * ks + 1][3] * fu1, hi[3], lo[3]);
#pragma unroll
                for (int half = 0; half <= ks; ++half) {
                    uint32_t xh[4], xl[4];
                    ldsm4_t(xh, sb + L::XH + (16 * ks + trow) * L::XP + tcol + half * 32);
                    ldsm4_t(xl, sb + L::XL + (16 * ks + trow) * L::XP + tcol + half * 32);
                    mma16816(e[2 * half], hi, xh[0], xh[1]);
                    mma16816(e[2 * half + 1], hi, xh[2], xh[3]);
                    mma16816(el[2 * half], lo, xh[0], xh[1]);
                    mma16816(el[2 * half + 1], lo, xh[2], xh[3]);
                    mma16816(el[2 * half], hi, xl[0], xl[1]);
                    mma16816(el[2 * half + 1], hi, xl[2], xl[3]);
                }
            }
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                e[t][0] = (e[t][0] + el[t][0]) * iu0;
                e[t][1] = (e[t][1] + el[t][1]) * iu0;
                e[t][2] = (e[t][2] + el[t][2]) * iu1;
                e[t][3] = (e[t][3] + el[t][3]) * iu1;
            }
        }
        {
            float *dst = args.e_out + (row * a.H + h) * a.dv + j0 + jr;
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const int tok = 8 * t + tc + (x & 1);
                    if (tok < valid && (KS == 1 || t / 2 == part))
                        dst[tok * vstride + (x >> 1) * 8] = e[t][x];
                }
        }
        // dV = dR = beta E; then Z -= (Gamma dR)^T K, in the scaled units of K'
        m0 = m1 = 0.f;
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const float2 b = *reinterpret_cast<const float2 *>(scal + L::BETA * kChunk + 8 * t + tc);
            const float2 ck = *reinterpret_cast<const float2 *>(scal + L::CK * kChunk + 8 * t + tc);
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                e[t][x] *= (x & 1) ? b.y : b.x;
                y[t][x] = -((x & 1) ? ck.y : ck.x) * e[t][x];
            }
            const __nv_bfloat162 w0 = __floats2bfloat162_rn(e[t][0], e[t][1]);
            const __nv_bfloat162 w1 = __floats2bfloat162_rn(e[t][2], e[t][3]);
            pk[t][0] = reinterpret_cast<const uint32_t &>(w0);
            pk[t][1] = reinterpret_cast<const uint32_t &>(w1);
            m0 = fmaxf(m0, fmaxf(fabsf(y[t][0]), fabsf(y[t][1])));
            m1 = fmaxf(m1, fmaxf(fabsf(y[t][2]), fabsf(y[t][3])));
        }
        {
            float iu0, iu1;
            const float fu0 = row_scale(quad_max(m0), iu0), fu1 = row_scale(quad_max(m1), iu1);
            uint32_t rh[2][4], rl[2][4];
#pragma unroll
            for (int ks = 0; ks < 2; ++ks)
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const int t = 2 * ks + (x >> 1), c = (x & 1) * 2;
                    const float f = (x & 1) ? fu1 : fu0;
                    split_half(y[t][c] * f, y[t][c + 1] * f, rh[ks][x], rl[ks][x]);
                }
            zm0 = zm1 = 0.f;
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
                    mma16816(acc[0], rh[ks], b0[0], b0[1]);
                    mma16816(acc[1], rh[ks], b0[2], b0[3]);
                    mma16816(acc[2], rh[ks], b1[0], b1[1]);
                    mma16816(acc[3], rh[ks], b1[2], b1[3]);
                    mma16816(acc[0], rl[ks], b0[0], b0[1]);
                    mma16816(acc[1], rl[ks], b0[2], b0[3]);
                    mma16816(acc[2], rl[ks], b1[0], b1[1]);
                    mma16816(acc[3], rl[ks], b1[2], b1[3]);
                }
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    z[i + t][0] = fmaf(iu0, acc[t][0], z[i + t][0]);
                    z[i + t][1] = fmaf(iu0, acc[t][1], z[i + t][1]);
                    z[i + t][2] = fmaf(iu1, acc[t][2], z[i + t][2]);
                    z[i + t][3] = fmaf(iu1, acc[t][3], z[i + t][3]);
                    zm0 = fmaxf(zm0, fmaxf(fabsf(z[i + t][0]), fabsf(z[i + t][1])));
                    zm1 = fmaxf(zm1, fmaxf(fabsf(z[i + t][2]), fabsf(z[i + t][3])));
                }
            }
        }
        if (KS == 1 || it + 1 == chunks) write_dv(row, valid);
        pipe.release(st);
    }
    if (ok && args.dstate_in) {
        float *out = args.dstate_in + state_off;
#pragma unroll
        for (int i = 0; i < NC; ++i)
#pragma unroll
            for (int x = 0; x < 4; ++x)
                out[(int64_t)(8 * i + (x & 1)) * a.dv + (x >> 1) * 8] = z[i][x];
    }
}

// ---------------------------------------------------------------- gradients of a block
constexpr int kBlock = 64;
constexpr int kGradWarps = 16, kGradThreads = kGradWarps * 32;

struct GradsArgs {
    const __nv_bfloat16 *q, *k, *dout, *g, *beta;
    const float *n_in, *e_in, *s_scales, *z_scales;
    const unsigned char *s_blocks, *z_blocks;
    const int32_t *cu, *owners;
    int64_t T, blocks;
    int Hk, H;
    uint32_t *err;
    uint32_t epoch;
    __nv_bfloat16 *dq, *dk, *dg, *dbeta;
};

template <int DK, int DV>
struct GradsSmem {
    static constexpr int KP = DK * 2 + 16, VP = DV * 2 + 16, MP = kBlock * 2 + 16;
    static constexpr int K = 0, Q = K + kBlock * KP;
    static constexpr int DO = Q + kBlock * KP, NN = DO + kBlock * VP, E = NN + kBlock * VP;
    static constexpr int S = E + kBlock * VP, Z = S + DK * VP;
    static constexpr int DP = Z + DK * VP, DA = DP + kBlock * MP;
    static constexpr int F = DA + kBlock * MP;   // floats from here
    // per-row values and partial sums
    enum { GH = 0, GL = 1, INTO = 2, OUT = 3, BETA = 4, DBETA = 5, ROW = 6 /* 4 */, STATE = 10 /* 4 */,
           WRITE = 14 /* 4 */, COL = 18 /* 4 */, COUNT = 22 };
    static constexpr int RED = F + COUNT * kBlock * 4;
    static constexpr int SC = RED + 6 * kGradWarps * 4;   // scales of S and Z: fp32 [2][DV / 16][2], then half2
    static constexpr int MU = SC + 2 * (DV / 16) * 2 * 4;
    static constexpr int BAR = MU + 2 * 2 * (DV / 16) * 4 + 4 * 4;
    static constexpr int BYTES = BAR + 16;
};

// A power of two that brings m (a tile's largest value) into [2^7, 2^8), and its inverse: a
// product of 128 such pairs stays below 2^23.
__device__ __forceinline__ float tile_scale(float m, float &inv) {
    int e = (int)((__float_as_uint(m) >> 23) & 255u);
    e = min(max(e, 16), 253);
    inv = __uint_as_float((uint32_t)(e - 7) << 23);
    return __uint_as_float((uint32_t)(261 - e) << 23);
}

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// C[16 rows][8 NT columns] = A B^T over K16 steps of 16, A [m][k] and B [n][k] fp16 in shared memory.
template <int NT, int K16>
__device__ __forceinline__ void product_nt(float (&c)[NT][4], uint32_t a, int ap, uint32_t b, int bp) {
    const int lane = threadIdx.x & 31;
    a += (lane & 15) * ap + (lane >> 4) * 16;
    b += ((lane & 7) + (lane >> 4) * 8) * bp + ((lane >> 3) & 1) * 16;
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int x = 0; x < 4; ++x) c[i][x] = 0.f;
#pragma unroll 2
    for (int kk = 0; kk < K16; ++kk) {
        uint32_t ra[4];
        ldsm4(ra, a + kk * 32);
#pragma unroll
        for (int i = 0; i < NT; i += 2) {
            uint32_t rb[4];
            ldsm4(rb, b + i * 8 * bp + kk * 32);
            mma16816(c[i], ra, rb[0], rb[1]);
            mma16816(c[i + 1], ra, rb[2], rb[3]);
        }
    }
}

// The same with the k steps of A times mult[kk]: powers of two that bring B's parts to one scale.
template <int NT, int K16>
__device__ __forceinline__ void product_nt_scaled(float (&c)[NT][4], uint32_t a, int ap, uint32_t b, int bp,
                                                  const __half2 *mult) {
    const int lane = threadIdx.x & 31;
    a += (lane & 15) * ap + (lane >> 4) * 16;
    b += ((lane & 7) + (lane >> 4) * 8) * bp + ((lane >> 3) & 1) * 16;
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int x = 0; x < 4; ++x) c[i][x] = 0.f;
#pragma unroll 2
    for (int kk = 0; kk < K16; ++kk) {
        uint32_t ra[4];
        ldsm4(ra, a + kk * 32);
        const __half2 m = mult[kk];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            const __half2 v = __hmul2(reinterpret_cast<const __half2 &>(ra[x]), m);
            ra[x] = reinterpret_cast<const uint32_t &>(v);
        }
#pragma unroll
        for (int i = 0; i < NT; i += 2) {
            uint32_t rb[4];
            ldsm4(rb, b + i * 8 * bp + kk * 32);
            mma16816(c[i], ra, rb[0], rb[1]);
            mma16816(c[i + 1], ra, rb[2], rb[3]);
        }
    }
}

// c += f A B over the k steps [k0, k1) of 16, B [k][n]; A [m][k], or [k][m] if TA.
template <int NT, bool TA>
__device__ __forceinline__ void product_add(float (&c)[NT][4], float f, uint32_t a, int ap, uint32_t b,
                                            int bp, int k0, int k1) {
    const int lane = threadIdx.x & 31;
    float acc[NT][4];
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int x = 0; x < 4; ++x) acc[i][x] = 0.f;
    a += TA ? ((lane & 7) + (lane >> 4) * 8) * ap + ((lane >> 3) & 1) * 16
            : (lane & 15) * ap + (lane >> 4) * 16;
    b += (lane & 15) * bp + (lane >> 4) * 16;
#pragma unroll 1
    for (int kk = k0; kk < k1; ++kk) {
        uint32_t ra[4];
        if (TA) ldsm4_t(ra, a + kk * 16 * ap);
        else ldsm4(ra, a + kk * 32);
#pragma unroll
        for (int i = 0; i < NT; i += 2) {
            uint32_t rb[4];
            ldsm4_t(rb, b + kk * 16 * bp + i * 16);
            mma16816(acc[i], ra, rb[0], rb[1]);
            mma16816(acc[i + 1], ra, rb[2], rb[3]);
        }
    }
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int x = 0; x < 4; ++x) c[i][x] = fmaf(f, acc[i][x], c[i][x]);
}

// Items are (64-token block, key head) pairs, spread over one CTA per SM; for each the CTA walks the
// value heads of the key head's group and sums dq and dk over them in registers, in order.  Warp w has
// rows 16 (w % 4) .. and the quarter w / 4 of the columns.  S and Z of the next head are copied in as
// soon as the last product with the present ones is done.
template <int DK, int DV>
__global__ void __launch_bounds__(kGradThreads, 1) gdr_grads_kernel(GradsArgs a) {
    using M = GradsSmem<DK, DV>;
    constexpr int NF = DK / 32;   // column tiles of a warp in [64][DK] results
    constexpr int G = DV / 16;    // column groups of S and Z with a scale each
    extern __shared__ __align__(1024) unsigned char smem[];
    float *rows = reinterpret_cast<float *>(smem + M::F);
    float *red = reinterpret_cast<float *>(smem + M::RED);
    float *sc = reinterpret_cast<float *>(smem + M::SC);            // [S, Z][G][2] inverse scales
    __half2 *mult = reinterpret_cast<__half2 *>(smem + M::MU);      // [S, Z][2][G], relative to the largest
    float *top = reinterpret_cast<float *>(smem + M::MU + 2 * 2 * G * 4);   // [S, Z][2]: the largest
    uint64_t *bar = reinterpret_cast<uint64_t *>(smem + M::BAR);
    volatile uint32_t *abort = reinterpret_cast<volatile uint32_t *>(bar + 1);
    const uint32_t sb = smem_u32(smem);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int wm = warp & 3, wn = warp >> 2, r0 = lane >> 2, cc = 2 * (lane & 3);
    const int group = a.H / a.Hk;
    const int64_t items = a.blocks * a.Hk;

    if (tid == 0) {
        mbar_init(bar, 1);
        mbar_fence_init();
        *abort = 0u;
    }
    __syncthreads();
    // the next item at or behind `i` whose block belongs to a sequence
    auto next_item = [&](int64_t i) {
        while (i < items && a.owners[i / a.Hk] < 0) i += gridDim.x;
        return i;
    };
    auto fetch_states = [&](int64_t i, int hg) {   // one thread
        const int64_t unit = (i / a.Hk) * a.H + (i % a.Hk) * group + hg;
        mbar_arrive_expect_tx(bar, 2 * DK * M::VP);
        bulk_load(sb + M::S, a.s_blocks + unit * DK * M::VP, DK * M::VP, bar);
        bulk_load(sb + M::Z, a.z_blocks + unit * DK * M::VP, DK * M::VP, bar);
    };
    uint32_t parity = 0;
    int64_t item = next_item(blockIdx.x);
    if (tid == 0 && item < items) fetch_states(item, 0);
    for (; item < items;) {
    const int64_t after = next_item(item + gridDim.x);
    const int hk = (int)(item % a.Hk);
    const int64_t slot = item / a.Hk;
    const int n = a.owners[slot];
    const Span span = sequence_span(a.cu, n, a.T);
    const int blk = (int)(slot - first_block(span, n));
    const int valid = min(kBlock, span.len - blk * kBlock);
    const int64_t row0 = span.row + (int64_t)blk * kBlock;

    // 64 rows of D elements as fp16 tiles with one power-of-two scale: loaded, and once the largest
    // value over the CTA is known, stored.  All of a head's tiles are loaded before any is waited for.
    auto load_bf16 = [&](auto dconst, auto &w, const __nv_bfloat16 *src, int64_t stride) {
        constexpr int D = decltype(dconst)::value, PER = kBlock * D / 8 / kGradThreads;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int x = i * kGradThreads + tid, r = x / (D / 8), c = x % (D / 8);
            w[i] = make_uint4(0u, 0u, 0u, 0u);
            if (r < valid) w[i] = __ldg(reinterpret_cast<const uint4 *>(src + r * stride) + c);
        }
    };
    auto load_f32 = [&](auto &w, const float *src, int64_t stride) {
        constexpr int PER = kBlock * DV / 4 / kGradThreads;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int x = i * kGradThreads + tid, r = x / (DV / 4), c = x % (DV / 4);
            w[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (r < valid) w[i] = __ldcs(reinterpret_cast<const float4 *>(src + r * stride) + c);
        }
    };
    // largest magnitude of this warp's values to a slot of `red`, and of the CTA's from it
    auto max_bf16 = [&](const auto &w, int at) {
        float m = 0.f;
        for (const uint4 &x : w)
            for (uint32_t u : {x.x, x.y, x.z, x.w}) m = fmaxf(m, fmaxf(fabsf(bf_lo(u)), fabsf(bf_hi(u))));
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
        if (lane == 0) red[at * kGradWarps + warp] = m;
    };
    auto max_f32 = [&](const auto &w, int at) {
        float m = 0.f;
        for (const float4 &x : w)
            m = fmaxf(m, fmaxf(fmaxf(fabsf(x.x), fabsf(x.y)), fmaxf(fabsf(x.z), fabsf(x.w))));
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
        if (lane == 0) red[at * kGradWarps + warp] = m;
    };
    auto cta_scale = [&](int at, float &inv) {
        float m = red[at * kGradWarps + (lane & (kGradWarps - 1))];
#pragma unroll
        for (int x = kGradWarps / 2; x > 0; x >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
        return tile_scale(m, inv);
    };
    auto store_bf16 = [&](auto dconst, const auto &w, int dst, int pitch, float f) {
        constexpr int D = decltype(dconst)::value, PER = kBlock * D / 8 / kGradThreads;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int x = i * kGradThreads + tid, r = x / (D / 8), c = x % (D / 8);
            *reinterpret_cast<uint4 *>(smem + dst + r * pitch + c * 16) =
                make_uint4(pack_half(bf_lo(w[i].x) * f, bf_hi(w[i].x) * f),
                           pack_half(bf_lo(w[i].y) * f, bf_hi(w[i].y) * f),
                           pack_half(bf_lo(w[i].z) * f, bf_hi(w[i].z) * f),
                           pack_half(bf_lo(w[i].w) * f, bf_hi(w[i].w) * f));
        }
    };
    auto store_f32 = [&](const auto &w, int dst, float f) {
        constexpr int PER = kBlock * DV / 4 / kGradThreads;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int x = i * kGradThreads + tid, r = x / (DV / 4), c = x % (DV / 4);
            *reinterpret_cast<uint2 *>(smem + dst + r * M::VP + c * 8) =
                make_uint2(pack_half(w[i].x * f, w[i].y * f), pack_half(w[i].z * f, w[i].w * f));
        }
    };

    using DKc = std::integral_constant<int, DK>;
    using DVc = std::integral_constant<int, DV>;
    const int64_t koff = (row0 * a.Hk + hk) * DK, kstride = (int64_t)a.Hk * DK;
    float sk, sq;
    {
        uint4 wk[kBlock * DK / 8 / kGradThreads], wq[kBlock * DK / 8 / kGradThreads];
        load_bf16(DKc{}, wk, a.k + koff, kstride);
        load_bf16(DKc{}, wq, a.q + koff, kstride);
        max_bf16(wk, 0);
        max_bf16(wq, 1);
        __syncthreads();
        store_bf16(DKc{}, wk, M::K, M::KP, cta_scale(0, sk));
        store_bf16(DKc{}, wq, M::Q, M::KP, cta_scale(1, sq));
    }
    __syncthreads();
    // Q K^T and K K^T, columns 16 wn ..
    float qk[2][4], kk[2][4];
    product_nt<2, DK / 16>(qk, sb + M::Q + wm * 16 * M::KP, M::KP, sb + M::K + wn * 16 * M::KP, M::KP);
    product_nt<2, DK / 16>(kk, sb + M::K + wm * 16 * M::KP, M::KP, sb + M::K + wn * 16 * M::KP, M::KP);

    float dq[NF][4], dk[NF][4];
#pragma unroll
    for (int i = 0; i < NF; ++i)
#pragma unroll
        for (int x = 0; x < 4; ++x) dq[i][x] = dk[i][x] = 0.f;

#pragma unroll 1
    for (int hg = 0; hg < group; ++hg) {
        const int h = hk * group + hg;
        const int64_t voff = (row0 * a.H + h) * DV, vstride = (int64_t)a.H * DV, unit = slot * a.H + h;
        uint4 wo[kBlock * DV / 8 / kGradThreads];
        float4 wnn[kBlock * DV / 4 / kGradThreads], we[kBlock * DV / 4 / kGradThreads];
        load_bf16(DVc{}, wo, a.dout + voff, vstride);
        load_f32(wnn, a.n_in + voff, vstride);
        load_f32(we, a.e_in + voff, vstride);
        float scale = 0.f;
        if (tid < 4 * G) scale = tid < 2 * G ? a.s_scales[unit * 2 * G + tid] : a.z_scales[unit * 2 * G + tid - 2 * G];
        __syncthreads();   // the head before has been read
        if (warp == 0) {
            // rows 2 lane and 2 lane + 1: running sums in 64 bits
            float g[2], b[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int r = 2 * lane + i;
                g[i] = b[i] = 0.f;
                if (r < valid) {
                    g[i] = log_decay(__bfloat162float(a.g[(row0 + r) * a.H + h]));
                    b[i] = __bfloat162float(a.beta[(row0 + r) * a.H + h]);
                }
            }
            double G = (double)g[0] + (double)g[1];
#pragma unroll
            for (int m = 1; m < 32; m <<= 1) {
                const double o = __shfl_up_sync(0xffffffffu, G, m);
                if (lane >= m) G += o;
            }
            const double Gend = __shfl_sync(0xffffffffu, G, 31);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int r = 2 * lane + i;
                const double Gr = i ? G : G - (double)g[1], G2 = Gr * 1.4426950408889634074;
                rows[M::GH * kBlock + r] = (float)G2;
                rows[M::GL * kBlock + r] = (float)(G2 - (double)(float)G2);
                rows[M::INTO * kBlock + r] = decay((float)Gr);
                rows[M::OUT * kBlock + r] = decay((float)(Gend - Gr));
                rows[M::BETA * kBlock + r] = b[i];
            }
        }
        if (tid < 4 * G) sc[tid] = scale;
        max_bf16(wo, 2);
        max_f32(wnn, 3);
        max_f32(we, 4);
        __syncthreads();
        float so, sn, se;
        store_bf16(DVc{}, wo, M::DO, M::VP, cta_scale(2, so));
        store_f32(wnn, M::NN, cta_scale(3, sn));
        store_f32(we, M::E, cta_scale(4, se));
        // S and Z: their scales, and <S, Z>
        if (tid < 4) {   // the largest of a half, and the groups' scales relative to it
            const int which = tid >> 1, half = tid & 1;
            float t = 0.f;
            for (int g = 0; g < G; ++g) t = fmaxf(t, sc[(which * G + g) * 2 + half]);
            top[tid] = t;
            for (int g = 0; g < G; ++g)
                mult[tid * G + g] = __float2half2_rn(__fdividef(sc[(which * G + g) * 2 + half], t));
        }
        const bool late = !warp_wait(bar, parity, a.err, a.epoch, abort);
        parity ^= 1u;
        {
            float dot = 0.f;
#pragma unroll 2
            for (int x = tid; x < DK * DV / 8; x += kGradThreads) {
                const int c = x / (DV / 8), j = x % (DV / 8), half = c >= DK / 2;
                const uint4 u = *reinterpret_cast<const uint4 *>(smem + M::S + c * M::VP + j * 16);
                const uint4 v = *reinterpret_cast<const uint4 *>(smem + M::Z + c * M::VP + j * 16);
                const uint32_t uu[4] = {u.x, u.y, u.z, u.w}, vv[4] = {v.x, v.y, v.z, v.w};
                float d = 0.f;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 p = __half22float2(reinterpret_cast<const __half2 &>(uu[e]));
                    const float2 q = __half22float2(reinterpret_cast<const __half2 &>(vv[e]));
                    d = fmaf(p.x, q.x, fmaf(p.y, q.y, d));
                }
                dot += d * sc[(j / 2) * 2 + half] * sc[(G + j / 2) * 2 + half];
            }
#pragma unroll
            for (int x = 16; x > 0; x >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, x);
            if (lane == 0) red[5 * kGradWarps + warp] = dot;
        }
        if (__syncthreads_or(late)) {   // the whole CTA leaves, S and Z landed (a bounded wait)
            if (tid == 0) mbar_wait(bar, parity ^ 1u, a.err);
            return;
        }

        const int ra = wm * 16 + r0, rb = ra + 8;   // this lane's rows
        const float ba = rows[M::BETA * kBlock + ra], bb = rows[M::BETA * kBlock + rb];
        const float ia = rows[M::INTO * kBlock + ra], ib = rows[M::INTO * kBlock + rb];
        // fp16 copies of dP and dA in units of the operands' scales, at most 2^15 for beta <= 4
        constexpr float kDown = 1.f / 4096.f;
        {
            float m1[2][4], m2[2][4], sum[2] = {0.f, 0.f}, col[2][2];
            product_nt<2, DV / 16>(m1, sb + M::DO + wm * 16 * M::VP, M::VP, sb + M::NN + wn * 16 * M::VP, M::VP);
            product_nt<2, DV / 16>(m2, sb + M::E + wm * 16 * M::VP, M::VP, sb + M::NN + wn * 16 * M::VP, M::VP);
            const float w1 = so * sn * (sq * sk), w2 = se * sn * (sk * sk);
            const float gha = rows[M::GH * kBlock + ra], gla = rows[M::GL * kBlock + ra];
            const float ghb = rows[M::GH * kBlock + rb], glb = rows[M::GL * kBlock + rb];
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                float p[4], d[4];
                col[t][0] = col[t][1] = 0.f;
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const int s = wn * 16 + t * 8 + cc + (x & 1), r = x < 2 ? ra : rb;
                    const float hs = rows[M::GH * kBlock + s], ls = rows[M::GL * kBlock + s];
                    const float bs = rows[M::BETA * kBlock + s];
                    const float D = s <= r ? exp2_approx(((x < 2 ? gha : ghb) - hs) + ((x < 2 ? gla : glb) - ls)) : 0.f;
                    if (s == r) rows[M::DBETA * kBlock + r] = m2[t][x] * se * sn;
                    p[x] = D * bs * m1[t][x];
                    d[x] = s < r ? -(x < 2 ? ba : bb) * bs * D * m2[t][x] : 0.f;
                    const float w = s < r ? p[x] * qk[t][x] * w1 + d[x] * kk[t][x] * w2 : 0.f;
                    sum[x >> 1] += w;
                    col[t][x & 1] += w;
                }
#pragma unroll
                for (int x = 0; x < 4; x += 2) {
                    const int at = (x ? rb : ra) * M::MP + (wn * 16 + t * 8 + cc) * 2;
                    *reinterpret_cast<uint32_t *>(smem + M::DP + at) = pack_half(p[x] * kDown, p[x + 1] * kDown);
                    *reinterpret_cast<uint32_t *>(smem + M::DA + at) = pack_half(d[x] * kDown, d[x + 1] * kDown);
                }
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], 1);
                sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], 2);
                if ((lane & 3) == 0) rows[(M::ROW + wn) * kBlock + (i ? rb : ra)] = sum[i];
            }
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
#pragma unroll
                    for (int m = 4; m < 32; m <<= 1) col[t][x] += __shfl_xor_sync(0xffffffffu, col[t][x], m);
                    if (lane < 4) rows[(M::COL + wm) * kBlock + wn * 16 + t * 8 + cc + x] = col[t][x];
                }
        }
        // the state's share: rows of dO S^T, E S^T and N Z^T, columns 8 NF wn ..
        {
            float f[NF][4], state[2] = {0.f, 0.f}, write[2] = {0.f, 0.f};
            const uint32_t bs = sb + M::S + wn * NF * 8 * M::VP, bz = sb + M::Z + wn * NF * 8 * M::VP;
            const int half = wn >> 1;   // of the channels: this warp's columns
            const float ss = top[half], sz = top[2 + half];
            const __half2 *ms = mult + half * G, *mz = mult + (2 + half) * G;
            // dot of the rows of f with the rows of a [64][DK] tile in shared memory
            auto row_dot = [&](int tile, float wa, float wb, float (&s)[2]) {
                float x0 = 0.f, x1 = 0.f;
#pragma unroll
                for (int i = 0; i < NF; ++i) {
                    const int at = (wn * NF + i) * 16 + cc * 2;
                    const float2 u = __half22float2(*reinterpret_cast<const __half2 *>(smem + tile + ra * M::KP + at));
                    const float2 v = __half22float2(*reinterpret_cast<const __half2 *>(smem + tile + rb * M::KP + at));
                    x0 += f[i][0] * u.x + f[i][1] * u.y;
                    x1 += f[i][2] * v.x + f[i][3] * v.y;
                }
                s[0] += wa * x0;
                s[1] += wb * x1;
            };
            auto add = [&](float (&acc)[NF][4], float wa, float wb) {
#pragma unroll
                for (int i = 0; i < NF; ++i) {
                    acc[i][0] = fmaf(wa, f[i][0], acc[i][0]);
                    acc[i][1] = fmaf(wa, f[i][1], acc[i][1]);
                    acc[i][2] = fmaf(wb, f[i][2], acc[i][2]);
                    acc[i][3] = fmaf(wb, f[i][3], acc[i][3]);
                }
            };
            product_nt_scaled<NF, DV / 16>(f, sb + M::DO + wm * 16 * M::VP, M::VP, bs, M::VP, ms);
            add(dq, ia * so * ss, ib * so * ss);
            row_dot(M::Q, ia * so * ss * sq, ib * so * ss * sq, state);
            product_nt_scaled<NF, DV / 16>(f, sb + M::E + wm * 16 * M::VP, M::VP, bs, M::VP, ms);
            add(dk, -ia * ba * se * ss, -ib * bb * se * ss);
            row_dot(M::K, -ia * ba * se * ss * sk, -ib * bb * se * ss * sk, state);
            const float oa = rows[M::OUT * kBlock + ra] * ba, ob = rows[M::OUT * kBlock + rb] * bb;
            product_nt_scaled<NF, DV / 16>(f, sb + M::NN + wm * 16 * M::VP, M::VP, bz, M::VP, mz);
            add(dk, oa * sn * sz, ob * sn * sz);
            row_dot(M::K, oa * sn * sz * sk, ob * sn * sz * sk, write);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                state[i] += __shfl_xor_sync(0xffffffffu, state[i], 1);
                state[i] += __shfl_xor_sync(0xffffffffu, state[i], 2);
                write[i] += __shfl_xor_sync(0xffffffffu, write[i], 1);
                write[i] += __shfl_xor_sync(0xffffffffu, write[i], 2);
                if ((lane & 3) == 0) {
                    rows[(M::STATE + wn) * kBlock + (i ? rb : ra)] = state[i];
                    rows[(M::WRITE + wn) * kBlock + (i ? rb : ra)] = write[i];
                }
            }
        }
        fence_proxy_async_shared();   // S and Z have been read: the next ones may come
        __syncthreads();
        if (tid == 0) {
            if (hg + 1 < group) fetch_states(item, hg + 1);
            else if (after < items) fetch_states(after, 0);
        }
        // dP and dA are lower triangular: rows 16 wm need columns up to 16 wm + 15, and the
        // transposed products rows from 16 wm
        const float up1 = so * sn / kDown, up2 = se * sn / kDown;
        const int c8 = wn * NF * 16;
        product_add<NF, false>(dq, up1 * sk, sb + M::DP + wm * 16 * M::MP, M::MP, sb + M::K + c8, M::KP, 0, wm + 1);
        product_add<NF, false>(dk, up2 * sk, sb + M::DA + wm * 16 * M::MP, M::MP, sb + M::K + c8, M::KP, 0, wm + 1);
        product_add<NF, true>(dk, up1 * sq, sb + M::DP + wm * 32, M::MP, sb + M::Q + c8, M::KP, wm, 4);
        product_add<NF, true>(dk, up2 * sk, sb + M::DA + wm * 32, M::MP, sb + M::K + c8, M::KP, wm, 4);
        if (warp == 0) {
            // rows 2 lane, 2 lane + 1: the sum from a row on, and of what is written before it
            float from[2], w[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float *p = rows + 2 * lane + i;
                auto four = [&](int at) {
                    return (p[at * kBlock] + p[(at + 1) * kBlock]) + (p[(at + 2) * kBlock] + p[(at + 3) * kBlock]);
                };
                from[i] = four(M::ROW) - four(M::COL) + four(M::STATE);
                w[i] = four(M::WRITE);
            }
            float suf = from[0] + from[1], pre = w[0] + w[1];
#pragma unroll
            for (int m = 1; m < 32; m <<= 1) {
                const float x = __shfl_down_sync(0xffffffffu, suf, m), y = __shfl_up_sync(0xffffffffu, pre, m);
                if (lane + m < 32) suf += x;
                if (lane >= m) pre += y;
            }
            float d = 0.f;
#pragma unroll
            for (int i = 0; i < kGradWarps; ++i) d += red[5 * kGradWarps + i];
            d *= rows[M::INTO * kBlock + kBlock - 1];
            const float before = pre - w[0] - w[1];
            const float dg[2] = {suf + before + d, suf - from[0] + before + w[0] + d};
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int r = 2 * lane + i;
                if (r < valid) {
                    a.dg[(row0 + r) * a.H + h] = __float2bfloat16_rn(dg[i]);
                    a.dbeta[(row0 + r) * a.H + h] = __float2bfloat16_rn(rows[M::DBETA * kBlock + r]);
                }
            }
        }
    }
#pragma unroll
    for (int i = 0; i < NF; ++i)
#pragma unroll
        for (int x = 0; x < 4; x += 2) {
            const int r = wm * 16 + r0 + (x ? 8 : 0);
            if (r >= valid) continue;
            const int64_t at = ((row0 + r) * a.Hk + hk) * DK + (wn * NF + i) * 8 + cc;
            *reinterpret_cast<__nv_bfloat162 *>(a.dq + at) = __floats2bfloat162_rn(dq[i][x], dq[i][x + 1]);
            *reinterpret_cast<__nv_bfloat162 *>(a.dk + at) = __floats2bfloat162_rn(dk[i][x], dk[i][x + 1]);
        }
    item = after;
    __syncthreads();   // K and Q have been read
    }
}

// ---------------------------------------------------------------- launches
template <int DK, int NCW, int KS>
static cudaError_t launch_adjoint_t(const AdjointArgs &a, const void *dout, int64_t rows, int64_t units,
                                    cudaStream_t st) {
    using M = Pipe<DK, NCW, KS, true, true, 0>;
    return launch_chain_kernel(gdr_adjoint_kernel<DK, NCW, KS>, a, dout, rows, M::W, units, M::WARPS * 32, M::BYTES,
                               st);
}

template <int DK>
static cudaError_t launch_adjoint_d(const AdjointArgs &a, const void *dout, int64_t rows, int64_t units,
                                    cudaStream_t st) {
    switch (chain_variant(units, a.in.dv, a.in.cu != nullptr)) {
        case 22: return launch_adjoint_t<DK, 2, 2>(a, dout, rows, units, st);
        case 41: return launch_adjoint_t<DK, 4, 1>(a, dout, rows, units, st);
        default: return launch_adjoint_t<DK, 8, 1>(a, dout, rows, units, st);
    }
}

template <int DK, int DV>
static cudaError_t launch_grads_t(const GradsArgs &a, int64_t blocks, cudaStream_t st) {
    constexpr int bytes = GradsSmem<DK, DV>::BYTES;
    static_assert(bytes <= 227 * 1024, "shared memory of a CTA");
    cudaError_t e = cudaFuncSetAttribute(gdr_grads_kernel<DK, DV>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    const int64_t items = blocks * a.Hk;
    gdr_grads_kernel<DK, DV><<<(unsigned)(items < 148 ? items : 148), kGradThreads, bytes, st>>>(a);
    e = cudaGetLastError();
    Profiler::mark(st);
    return e;
}

static int64_t block_slots(int64_t rows, int N) { return rows / kBlock + N + 1; }
static size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }

}  // namespace gdr

size_t gdr_backward_workspace_bytes(int64_t rows, int N, int Hk, int H, int dk, int dv, bool bf16) {
    using namespace gdr;
    if (!bf16) return token_backward_workspace_bytes(rows, N, H, dk, dv);
    const size_t slots = (size_t)block_slots(rows, N) * H;
    return 2 * (up256((size_t)rows * H * dv * 4) + up256(slots * dk * block_row(dv)) + up256(slots * (dv / 8) * 4)) +
           up256(slots / H * 4) + gdr_image_bytes(rows, N, Hk, H, dk, true);
}

cudaError_t launch_gdr_backward(const GdrArgs &p, const GdrGrads &g, int64_t rows, bool bf16,
                                void *workspace, cudaStream_t st) {
    using namespace gdr;
    using bf = __nv_bfloat16;
    if (!bf16) return launch_token_backward(p, g, rows, workspace, st);
    const size_t slots = (size_t)block_slots(rows, p.N) * p.H;
    unsigned char *w = static_cast<unsigned char *>(workspace);
    auto take = [&](size_t bytes) {
        float *r = reinterpret_cast<float *>(w);
        w += up256(bytes);
        return r;
    };
    GdrBackwardSpace s;
    s.n = take((size_t)rows * p.H * p.dv * 4);
    s.e = take((size_t)rows * p.H * p.dv * 4);
    s.s_blocks = reinterpret_cast<unsigned char *>(take(slots * p.dk * block_row(p.dv)));
    s.z_blocks = reinterpret_cast<unsigned char *>(take(slots * p.dk * block_row(p.dv)));
    s.s_scales = take(slots * (p.dv / 8) * 4);
    s.z_scales = take(slots * (p.dv / 8) * 4);
    s.owners = reinterpret_cast<int32_t *>(take(slots / p.H * 4));
    cudaError_t e = cudaMemsetAsync(s.owners, 0xff, slots / p.H * 4, st);
    if (e != cudaSuccess) return e;
    const GdrImages m = gdr_images(w, p, true);
    e = launch_gdr_prep(p, m, st);
    if (e != cudaSuccess) return e;
    e = launch_gdr_recompute(p, m, s, st);
    if (e != cudaSuccess) return e;
    const int64_t units = (int64_t)p.N * p.H;
    AdjointArgs a{{m.keys, m.adjoint, p.cu_seqlens, m.order, p.T, p.Hk, p.H, p.dv, p.err, p.epoch},
                  g.dstate_out, (bf *)g.dv, g.dstate_in, s.e, s.z_blocks, s.z_scales};
    e = p.dk == 64 ? launch_adjoint_d<64>(a, g.dout, rows, units, st) : launch_adjoint_d<128>(a, g.dout, rows, units, st);
    if (e != cudaSuccess) return e;
    GradsArgs b{(const bf *)p.q, (const bf *)p.k, (const bf *)g.dout, (const bf *)p.g, (const bf *)p.beta,
                s.n, s.e, s.s_scales, s.z_scales, s.s_blocks, s.z_blocks, p.cu_seqlens, s.owners, p.T,
                block_slots(rows, p.N), p.Hk, p.H, p.err, p.epoch,
                (bf *)g.dq, (bf *)g.dk, (bf *)g.dg, (bf *)g.dbeta};
    const int64_t blocks = block_slots(rows, p.N);
    if (p.dk == 64) return p.dv == 64 ? launch_grads_t<64, 64>(b, blocks, st) : launch_grads_t<64, 128>(b, blocks, st);
    return p.dv == 64 ? launch_grads_t<128, 64>(b, blocks, st) : launch_grads_t<128, 128>(b, blocks, st);
}

}  // namespace kda
