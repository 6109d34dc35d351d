// Device helpers shared by the gated-delta-rule kernels: warp matrix products, the two-term
// fp16 split of fp32 operands, sequence bounds, the layout of a chunk and the pipeline that
// feeds it to the chain kernels.
#pragma once

#include "kda_common.cuh"
#include "kda_launch.h"
#include "kda_tma.h"

#include <cuda_fp16.h>

namespace kda {
namespace gdr {

constexpr int kChunk = 32;          // tokens per chunk of the chained kernels
constexpr float kMinLogDecay = -100.f;
// Limits of the bf16 calls (kda.h): beta |k|^2, beta |k_r| |k_s| in a chunk, beta in the backward.
constexpr float kMaxStep = 2.f + 1.f / 32, kMaxCross = 16384.f, kMaxBeta = 4.f;
// A log-decay, -infinity among them, as the kernels sum it: not below the clamp.  A NaN stays one.
__device__ __forceinline__ float log_decay(float g) { return g < kMinLogDecay ? kMinLogDecay : g; }
// exp of a log-decay or a sum of them, exactly 0 from the clamp down: a token that forgets leaves nothing
// of any state (exp(-100) is 3.7e-44, which is something beside a state of 1e38).
// (A choice between 0 and expf(g) becomes a branch, which took the fp32 prefill from 62 to 82 us.)
__device__ __forceinline__ float decay(float g) { return expf(g <= kMinLogDecay ? -INFINITY : g); }

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
// Contiguous bytes (a multiple of 16, both addresses 16-byte aligned) to and from shared memory.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::
            "r"(dst), "l"(src), "r"(bytes), "r"(smem_u32(bar))
        : "memory");
}
__device__ __forceinline__ void bulk_store(void *dst, uint32_t src, uint32_t bytes) {
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(src),
                 "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ void bulk_store_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
// This thread's bulk stores have read their shared memory / have been written.
__device__ __forceinline__ void bulk_store_wait_read() {
    asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
}
__device__ __forceinline__ void bulk_store_wait() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }
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

// The state before (or the adjoint state behind) a 64-token block as the block kernel reads it: fp16
// [DK][dv] in padded rows, each warp's part scaled by a power of two; the inverse scales lie beside it
// in [dv / 16][2] slots, one for each half of the channels (both written where one warp has them all).
__host__ __device__ constexpr int block_row(int dv) { return dv * 2 + 16; }
// One chain warp's part: channels c0 .. c0 + 8 NC - 1 of columns j0 .. j0 + 15.  m: this lane's largest
// magnitude.  `tile`: 32 rows of shared memory of this warp's own, at a pitch of 48 bytes.
template <int NC>
__device__ __forceinline__ void store_block(unsigned char *image, float *scale, const float (&s)[NC][4], float m,
                                            int halves, int part, int c0, int j0, int dv, unsigned char *tile) {
    constexpr int OP = 48;
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
    float inv;
    const float f = row_scale(m, inv);
    if (halves == 2 ? lane == 0 : lane < 2) scale[halves == 2 ? part : lane] = inv;
    const int nrow = (lane & 7) + (lane >> 4) * 8, ncol = ((lane >> 3) & 1) * 16;
#pragma unroll
    for (int i = 0; i < NC; i += 4) {
        __syncwarp();   // the rows before have been read
#pragma unroll
        for (int t = 0; t < 4; t += 2)
            stsm4_t(smem_u32(tile) + (8 * t + nrow) * OP + ncol, pack_half(s[i + t][0] * f, s[i + t][1] * f),
                    pack_half(s[i + t][2] * f, s[i + t][3] * f),
                    pack_half(s[i + t + 1][0] * f, s[i + t + 1][1] * f),
                    pack_half(s[i + t + 1][2] * f, s[i + t + 1][3] * f));
        __syncwarp();
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int c = u * 16 + (lane >> 1);
            *reinterpret_cast<uint4 *>(image + (c0 + 8 * i + c) * block_row(dv) + j0 * 2 + (lane & 1) * 16) =
                *reinterpret_cast<const uint4 *>(tile + c * OP + (lane & 1) * 16);
        }
    }
    __syncwarp();
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
// First 32-token chunk of a sequence in the arrays of chunk images, and first 64-token block in the
// backward's per-block arrays: distinct
// for all sequences, since a sequence of len rows from `row` has at most
// (row + len) / 64 - row / 64 + 1 blocks (chunks likewise).
__device__ __forceinline__ int64_t first_block(const Span &s, int n) { return s.row / 64 + n; }
__device__ __forceinline__ int64_t first_chunk(const Span &s, int n) { return s.row / kChunk + n; }
__host__ __device__ __forceinline__ int64_t chunk_slots(int64_t rows, int N) { return rows / kChunk + N + 1; }

// ---------------------------------------------------------------- a chunk in shared memory
// A chunk as the chain reads it.  The keys and queries of a key head and what follows from them
// for a value head are made once per chunk by gdr_prep_kernel and lie in global memory as images of
// these tiles; the values come from the input tensor.  Rows are padded by 16 bytes, so the eight
// rows of an ldmatrix lie in different banks.
template <int DK>
struct KeyImage {   // per (chunk, key head): scaled keys and queries, fp16 [32][DK]
    static constexpr int KP = DK * 2 + 16;
    static constexpr int K = 0, Q = kChunk * KP, BYTES = 2 * kChunk * KP;
};
// per (chunk, value head): X = (I + A)^-1 as fp16 hi + lo, per-row scalars (8 x 32 fp32), P as fp16
// hi (+ lo for the adjoint)
template <bool ADJ>
struct HeadImage {
    static constexpr int XP = kChunk * 2 + 16;
    static constexpr int XH = 0, XL = XH + kChunk * XP, S = XL + kChunk * XP, P = S + 8 * kChunk * 4;
    static constexpr int PL = P + kChunk * XP, BYTES = PL + (ADJ ? kChunk * XP : 0);
    // rows of the scalars: IK, IQ inverse scales of k and q; CK, CQ = Gamma times them; OK =
    // exp(G_end - G) ik (times beta in the forward's image); BK = beta ik; MISC[0] = exp(G_end)
    enum { IK = 0, CK = 1, OK = 2, BETA = 3, IQ = 4, CQ = 5, MISC = 6, BK = 7 };
};

template <int DK, int W, bool ADJ, bool WANT_Q>
struct Stage {
    using KI = KeyImage<DK>;
    using HI = HeadImage<ADJ>;
    static constexpr int KP = KI::KP, XP = HI::XP;
    static constexpr int K = 0, Q = KI::Q, KEYS = WANT_Q ? KI::BYTES : KI::Q;   // queries where wanted
    static constexpr int HEAD = KEYS, HEADS = WANT_Q ? HI::BYTES : HI::P;       // P with the queries
    static constexpr int XH = HEAD + HI::XH, XL = HEAD + HI::XL, S = HEAD + HI::S, P = HEAD + HI::P,
                         PL = HEAD + HI::PL;
    static constexpr int V = (HEAD + HEADS + 1023) / 1024 * 1024;
    static constexpr int VBYTES = kChunk * W * 2;
    static constexpr int BYTES = (V + VBYTES + 1023) / 1024 * 1024;
    enum { IK = HI::IK, CK = HI::CK, OK = HI::OK, BETA = HI::BETA, IQ = HI::IQ, CQ = HI::CQ, MISC = HI::MISC,
           BK = HI::BK };
    // 16-byte piece c of row r of the values (or output gradients), bf16 as the TMA writes them:
    // panels of 64 columns with the 128-byte swizzle, or one plain panel of 32
    static __device__ __forceinline__ int v_at(int r, int c) {
        return V + (W < 64 ? r * 64 + c * 16 : (c >> 3) * 4096 + r * 128 + (((c & 7) ^ (r & 7)) << 4));
    }
};

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

// ---------------------------------------------------------------- the chain kernels' pipeline
// What both chain kernels get.
struct ChainInput {
    const unsigned char *keys, *heads;   // images: [chunk_slots, Hk], [chunk_slots, H]
    const int32_t *cu, *order;           // order: sequences from the longest, or nullptr
    int64_t T;
    int Hk, H, dv;
    uint32_t *err;
    uint32_t epoch;
};

// NCW groups of 16 value columns per CTA, KS warps per group (each with dk / KS channels).  A loader
// warp copies chunk after chunk into a ring of ST stages: two images and a box of the values.  With
// OUTW > 0 an output warp per group finishes what the chain leaves it, OUTW bytes a chunk and group in
// a buffer per stage (so that a full stage's buffer is free: the output warp has released it too).
//
// The chain warps' loop is long straight code (about 20 KiB); what runs beside it on an SM has to
// be little, or the warps wait for instructions.  (The chunks' images were made here first, by
// four to six more warps, in place or shared in a cluster: 476 to 640 us for 8192 tokens of 32 heads
// against 60 + 350 us with a kernel of their own.)
template <int DK, int NCW, int KS, bool ADJ, bool WANT_Q, int OUTW>
struct Pipe {
    static constexpr int W = NCW * 16;
    using L = Stage<DK, W, ADJ, WANT_Q>;
    static constexpr int ST = NCW == 8 ? 4 : 5;
    static constexpr int CHAIN = NCW * KS, OW = OUTW > 0 ? NCW : 0, WARPS = CHAIN + 1 + OW;
    static constexpr int OP = 48;                         // row pitch of a warp's 32 x 16 output tile
    static constexpr int OUT = ST * L::BYTES;
    static constexpr int SWAP = OUT + CHAIN * kChunk * OP;
    static constexpr int HAND = SWAP + (KS == 2 ? NCW * 2 * 2 * 16 * 32 * 4 : 0);
    static constexpr int BARS = HAND + OW * ST * OUTW;
    static constexpr int BYTES = BARS + (2 * ST + NCW + OW * ST) * 8 + 16;
    static_assert(BYTES <= 227 * 1024, "shared memory of a CTA");

    unsigned char *smem;
    // swapped: KS = 2's exchange, one barrier per group at which both warps arrive and wait.  Its phase
    // c + 1 needs both warps' arrivals for c + 1, and each follows that warp's wait for c: no phase ends
    // before the one before it has been waited for.  (A barrier at which only the other warp arrives could
    // be a phase further on when this one comes to wait, whose parity then names a phase to come.)
    uint64_t *full, *empty, *swapped, *handed;
    volatile uint32_t *abort;
    uint32_t *err;
    uint32_t epoch;

    __device__ __forceinline__ Pipe(unsigned char *s, uint32_t *e, uint32_t ep) : smem(s), err(e), epoch(ep) {
        full = reinterpret_cast<uint64_t *>(smem + BARS);
        empty = full + ST, swapped = empty + ST, handed = swapped + NCW;
        abort = reinterpret_cast<volatile uint32_t *>(handed + OW * ST);
        if (threadIdx.x == 0) {
            for (int i = 0; i < ST; ++i) {
                mbar_init(full + i, 1);
                mbar_init(empty + i, CHAIN + OW);
            }
            for (int i = 0; i < NCW; ++i) mbar_init(swapped + i, KS);
            for (int i = 0; i < OW * ST; ++i) mbar_init(handed + i, KS);
            mbar_fence_init();
            *abort = 0u;
        }
        __syncthreads();
    }
    __device__ __forceinline__ bool wait(uint64_t *bar, uint32_t parity) const {
        return warp_wait(bar, parity, err, epoch, abort);
    }
    __device__ __forceinline__ unsigned char *stage(int i) const { return smem + i * L::BYTES; }
    // stage s of a group's hand-over to its output warp
    __device__ __forceinline__ unsigned char *hand(int group, int s) const {
        return smem + HAND + (group * ST + s) * OUTW;
    }

    // The loader warp.  REVERSE: the sequence's chunks from the last to the first.  Its lane 0 leaves only
    // when all its copies have landed (a bounded wait), also where a wait gave up: no copy may arrive in the
    // shared memory of a CTA that is gone.
    template <bool REVERSE>
    __device__ __forceinline__ void load(const ChainInput &a, const CUtensorMap *vmap, const Span &span, int n,
                                         int h, int hk, int column, int chunks) const {
        const int64_t slot0 = first_chunk(span, n);
        int i = 0;
        for (int s = 0, use = 0; i < chunks; ++i) {
            if (use > 0 && !wait(empty + s, (use - 1) & 1)) break;
            if ((threadIdx.x & 31) == 0) {
                const int c = REVERSE ? chunks - 1 - i : i;
                const uint32_t at = smem_u32(stage(s));
                mbar_arrive_expect_tx(full + s, L::KEYS + L::HEADS + L::VBYTES);
                bulk_load(at, a.keys + ((slot0 + c) * a.Hk + hk) * L::KI::BYTES, L::KEYS, full + s);
                bulk_load(at + L::HEAD, a.heads + ((slot0 + c) * a.H + h) * L::HI::BYTES, L::HEADS, full + s);
#pragma unroll
                for (int p = 0; p < W; p += 64)
                    tma_rows(at + L::V + p * kChunk * 2, vmap, column + p, h, (int)span.row + c * kChunk, full + s);
            }
            __syncwarp();
            if (++s == ST) s = 0, ++use;
        }
        if ((threadIdx.x & 31) == 0)
            for (int c = i > ST ? i - ST : 0; c < i; ++c)
                if (!mbar_wait(full + c % ST, (c / ST) & 1, err)) break;
    }
    // This warp is through with stage s.
    __device__ __forceinline__ void release(int s) const {
        __syncwarp();
        if ((threadIdx.x & 31) == 0) mbar_arrive(empty + s);
    }
};

// Launch of a chain kernel over `rows` rows, CTAs of `cols` columns.  v: the values, or the output
// gradients in their place.
template <typename Args>
inline cudaError_t launch_chain_kernel(void (*kernel)(const CUtensorMap, const Args), const Args &a, const void *v,
                                       int64_t rows, int cols, int64_t units, int threads, int smem,
                                       cudaStream_t st) {
    CUtensorMap map = {};
    const bool narrow = cols < 64;
    if (rows > 0 &&   // with no rows nothing is loaded
        !make_rows_heads_tmap(&map, v, rows, a.in.H, a.in.dv, narrow ? cols : 64, kChunk,
                              narrow ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B))
        return cudaErrorInvalidValue;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    kernel<<<(unsigned)(units * (a.in.dv / cols)), threads, smem, st>>>(map, a);
    e = cudaGetLastError();
    Profiler::mark(st);
    return e;
}

// Columns per CTA (16 NCW) and warps per 16 columns (KS) of a chain, as NCW * 10 + KS.  A round of CTAs
// over the 148 SMs took, for 4096 tokens at dk = dv = 128 (prefill): 32 columns with two warps per 16,
// 179 us (37 units a round at dv = 128); 64 columns with one, 216 us (74 units); 128 with one, 377 us
// (148 units).  So 32 and 48 heads take 179 against 215 and 377 us, and 349 against 216 and 377; 96
// heads 520 against 420 and 378; 160 heads 862 against 626 and 740.  The choice is the least of rounds
// times that; packed sequences, which are ragged, fill the rounds' ends, so there their number is not
// rounded up.  The same numbers serve the adjoint, whose rounds take 243, 353 and 640 us, and d = 64 (154
// us a round of 32 or 64 columns): their least is the same variant at 16, 32, 37, 48, 74, 96, 148 and 160
// heads.
inline int chain_variant(int64_t units, int dv, bool packed) {
    struct { int columns, variant; double us; } const all[3] = {{32, 22, 179.}, {64, 41, 216.}, {128, 81, 377.}};
    int best = 0;
    double least = 0.;
    for (const auto &v : all) {
        if (v.columns > dv) break;
        const int64_t ctas = units * (dv / v.columns);
        double rounds = packed ? (double)ctas / 148. : (double)((ctas + 147) / 148);
        if (rounds < 1.) rounds = 1.;
        if (best == 0 || rounds * v.us < least) best = v.variant, least = rounds * v.us;
    }
    return best;
}

}  // namespace gdr
}  // namespace kda
