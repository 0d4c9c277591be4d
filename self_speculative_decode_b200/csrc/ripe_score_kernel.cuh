// Attention over a RIPE cache whose deepest-plane region is held in 8 bits (Q8), or with capped or
// distance-biased scores (MOD; 2: with a cap from kCapSeries on); included by the translation units that instantiate it.
//
// What is computed: for every query row of block position p = T + j, over the keys t <= p with the
// plane rule of ripe_verify_attn,
//   x_t = scale <q, K_t>;  cap c > 0: x_t <- c tanh(x_t / c);  bias: x_t <- x_t - slope_h (p - t)
//   out = sum_t softmax(x)_t V_t
// with K_t, V_t of blocks in the 8-bit region read as u * s, s the block's scale.
//
// The skeleton is that of ripe_verify.cu: one persistent launch, one producer thread streaming tiles
// into a ring of stages, consumer warps on the transposed products S^T = K Q^T and O^T += V^T P^T,
// lazily moved softmax reference in base 2, partials merged by the last arrival.  What differs:
//   * 8-bit tiles are two blocks of 64 keys, one bulk copy each tile (a stage then holds as many bytes
//     as a bf16 tile).  The bytes are in fragment order (ripe_score.cuh): a 16-byte shared-memory load
//     gives a lane two A fragments, and one byte permute and one subtraction turn two bytes into two
//     f16 values (0x6400 | u + 128 is 1152 + u).  Integers up to 127 are exact in f16 and in bf16; f16
//     takes two instructions a pair, bf16 four (its 7 mantissa bits cannot hold u + 128).
//   * Q of those tiles is bf16 scaled by a power of two per row into f16's range, exact for elements
//     down to 2^-18 of the row's largest; P is rounded to f16 (2^-11 relative).  Q lies in shared memory in
//     fragment order, once in each form.
//   * From 17 rows on (WIDE) the four warps of a tile group split the keys for S and head_dim for O: a warp
//     turns its 16 keys of K and its quarter of V into f16 for all 32 rows, once, and P goes from one product
//     to the other through shared memory.  O then takes 32 registers a thread instead of 128, so that three
//     tile groups fit an SM and hide one another's latencies.  More than 32 rows of a kv head are two groups
//     that stream the keys one after the other, each a head of its own in the tile lists.
//   * The K scale enters with the softmax scale; the V scale enters the exponent: p' = 2^(x + log2 s -
//     m), O sums p' u, and the normaliser sums p' / s.  So a block costs no multiply of its own per
//     element, and the reference m follows the size of p' u, which is what O accumulates.  s spans 2^-80 to 2^80:
//     where p' leaves fp32 the key's weight still counts.  Blocks with s below kTinyScale take their share of the
//     normaliser from 2^(x - m), and where it is rescaled by less than fp32 holds that goes in two steps.
//   * tanh y = 1 - 2 / (1 + e^2y): one exponential and one reciprocal, absolute error 2^-22 of the cap
//     (the hardware's tanh is 2^-11 relative: 0.02 at a cap of 50).  That error moves the weights as much however
//     small the scores are, so that caps from kCapSeries on take the odd series where |y| is small (capped): an
//     error of 2^-19 of the score itself.  They are instances of their own: with both forms in one, capped launches
//     took up to 4 % longer.
//   * A masked value never reaches a sum: stale ring rows or later draft rows may hold NaN or infinity.
//
// Measured (one B200, 8 sequences x 32768 keys, 8 kv heads x 128; 6456 GB/s is the measured copy): over the 8-bit
// region 87 us at 4 rows a kv head (0.96 of it), 102 us at 16 (0.82), 160 to 166 us at 32 (0.50 to 0.52: paced by instructions,
// 3.25 warps a scheduler; 178 us with 16 rows and 32 keys a warp, 180 us with 32 rows, 16 keys and all of head_dim a warp,
// 194 us with two groups instead of three), 297 us at 64; capped, over bf16, 193 to 200 us at 32 rows (0.83 to 0.86), 209 us
// with a cap from kCapSeries on.
#pragma once

#include <cuda_fp16.h>

#include <mutex>
#include <type_traits>

#include "ripe_score.cuh"

namespace ripe {

// softmax reference: moved when a score exceeds it by more than kHi, and then to kLo below the maximum, so
// that the probabilities lie in (0, 2^15], within f16's range, and are exact down to 2^-(14 + 10 + kLo)
constexpr float kScoreHi = 15.f, kScoreLo = 7.f;
// log2 of the smallest V scale whose p' / s is summed: beside values of the largest scale the reference is at most
// 2^73 times the largest weight, and p' of that weight at least 2^-93, 33 bits above what fp32 flushes to zero
constexpr float kTinyScale = -20.f;

// Query-side shapes as VCfg (ripe_verify.cu): NQT 8-query tiles per warp, WR row groups, WK key groups
// per 64-key block, TG tile groups consuming alternate tiles.
template <int D, int NQT, int WR, int WK, int TG, bool Q8>
struct SCfg {
    static constexpr bool WIDE = NQT >= 4;  // keys and head_dim split over the warps of a group
    static_assert(!WIDE || (WR == 1 && WK == 4), "a wide group is four warps");
    static constexpr int NQ = 8 * NQT;
    static constexpr int ROWS = NQ * WR;
    static constexpr int GW = WR * WK;
    static constexpr int NCW = GW * TG;
    static constexpr int NP = WK * TG;  // warps that share a query row
    // with two query tiles per warp the producer warp heads a warpgroup that gives registers up
    static constexpr bool SPLIT = NQT == 2;
    static constexpr int THREADS = SPLIT ? (NCW + 4) * 32 : (NCW + 1) * 32;
    static constexpr int LAUNCH_REGS = (65536 / THREADS) / 8 * 8 > 255 ? 248 : (65536 / THREADS) / 8 * 8;
    static constexpr int REG_PRODUCER = 72;
    static constexpr int REG_FREE = ((LAUNCH_REGS * (NCW + 4) - 4 * REG_PRODUCER) / NCW) / 8 * 8;
    static constexpr int REG_CONSUMER = REG_FREE > 248 ? 248 : REG_FREE;
    static_assert(WIDE || NCW % 4 == 0, "consumer warps form whole warpgroups");
    static_assert(!SPLIT || NCW * REG_CONSUMER + 4 * REG_PRODUCER <= (NCW + 4) * LAUNCH_REGS, "register split");
    static constexpr int SB = 4 / WK;  // 16-key sub-blocks per warp and block
    static constexpr int MT = WIDE ? (D == 64 ? 1 : 2) : D / 16;  // 16-column tiles of O per warp
    static constexpr int NBOX = D / kBoxCols;
    static constexpr int BOX_ROWS = WIDE && Q8 ? kWideRingRows : kTileRows;  // rows of a ring tile's boxes
    static constexpr int RING_BYTES = 2 * NBOX * BOX_ROWS * 64;
    static constexpr int DEEP_BYTES = Q8 ? (WIDE ? 1 : 2) * q8_record_bytes(D) : RING_BYTES;
    // a multiple of the 64-byte swizzle's 512-byte period
    static constexpr int STAGE_BYTES = ((DEEP_BYTES > RING_BYTES ? DEEP_BYTES : RING_BYTES) + 511) / 512 * 512;
    // Q in fragment order, [form][row tile][D / 32][lane] of 16 bytes: bf16, and f16 for 8-bit tiles
    static constexpr int QF_BYTES = ROWS * D * 2;
    static constexpr int Q_BYTES = (Q8 ? 2 : 1) * QF_BYTES;
    // WIDE: P, [group][2][16-key sub-block][row tile] of two 8 x 8 matrices
    static constexpr int P_BYTES = WIDE ? TG * 2 * 4 * (NQT / 2) * 512 : 0;
    // merge buffer: rows of o per warp, or per group of a wide one; (m, l_out, l_lse) per warp
    static constexpr int DP = D + 4;
    static constexpr int SLOTS = WIDE ? TG : NCW;
    static constexpr int NPF = WIDE ? TG : NP;  // partials of a row of o
    static constexpr int MERGE_FLOATS = SLOTS * NQ * DP;
    // WIDE: column maxima and l_fix of each warp, references of each group
    static constexpr int GM_FLOATS = WIDE ? (2 * NCW + TG) * NQ : 0;
    static constexpr int MLF = NCW * NQ * 4 + ROWS * (NPF + 4) + 3 * ROWS + 4 * ROWS + GM_FLOATS + (WIDE ? 4 * TG : 0);
    static_assert(MLF % 4 == 0 && (ROWS * NPF) % 4 == 0, "alignment");
    static constexpr int MISC = 1024 + 1024;
    static constexpr int AVAIL =
        kSmemLimit - MISC - Q_BYTES - P_BYTES - 4 * (MERGE_FLOATS + MLF) - 4 * (3 * kMaxBatch + 2);
    static constexpr int NS_RAW = AVAIL / STAGE_BYTES > 8 ? 8 : AVAIL / STAGE_BYTES;
    static constexpr int NS = NS_RAW - NS_RAW % TG;  // a stage always serves the same tile group
    static_assert(NS >= 2, "not enough shared memory for the pipeline");
    static constexpr int SMEM_FIXED = MISC + Q_BYTES + P_BYTES + NS * STAGE_BYTES + 4 * (MERGE_FLOATS + MLF);
    static_assert(SMEM_FIXED + 4 * (3 * kMaxBatch + 2) <= kSmemLimit, "shared memory");
    static constexpr int MAX_PARTS =
        (NS * STAGE_BYTES) / (2 * ROWS * 4) < 256 ? (NS * STAGE_BYTES) / (2 * ROWS * 4) : 256;
    static_assert(MAX_PARTS >= 148, "stage buffers too small for the end-of-CTA merge");
    static constexpr int smem_bytes(int N) { return SMEM_FIXED + (3 * N + 2) * 4; }
};

// cap tanh(z / cap) for a score z, both in log2 units; rcap = 1 / cap.  Up to |y| = 0.35 the series to y^9 (the next
// term is 2^-21 of the sum there), beyond it 1 - 2 / (1 + e^2y), whose error of 2^-21.4 (one step of the exponential's and
// of the reciprocal's 2^-22 each) is 2^-19.8 of tanh 0.35.  A NaN fails the comparison and goes through the exponential.
__device__ __forceinline__ float capped(float z, float cap, float rcap) {
    const float y = z * rcap, s = y * y;
    const float series =
        fmaf(s, fmaf(s, fmaf(s, fmaf(s, 62.f / 2835.f, -17.f / 315.f), 2.f / 15.f), -1.f / 3.f), 1.f);
    const float far = fmaf(-2.f, __fdividef(1.f, 1.f + exp2f(y * 2.8853900817779268f)), 1.f);
    return fabsf(y) < 0.35f ? z * series : cap * far;
}

__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(bar)
                 : "memory");
}

__device__ __forceinline__ void l2_prefetch(const void *p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

__device__ __forceinline__ void sts32(uint32_t addr, uint32_t v) {
    asm volatile("st.shared.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

__device__ __forceinline__ uint2 lds64(uint32_t addr) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr) : "memory");
    return v;
}

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

// two fp32 operations in one instruction
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
        "fma.rn.f32x2 x, x, y, z;\n\tmov.b64 {%0, %1}, x;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tadd.rn.f32x2 x, x, y;\n\t"
        "mov.b64 {%0, %1}, x;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}

// D = A * B (+ D): f16 or bf16 operands, fp32 sums; the first product of a chain needs no zeroed registers
template <bool HALF, bool FIRST>
__device__ __forceinline__ void mma_step(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (FIRST && HALF)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                     "{%10, %10, %10, %10};"
                     : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
    else if constexpr (FIRST)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                     "{%10, %10, %10, %10};"
                     : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
    else if constexpr (HALF)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                     "{%0, %1, %2, %3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        mma_16816(d, a, b0, b1);
}

// four bytes u + 128 -> two pairs of f16 u: (bytes 0, 1) and (bytes 2, 3)
__device__ __forceinline__ void q8_to_f16(uint32_t w, uint32_t &lo, uint32_t &hi) {
    const __half2 off = __floats2half2_rn(1152.f, 1152.f);
    uint32_t a = __byte_perm(w, 0x64646464u, 0x4140), b = __byte_perm(w, 0x64646464u, 0x4342);
    const __half2 x = __hsub2(*reinterpret_cast<__half2 *>(&a), off);
    const __half2 y = __hsub2(*reinterpret_cast<__half2 *>(&b), off);
    lo = *reinterpret_cast<const uint32_t *>(&x);
    hi = *reinterpret_cast<const uint32_t *>(&y);
}

// whether either bf16 of a pair is an infinity or a NaN
__device__ __forceinline__ bool bf16x2_nonfinite(uint32_t r) {
    return (r & 0x7F80u) == 0x7F80u || (r & 0x7F800000u) == 0x7F800000u;
}

// The chunk of the heads' tile lists that this CTA streams (score_begin, score_first): from tile lt of pair p_first on,
// ntiles tiles, the last of them in pair p_last.  cum[n] is where sequence n's heads begin on the line of costs,
// real[n] the number of tiles before them.
struct ScoreChunk {
    int chunk, pieces;  // costs; pieces > 0: every head is cut into that many pieces of its own
    int p_first, lt, p_last, ntiles;
};

// Tiles that begin before offset g of the line (with `upto`: at or before it); the pair of the tile that comes next
// (upto: of the last of them), and its index.
__host__ __device__ __forceinline__ int3 score_tiles_before(const ScoreArgs &a, const int *cum, const int *real,
                                                            const int *Ts, int kvH, int g, bool upto) {
    const int n = seq_of(cum, a.N, g);
    const ScoreGeom sg = score_geom(Ts[n], a.plan);
    const int kh = (g - cum[n]) / sg.cost, off = g - cum[n] - kh * sg.cost;
    int lt = score_first(sg, off + (upto ? 1 : 0), a.plan), pair = n * kvH + kh;
    const int before = real[n] + kh * sg.total + lt;
    if (upto) {
        if (--lt < 0) --pair;  // the last tile is the previous head's
    } else if (lt == sg.total) {
        lt = 0;  // the rest of the head's cost holds no tile; kh + 1 == kvH is the next sequence's first head
        ++pair;
    }
    return make_int3(before, pair, lt);
}

// The CTAs that hold tiles of a pair: the first of them, and how many.
__host__ __device__ __forceinline__ int2 score_parts(const ScoreArgs &a, const ScoreChunk &c, const int *cum,
                                                     const int *Ts, int kvH, int p) {
    const int n = p / kvH;
    const ScoreGeom sg = score_geom(Ts[n], a.plan);
    const int last = score_begin(sg, sg.total - 1, a.plan);
    if (c.pieces) return make_int2(p * c.pieces, last / c.chunk + 1);
    const int start = cum[n] + (p - n * kvH) * sg.cost, first = start / c.chunk;
    return make_int2(first, (start + last) / c.chunk - first + 1);
}

// Chunks of `chunk` costs, or, where all heads cost the same (cost0) and there are no more of them than CTAs, `pieces`
// equal pieces of every head.  A head that a CTA shares costs it head_cost once more, so that pieces, which share
// nothing across heads, are taken when they are no longer than a chunk (their own head_cost left out) or short
// anyway; with more heads, chunks end on heads when that lengthens them by at most head_cost.
__host__ __device__ __forceinline__ int most_of(int x, int y) { return x > y ? x : y; }
__host__ __device__ __forceinline__ int2 score_cut(const ScoreArgs &a, int grid, int total, int cost0, bool same, int kvH) {
    const int head = a.plan.head_cost, heads = a.N * kvH;
    int chunk = most_of(cdiv(total, grid), a.min_chunk);
    if (same && heads <= grid) {
        const int most = most_of((cost0 - head) / a.min_chunk, 1), P = grid / heads < most ? grid / heads : most;
        const int piece = most_of(cdiv(cost0 - head, P), a.plan.ring_cost);  // no shorter than a tile: each holds one
        if (piece <= most_of(chunk, a.min_chunk + head)) return make_int2(piece, P);
    } else if (same && chunk >= cost0) {
        const int whole = cdiv(chunk, cost0) * cost0;
        if (whole <= chunk + head) chunk = whole;
    }
    return make_int2(chunk, 0);
}

// The tiles of CTA `cta`: of a piece of a head with geometry sg (in that head's list), or of a chunk of the line.
__host__ __device__ __forceinline__ void score_piece(const ScoreArgs &a, const ScoreGeom &sg, int cta, ScoreChunk &c) {
    const int at = (cta - c.p_first * c.pieces) * c.chunk;
    c.lt = score_first(sg, at, a.plan);
    c.ntiles = score_first(sg, at + c.chunk, a.plan) - c.lt;
}
__host__ __device__ __forceinline__ void score_line(const ScoreArgs &a, const int *cum, const int *real, const int *Ts,
                                                    int kvH, int cta, ScoreChunk &c) {
    const int begin = cta * c.chunk, end = cum[a.N] < begin + c.chunk ? cum[a.N] : begin + c.chunk;
    if (begin >= end) return;
    int before = 0;
#pragma unroll 1  // one copy of the code: a small launch is paced by fetching instructions
    for (int k = 0; k < 2; ++k) {
        const int3 at = score_tiles_before(a, cum, real, Ts, kvH, k ? end - 1 : begin, k);
        if (k == 0) {
            before = at.x;
            c.p_first = at.y;
            c.lt = at.z;
        } else {
            c.ntiles = at.x - before;
            c.p_last = at.y;
        }
    }
}

__device__ __forceinline__ ScoreChunk score_chunks(const ScoreArgs &a, int *cum, int *real, int *Ts, int *sflag, int tid,
                                                   int warp, int lane) {
    const int N = a.N, kvH = a.kvH * a.groups;
    ScoreChunk c;
    c.ntiles = 0;
    if (N == 1) {  // one sequence: every thread reads its length and cuts the list itself
        const int T = a.T[0];
        const ScoreGeom sg = score_geom(T, a.plan);
        if (tid == 0) {
            Ts[0] = T;
            cum[0] = 0;
            cum[1] = sg.cost * kvH;
            real[0] = 0;
        }
        const int2 cut = score_cut(a, gridDim.x, sg.cost * kvH, sg.cost, true, kvH);
        c.chunk = cut.x;
        c.pieces = cut.y;
        __syncthreads();
        pdl_trigger();  // the next kernel may be scheduled; it waits for this one to finish
        if (c.pieces) {
            c.p_first = c.p_last = blockIdx.x / c.pieces;
            if (c.p_first < kvH) score_piece(a, sg, blockIdx.x, c);
            return c;
        }
    } else {
        for (int n = tid; n < N; n += blockDim.x) {
            const int T = a.T[n];
            const ScoreGeom sg = score_geom(T, a.plan);
            Ts[n] = T;
            cum[n + 1] = sg.cost * kvH;
            real[n] = sg.total * kvH;
        }
        if (tid == 0) cum[0] = 0;
        __syncthreads();
        pdl_trigger();
        if (warp == 0) {
            int carry = 0, rcarry = 0;
            bool same = true;
            const int first = cum[1];
            for (int b = 0; b < N; b += 32) {
                const int own = (b + lane < N) ? cum[b + lane + 1] : 0;
                const int rown = (b + lane < N) ? real[b + lane] : 0;
                same = same && __all_sync(0xffffffffu, b + lane >= N || own == first);
                int v = own, r = rown;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int u = __shfl_up_sync(0xffffffffu, v, o), w = __shfl_up_sync(0xffffffffu, r, o);
                    if (lane >= o) {
                        v += u;
                        r += w;
                    }
                }
                if (b + lane < N) {
                    cum[b + lane + 1] = v + carry;
                    real[b + lane] = r + rcarry - rown;
                }
                carry += __shfl_sync(0xffffffffu, v, 31);
                rcarry += __shfl_sync(0xffffffffu, r, 31);
            }
            if (lane == 0) {
                const int2 cut = score_cut(a, gridDim.x, carry, first / kvH, same, kvH);
                sflag[6] = cut.x;
                sflag[7] = cut.y;
            }
        }
        __syncthreads();
        c.chunk = sflag[6];
        c.pieces = sflag[7];
        if (c.pieces) {
            c.p_first = c.p_last = blockIdx.x / c.pieces;
            if (c.p_first < N * kvH) score_piece(a, score_geom(Ts[c.p_first / kvH], a.plan), blockIdx.x, c);
            return c;
        }
    }
    score_line(a, cum, real, Ts, kvH, blockIdx.x, c);
    return c;
}

template <int D, int NQT, int WR, int WK, int TG, bool Q8, int MOD>
__global__ void __launch_bounds__(SCfg<D, NQT, WR, WK, TG, Q8>::THREADS, 1)
ripe_score_kernel(const __grid_constant__ CUtensorMap tmKd, const __grid_constant__ CUtensorMap tmVd,
                  const __grid_constant__ CUtensorMap tmKw, const __grid_constant__ CUtensorMap tmVw,
                  const __grid_constant__ ScoreArgs a) {
    using C = SCfg<D, NQT, WR, WK, TG, Q8>;
    constexpr int NS = C::NS;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *stages = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                  ~static_cast<uintptr_t>(1023));
    uint8_t *qf = stages + NS * C::STAGE_BYTES;                           // Q fragments, then P (WIDE)
    float *mo = reinterpret_cast<float *>(qf + C::Q_BYTES + C::P_BYTES);  // [SLOTS][NQ][DP]
    float *mml = mo + C::MERGE_FLOATS;                                    // [NCW][NQ][4] m, l_out, l_lse
    float *wq = mml + C::NCW * C::NQ * 4;                                 // [ROWS][NPF] weights
    float *fin = wq + C::ROWS * C::NPF;                                   // [ROWS][4] final m, l_out, l_lse
    float *qscale = fin + C::ROWS * 4;                                    // [ROWS] sx over the row's power of two
    float *qslope = qscale + C::ROWS;                                     // [ROWS] distance bias of the row's head
    int *qpos = reinterpret_cast<int *>(qslope + C::ROWS);                // [ROWS] block position, -1: no such row
    int4 *qsees = reinterpret_cast<int4 *>(qpos + C::ROWS);               // [ROWS] keys a row sees (stage_q)
    float *gmax = reinterpret_cast<float *>(qsees + C::ROWS);             // WIDE [NCW][NQ] column maxima
    float *gfix = gmax + C::NCW * C::NQ;                                  // WIDE [NCW][NQ] l_fix
    float *gref = gfix + C::NCW * C::NQ;                                  // WIDE [TG][NQ] m_ref
    // WIDE [TG][4]: the last even and the last odd block that moves a reference; the group has given up; -
    int *gflag = reinterpret_cast<int *>(gmax + C::GM_FLOATS);
    uint64_t *bars = reinterpret_cast<uint64_t *>(mml + C::MLF);          // full[NS], empty[NS]
    TileDesc *sdesc = reinterpret_cast<TileDesc *>(bars + 2 * NS);        // [NS]
    int *sflag = reinterpret_cast<int *>(sdesc + NS);                     // [16]
    int *cum = sflag + 16;                                                // [N + 1]
    int *Ts = cum + a.N + 1;                                              // [N]
    int *real = Ts + a.N;                                                 // [N]

    const int tid = threadIdx.x;
    const int warp = tid >> 5;
    const int lane = tid & 31;
    const ScorePlan &pa = a.plan;
    const int N = a.N, kvH = a.kvH * a.groups;  // each row group of a kv head counts as a head

    if (warp == C::NCW && lane == 0) {
        tma_prefetch_desc(&tmKw);
        tma_prefetch_desc(&tmVw);
        if (!Q8 && a.has_deep) {
            tma_prefetch_desc(&tmKd);
            tma_prefetch_desc(&tmVd);
        }
    }
    if (tid == 0) {
        sflag[1] = 0;  // abort flag
        sflag[3] = 0;  // pairs this CTA merges at the end (its first and last at most): sflag[4..5]
        for (int s = 0; s < NS; ++s) {
            mbar_init(smem_addr(&bars[s]), 1);
            mbar_init(smem_addr(&bars[NS + s]), C::GW);
        }
        mbar_fence_init();
    }
    if (C::WIDE && tid < 4 * TG) gflag[tid] = -1;
    if (!a.early) pdl_wait();
    const ScoreChunk cp = score_chunks(a, cum, real, Ts, sflag, tid, warp, lane);
    const int ntiles = cp.ntiles, P_first = cp.p_first, P_last = cp.p_last;
    if (ntiles <= 0) {
        if (a.early) pdl_wait();  // the launch completes only after its predecessor
        return;
    }
    const uint32_t full0 = smem_addr(&bars[0]);
    const uint32_t empty0 = smem_addr(&bars[NS]);
    const uint32_t stage0 = smem_addr(stages);

    if (warp >= C::NCW) {
        // ================================================================ producer (one thread)
        if constexpr (C::SPLIT) setmaxnreg_dec<C::REG_PRODUCER>();
        if (warp != C::NCW || lane != 0) return;
        int n = P_first / kvH, kh = P_first - (P_first / kvH) * kvH;
        ScoreGeom sg = score_geom(Ts[n], pa);
        int lt = cp.lt;
        bool waited = !a.early;
        int i = 0;
        for (; i < ntiles; ++i) {
            const int s = i % NS;
            if (i >= NS && !mbar_wait_bounded(empty0 + 8 * s, ((i / NS) - 1) & 1)) break;
            const Tile t = score_tile(sg, lt, pa);
            const bool deep = t.kind == kDeep;
            if (!waited && !deep) {  // ring rows: the previous launch may be writing the block
                pdl_wait();
                waited = true;
            }
            TileDesc &dsc = sdesc[s];
            dsc.pair = n * kvH + kh; dsc.n = n; dsc.kh = kh; dsc.T = sg.T;
            dsc.kind = t.kind; dsc.t0 = t.t0; dsc.cnt = t.cnt; dsc.plane = t.plane;
            const uint32_t fb = full0 + 8 * s;
            const uint32_t kdst = stage0 + s * C::STAGE_BYTES;
            if constexpr (kDebug) {  // the tile lies inside its region
                const bool bad = t.cnt < 1 || (deep ? t.t0 < 0 || t.t0 + t.cnt > a.dbg_deep_rows
                                                    : t.y < 0 || t.y + t.cnt > pa.S ||
                                                          (t.y - t.t0 % pa.S + pa.S) % pa.S != 0);
                if (bad) atomicOr(a.err, RIPE_DEVERR_BOUNDS);
            }
            if (Q8 && deep) {
                const uint32_t bytes = static_cast<uint32_t>(t.cnt >> 6) * q8_record_bytes(D);
                const size_t r = (static_cast<size_t>(a.layer) * N + n) * a.kvH + kh / a.groups;
                mbar_expect_tx(fb, bytes);
                bulk_load(kdst, a.rec + (r * a.rec_blocks + (t.t0 >> 6)) * q8_record_bytes(D), bytes, fb);
            } else {
                const int rows = deep ? pa.deep_box : pa.ring_box;
                const CUtensorMap *mk = deep ? &tmKd : &tmKw;
                const CUtensorMap *mv = deep ? &tmVd : &tmVw;
                const int z = (deep ? a.layer * N + n : (a.layer * N + n) * pa.R + t.plane) * a.kvH + kh / a.groups;
                const uint32_t vdst = kdst + C::RING_BYTES / 2;
                mbar_expect_tx(fb, 2 * C::NBOX * rows * 64);
#pragma unroll
                for (int b = 0; b < C::NBOX; ++b) {
                    tma_load_3d(kdst + b * C::BOX_ROWS * 64, mk, fb, b * kBoxCols, t.y, z);
                    tma_load_3d(vdst + b * C::BOX_ROWS * 64, mv, fb, b * kBoxCols, t.y, z);
                }
            }
            if (++lt == sg.total) {
                lt = 0;
                if (++kh == kvH) {
                    kh = 0;
                    if (++n < N) sg = score_geom(Ts[n], pa);
                }
                if (i + 1 < ntiles) {  // bring the next pair's queries into L2
                    const int h = kh / a.groups, row0 = kh % a.groups * a.grows, rows = min(a.grows, a.Mq - row0);
                    for (int x = 0; x < rows; ++x) {
                        const int j = (row0 + x) / a.g, hg = row0 + x - j * a.g;
                        const char *qp = reinterpret_cast<const char *>(
                            a.q + ((static_cast<size_t>(n) * a.qB + j) * a.Hq + h * a.g + hg) * D);
                        for (int u = 0; u < 2 * D; u += 128) l2_prefetch(qp + u);
                    }
                }
            }
        }
        if (i < ntiles) {
            atomicOr(a.err, RIPE_DEVERR_WAIT_TIMEOUT);
            // drain: the last issue of every stage must land before the CTA exits
            for (int k = (i > NS ? i - NS : 0); k < i; ++k) mbar_wait_bounded(full0 + 8 * (k % NS), (k / NS) & 1);
        }
        return;  // the producer warp takes part in no consumer barrier (id 1)
    }
    if constexpr (C::SPLIT) setmaxnreg_inc<C::REG_CONSUMER>();

    // ==================================================================== consumers
    const int tg = warp / C::GW;         // tiles i with i % TG == tg
    const int rg = (warp % C::GW) / WK;  // queries NQ*rg .. NQ*rg + NQ-1
    const int kg = warp % WK;            // sub-blocks kg*SB .. kg*SB + SB-1
    const int g4 = lane >> 2, c4 = lane & 3;
    const int nct = C::NCW * 32;
    // a thread holds the query columns NQ*rg + 8*nq + 2*c4 + e
    const int col0 = C::NQ * rg + 2 * c4;

    // ldmatrix lane geometry of the bf16 tiles (64-byte swizzle: 16-byte chunk ^= (row >> 1) & 3)
    const int mi = lane >> 3, r8 = lane & 7;
    const uint32_t swz = static_cast<uint32_t>(r8 >> 1);
    const uint32_t krow_off = static_cast<uint32_t>((mi & 1) * 8 + r8);
    const uint32_t kcol_sel = static_cast<uint32_t>(mi >> 1);
    const uint32_t vrow_off = static_cast<uint32_t>((mi >> 1) * 8 + r8);
    const uint32_t vcol_sel = static_cast<uint32_t>(mi & 1);
    // this lane's Q fragments of row tile NQT*rg
    const uint32_t qf0 = smem_addr(qf) + NQT * rg * (D / 32) * 512 + lane * 16;

    float o[C::MT][NQT][4];
    // l_lse sums the probabilities in fp32; l_fix sums what rounding adds to them in bf16 tiles, where the P V
    // product sees 2^-8: the output is normalised by both together, which is what O sums.  A column's reference means nothing until some lane's l_lse is not zero
    // (WIDE: m_ref and l_fix are in shared memory, a column's by the lane with g4 == 0, to fit 128 registers)
    float l_lse[NQT][2], m_ref[C::WIDE ? 1 : NQT][2], l_fix[C::WIDE ? 1 : NQT][2];
    uint32_t seen = 0;  // WIDE: bit 2 nq + e is set once the column has a reference
    uint32_t qb[C::WIDE ? 1 : D / 16][C::WIDE ? 1 : NQT][2];  // Q as B fragments

    int st_half = -1;  // qb holds the f16 (1) or bf16 (0) form
    bool aborted = false;

    auto reset_state = [&]() {
        seen = 0;
#pragma unroll
        for (int mt = 0; mt < C::MT; ++mt)
#pragma unroll
            for (int nq = 0; nq < NQT; ++nq) o[mt][nq][0] = o[mt][nq][1] = o[mt][nq][2] = o[mt][nq][3] = 0.f;
#pragma unroll
        for (int nq = 0; nq < NQT; ++nq) {
            l_lse[nq][0] = l_lse[nq][1] = 0.f;
            if constexpr (!C::WIDE) {
                m_ref[nq][0] = m_ref[nq][1] = 0.f;
                l_fix[nq][0] = l_fix[nq][1] = 0.f;
            }
        }
        if constexpr (C::WIDE) {  // (the barrier of stage_q follows)
            gfix[warp * C::NQ + lane] = 0.f;
            if (kg == 0) gref[tg * C::NQ + lane] = 0.f;
        }
    };
    // references of columns 8 nq + 2 c4 and the next
    auto refs = [&](int nq) -> float2 {
        if constexpr (C::WIDE) return *reinterpret_cast<const float2 *>(&gref[tg * C::NQ + 8 * nq + 2 * c4]);
        else return make_float2(m_ref[nq][0], m_ref[nq][1]);
    };

    // kv head of pair p, its first query row, and how many rows the pair has
    auto head_of = [&](int p) { return (p % kvH) / a.groups; };
    auto group_row = [&](int p) { return (p % kvH) % a.groups * a.grows; };
    auto rows_of = [&](int p) { return min(a.grows, a.Mq - group_row(p)); };

    // All consumer warps: Q of pair p into shared memory, in fragment order.  bf16: of each 16 columns, lane
    // (g4, c4) has 2 c4, 2 c4 + 1 and 8 more; f16: 4 c4 .. 4 c4 + 3, the order of the 8-bit K fragments.
    // fetch_q starts the loads (a warp has rows warp, warp + NCW, ..; all of them in flight together; not on the
    // read-only path, as ripe_verify.cu), stage_q writes the rows.
    constexpr int QW = (D + 63) / 64, QR = (C::ROWS + C::NCW - 1) / C::NCW;
    uint32_t qw[QR][QW];
    auto fetch_q = [&](int p) {
        const int h = head_of(p), row0 = group_row(p), mq = rows_of(p);
#pragma unroll
        for (int r = 0; r < QR; ++r) {
            const int i = warp + r * C::NCW;
            const bool have = i < mq;
            const int row = row0 + i, j = have ? row / a.g : 0, hg = have ? row - j * a.g : 0;
            const uint32_t *qp = reinterpret_cast<const uint32_t *>(
                a.q + ((static_cast<size_t>(p / kvH) * a.qB + j) * a.Hq + h * a.g + hg) * D);
#pragma unroll
            for (int u = 0; u < QW; ++u) qw[r][u] = have && u * 32 + lane < D / 2 ? qp[u * 32 + lane] : 0u;
        }
    };
    auto stage_q = [&](int p) {
        if (tid < C::ROWS) {  // a thread for each row's position, bias and visible keys
            const int h = head_of(p), row = group_row(p) + tid, j = row / a.g;
            const bool have = tid < rows_of(p);
            // keys [x, y) of RING tiles at plane w, keys [0, z) of DUAL tiles; of other tiles, keys before T
            int4 r = make_int4(0, 0, 0, -1);
            if (have) {
                int lo;
                const int T = Ts[p / kvH], lq = pa.jloop[pa.j0 + j];
                score_range(pa, T, kDual, pa.R - 1, pa.j0 + j, lq, lo, r.z);
                score_range(pa, T, kRing, lq, pa.j0 + j, lq, r.x, r.y);
                r.w = lq;
            }
            qsees[tid] = r;
            qpos[tid] = have ? pa.j0 + j : -1;
            if (MOD)
                qslope[tid] = a.slopes && have ? __ldg(a.slopes + h * a.g + row - j * a.g) * 1.4426950408889634f : 0.f;
        }
#pragma unroll
        for (int r = 0; r < QR; ++r) {
            const int i = warp + r * C::NCW;
            if (i >= C::ROWS) break;
            float up = 1.f;
            if constexpr (Q8) {
                uint32_t most = 0;  // largest magnitude of the row, as bf16 bits
#pragma unroll
                for (int u = 0; u < QW; ++u) most = max(most, max(qw[r][u] & 0x7FFFu, (qw[r][u] >> 16) & 0x7FFFu));
                most = __reduce_max_sync(0xffffffffu, most);
                // 2^k that brings the row's largest element into [16, 32); 1 for a row with infinities or NaN
                const int ex = static_cast<int>(most >> 7);
                const int k = ex == 255 ? 0 : min(131 - ex, 126);
                up = __uint_as_float(static_cast<uint32_t>(127 + k) << 23);
                if (lane == 0) qscale[i] = a.sx * __uint_as_float(static_cast<uint32_t>(127 - k) << 23);
            }
            uint8_t *dst = qf + (i >> 3) * (D / 32) * 512 + (i & 7) * 64;
#pragma unroll
            for (int u = 0; u < QW; ++u) {
                const int at = u * 32 + lane, ks = at >> 3, x = at & 7;  // columns 2 at, 2 at + 1
                if (at < D / 2) {
                    uint8_t *f = dst + (ks >> 1) * 512 + (ks & 1) * 8;
                    *reinterpret_cast<uint32_t *>(f + (x & 3) * 16 + (x >> 2) * 4) = qw[r][u];
                    if constexpr (Q8) {
                        const __half2 hq = __floats2half2_rn(__uint_as_float(qw[r][u] << 16) * up,
                                                             __uint_as_float(qw[r][u] & 0xFFFF0000u) * up);
                        *reinterpret_cast<uint32_t *>(f + C::QF_BYTES + (x >> 1) * 16 + (x & 1) * 4) =
                            *reinterpret_cast<const uint32_t *>(&hq);
                    }
                }
            }
        }
        st_half = -1;
        named_bar_sync(1, nct);
        if constexpr (C::WIDE) {  // columns without a row need no reference
#pragma unroll
            for (int nq = 0; nq < NQT; ++nq)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    if (qpos[col0 + 8 * nq + e] < 0) seen |= 1u << (2 * nq + e);
        }
    };

    // The CTAs holding tiles of pair p (x: the first of them, y: how many).  Only this CTA's first and last pair can be
    // shared; one thread looks them up at the start.
    auto parts_of = [&](int p) -> int2 {
        return p == P_first ? make_int2(sflag[8], sflag[9]) : p == P_last ? make_int2(sflag[10], sflag[11])
                                                                          : make_int2(static_cast<int>(blockIdx.x), 1);
    };

    // four columns of the output of row i (block position, head) of pair p, and its log-sum-exp
    auto write_row = [&](int p, int i, int c0, float4 acc, float m, float lo, float ll) {
        const float inv = 1.f / lo;
        const int row = group_row(p) + i, j = row / a.g, h = head_of(p) * a.g + (row - j * a.g);
        const size_t orow = (static_cast<size_t>(p / kvH) * a.qB + j) * a.Hq + h;
        __nv_bfloat162 *op = reinterpret_cast<__nv_bfloat162 *>(&a.out[orow * D + c0]);
        op[0] = __floats2bfloat162_rn(acc.x * inv, acc.y * inv);
        op[1] = __floats2bfloat162_rn(acc.z * inv, acc.w * inv);
        if (c0 == 0 && a.lse) a.lse[orow] = (m + __log2f(ll)) * 0.69314718055994531f;
    };

    // Publish this CTA's partial of the pair that tid 0 remembers (finalize's barrier and one fence cover every
    // thread's writes); the last CTA to arrive merges the pair at its end.  Called a tile after the partial was
    // written, when the fence no longer has to wait for the writes, and after the last tile.
    int pending = -1;
    auto publish = [&]() {
        if (tid == 0 && pending >= 0) {
            __threadfence();
            if (arrive_last(&a.counters[pending], parts_of(pending).y, 0)) {
                __threadfence();
                sflag[4 + sflag[3]] = pending;
                sflag[3] += 1;
            }
            pending = -1;
        }
    };

    // ---------------------------------------------------------------- finalize one pair
    auto finalize = [&](int p) {
        const int slot = (tg * WK + kg) * WR + rg;  // this warp's (m, l)
        publish();  // of an earlier pair, if no tile followed it
        if (!C::WIDE || 16 * C::MT * kg < D) {
            float *mw = mo + (C::WIDE ? tg : slot) * C::NQ * C::DP + (C::WIDE ? 16 * C::MT * kg : 0);
#pragma unroll
            for (int mt = 0; mt < C::MT; ++mt)
#pragma unroll
                for (int nq = 0; nq < NQT; ++nq) {
                    const int q0 = 8 * nq + 2 * c4;
                    mw[q0 * C::DP + 16 * mt + g4] = o[mt][nq][0];
                    mw[(q0 + 1) * C::DP + 16 * mt + g4] = o[mt][nq][1];
                    mw[q0 * C::DP + 16 * mt + 8 + g4] = o[mt][nq][2];
                    mw[(q0 + 1) * C::DP + 16 * mt + 8 + g4] = o[mt][nq][3];
                }
        }
#pragma unroll
        for (int nq = 0; nq < NQT; ++nq)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float l = l_lse[nq][e], fix = 0.f;
                if constexpr (!C::WIDE) fix = l_fix[nq][e];
#pragma unroll
                for (int x = 4; x < 32; x <<= 1) {
                    l += __shfl_xor_sync(0xffffffffu, l, x);
                    if (!C::WIDE) fix += __shfl_xor_sync(0xffffffffu, fix, x);
                }
                if (C::WIDE) fix = gfix[warp * C::NQ + 8 * nq + 2 * c4 + e];
                const bool none = C::WIDE ? !(seen >> (2 * nq + e) & 1) : l == 0.f;  // (the same for a wide group)
                const float2 m = refs(nq);
                if (g4 == 0)
                    *reinterpret_cast<float4 *>(&mml[(slot * C::NQ + 8 * nq + 2 * c4 + e) * 4]) =
                        make_float4(none ? -INFINITY : e ? m.y : m.x, l + fix, l, 0.f);
            }
        named_bar_sync(1, nct);
        const bool abort_now = *reinterpret_cast<volatile int *>(&sflag[1]) != 0;
        const bool sole = parts_of(p).y == 1;
        for (int i = tid; i < C::ROWS; i += nct) {
            const int rgi = i / C::NQ, q = i - rgi * C::NQ;
            float M = -INFINITY;
#pragma unroll
            for (int w = 0; w < C::NP; ++w) M = fmaxf(M, mml[((w * WR + rgi) * C::NQ + q) * 4]);
            float L = 0.f, Ll = 0.f;
#pragma unroll
            for (int w = 0; w < C::NP; ++w) {
                const float4 ml = *reinterpret_cast<const float4 *>(&mml[((w * WR + rgi) * C::NQ + q) * 4]);
                const float h = ml.x == -INFINITY ? 0.f : exp2f(0.5f * (ml.x - M));  // twice: the sums may be large
                if (!C::WIDE || w % WK == 0) wq[i * C::NPF + (C::WIDE ? w / WK : w)] = h * h;
                L += h * ml.y * h;
                Ll += h * ml.z * h;
            }
            *reinterpret_cast<float4 *>(&fin[i * 4]) = make_float4(M, L, Ll, 0.f);
        }
        named_bar_sync(1, nct);
        constexpr int D4 = D / 4;
        const int rows = sole ? rows_of(p) : C::ROWS;
        for (int e = tid; e < rows * D4 && !abort_now; e += nct) {
            const int i = e / D4, c0 = 4 * (e - i * D4);
            const int rgi = i / C::NQ, q = i - rgi * C::NQ;
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < C::NPF; ++w) {
                const float f = wq[i * C::NPF + w];  // 0 too: what a weight of 0 does to a NaN stays a NaN
                const float4 v = *reinterpret_cast<const float4 *>(&mo[((w * WR + rgi) * C::NQ + q) * C::DP + c0]);
                acc.x += f * v.x; acc.y += f * v.y; acc.z += f * v.z; acc.w += f * v.w;
            }
            if (sole) {
                write_row(p, i, c0, acc, fin[i * 4], fin[i * 4 + 1], fin[i * 4 + 2]);
            } else {
                if (kDebug && static_cast<int>(blockIdx.x) + p >= a.dbg_part_slots) {
                    atomicOr(a.err, RIPE_DEVERR_BOUNDS);
                    continue;
                }
                const size_t prow = (static_cast<size_t>(blockIdx.x) + p) * C::ROWS + i;
                *reinterpret_cast<float4 *>(&a.part_o[prow * D + c0]) = acc;
                if (c0 == 0)
                    *reinterpret_cast<float4 *>(&a.part_ml[prow * 4]) = *reinterpret_cast<const float4 *>(&fin[i * 4]);
            }
        }
        named_bar_sync(1, nct);  // partials written; the merge buffer is free again
        if (!sole && !abort_now && tid == 0) pending = p;
    };

    // ---------------------------------------------------------------- merge the partials of one pair
    // Runs in the CTA that arrived last, after all of its own tiles (the stage buffers are free).
    auto merge_pair = [&](int p) {
        const int c_first = parts_of(p).x, nparts = parts_of(p).y, mq = rows_of(p);
        constexpr int FEW = 4;
        if (nparts <= FEW) {  // every thread weighs for itself: all loads in flight at once, no barrier
            for (int e = tid; e < mq * (D / 4); e += nct) {
                const int i = e / (D / 4), cx = e - (e / (D / 4)) * (D / 4);
                float4 ml[FEW], v[FEW];
#pragma unroll
                for (int c = 0; c < FEW; ++c) {
                    const size_t prow = (static_cast<size_t>(c_first + (c < nparts ? c : 0)) + p) * C::ROWS + i;
                    ml[c] = __ldcg(reinterpret_cast<const float4 *>(&a.part_ml[prow * 4]));
                    v[c] = __ldcg(reinterpret_cast<const float4 *>(&a.part_o[prow * D + 4 * cx]));
                }
                float M = -INFINITY;
#pragma unroll
                for (int c = 0; c < FEW; ++c)
                    if (c < nparts) M = fmaxf(M, ml[c].x);
                float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
                float L = 0.f, Ll = 0.f;
#pragma unroll
                for (int c = 0; c < FEW; ++c) {
                    if (c >= nparts) continue;
                    // a partial of weight 0 is added all the same: one that has seen a NaN alone has no maximum, and
                    // its NaN has to reach the row
                    const float h = ml[c].x == -INFINITY ? 0.f : exp2f(0.5f * (ml[c].x - M)), w = h * h;
                    acc.x += w * v[c].x; acc.y += w * v[c].y; acc.z += w * v[c].z; acc.w += w * v[c].w;
                    L += h * ml[c].y * h;
                    Ll += h * ml[c].z * h;
                }
                write_row(p, i, 4 * cx, acc, M, L, Ll);
            }
            if (tid == 0) a.counters[p] = 0;
            return;
        }
        float *pw = reinterpret_cast<float *>(stages);  // [nparts][ROWS] m, then weights
        float *pl = pw + nparts * C::ROWS;              // [nparts][ROWS] l
        for (int e = tid; e < nparts * mq; e += nct) {
            const int c = e / mq, i = e - (e / mq) * mq;
            const size_t prow = (static_cast<size_t>(c_first + c) + p) * C::ROWS + i;
            const float2 ml = __ldcg(reinterpret_cast<const float2 *>(&a.part_ml[prow * 4]));
            pw[c * C::ROWS + i] = ml.x;
            pl[c * C::ROWS + i] = ml.y;
        }
        named_bar_sync(1, nct);
        for (int i = tid; i < mq; i += nct) {
            float M = -INFINITY;
            for (int c = 0; c < nparts; ++c) M = fmaxf(M, pw[c * C::ROWS + i]);
            float L = 0.f, Ll = 0.f;
            for (int c = 0; c < nparts; ++c) {
                const float mk = pw[c * C::ROWS + i];
                const size_t prow = (static_cast<size_t>(c_first + c) + p) * C::ROWS + i;
                const float h = mk == -INFINITY ? 0.f : exp2f(0.5f * (mk - M));
                pw[c * C::ROWS + i] = h * h;
                L += h * pl[c * C::ROWS + i] * h;
                Ll += h * __ldcg(&a.part_ml[prow * 4 + 2]) * h;
            }
            fin[i * 4] = M;
            fin[i * 4 + 1] = L;
            fin[i * 4 + 2] = Ll;
        }
        named_bar_sync(1, nct);
        for (int e = tid; e < mq * (D / 4); e += nct) {
            const int i = e / (D / 4), cx = e - (e / (D / 4)) * (D / 4);
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
            for (int c = 0; c < nparts; ++c) {
                const float w = pw[c * C::ROWS + i];
                const float4 v = __ldcg(reinterpret_cast<const float4 *>(
                    &a.part_o[((static_cast<size_t>(c_first + c) + p) * C::ROWS + i) * D + 4 * cx]));
                acc.x += w * v.x; acc.y += w * v.y; acc.z += w * v.z; acc.w += w * v.w;
            }
            write_row(p, i, 4 * cx, acc, fin[i * 4], fin[i * 4 + 1], fin[i * 4 + 2]);
        }
        if (tid == 0) a.counters[p] = 0;
        named_bar_sync(1, nct);
    };

    // Q fragments of columns 32 kp .. + 31 of query tile nq: k-steps 2 kp and 2 kp + 1
    auto q_frag = [&](int kp, int nq, bool half) -> uint4 {
        return lds128(qf0 + (half ? C::QF_BYTES : 0) + (nq * (D / 32) + kp) * 512);
    };
    auto load_q = [&](bool half) {
        if constexpr (!C::WIDE) {
#pragma unroll
            for (int nq = 0; nq < NQT; ++nq)
#pragma unroll
                for (int kp = 0; kp < D / 32; ++kp) {
                    const uint4 w = q_frag(kp, nq, half);
                    qb[2 * kp][nq][0] = w.x;
                    qb[2 * kp][nq][1] = w.y;
                    qb[2 * kp + 1][nq][0] = w.z;
                    qb[2 * kp + 1][nq][1] = w.w;
                }
        }
        st_half = half ? 1 : 0;
    };

    // ---------------------------------------------------------------- one block of keys, in pieces
    // kb0: shared-memory address of the keys (a bf16 tile or an 8-bit record); t0, cnt: first key, keys.
    // FAST: every query sees all 64 keys; HALF: an 8-bit block.
    constexpr uint32_t kBox = C::BOX_ROWS * 64;  // bytes of a box
    struct Scales { float ks, lv, iv; };         // of an 8-bit block: K scale, log2 of the V scale and 1 / it
    auto scales_of = [&](uint32_t kb0) -> Scales {
        const uint4 sc = lds128(kb0 + 128 * D);
        return {__uint_as_float(sc.x), __uint_as_float(sc.y), __uint_as_float(sc.z)};
    };

    // S^T of 16 keys (sub-block kb) and this warp's query columns
    auto scores = [&](uint32_t kb0, int kb, float (&x)[NQT][4], auto half_tag) {
        constexpr bool HALF = decltype(half_tag)::value;
#pragma unroll
        for (int kp = 0; kp < D / 32; ++kp) {
            uint32_t a0[4], a1[4];  // K of k-steps 2 kp, 2 kp + 1
            if constexpr (HALF) {
                const uint4 w = lds128(kb0 + kb * 16 * D + (kp * 32 + lane) * 16);
                q8_to_f16(w.x, a0[0], a0[2]);
                q8_to_f16(w.y, a0[1], a0[3]);
                q8_to_f16(w.z, a1[0], a1[2]);
                q8_to_f16(w.w, a1[1], a1[3]);
            } else {
                const uint32_t row = kb0 + kp * kBox + (static_cast<uint32_t>(16 * kb) + krow_off) * 64;
                ldsm_x4(row + ((kcol_sel ^ swz) << 4), a0[0], a0[1], a0[2], a0[3]);
                ldsm_x4(row + (((2 + kcol_sel) ^ swz) << 4), a1[0], a1[1], a1[2], a1[3]);
            }
#pragma unroll
            for (int nq = 0; nq < NQT; ++nq) {
                uint4 b;
                if constexpr (C::WIDE) b = q_frag(kp, nq, HALF);
                else b = make_uint4(qb[2 * kp][nq][0], qb[2 * kp][nq][1], qb[2 * kp + 1][nq][0], qb[2 * kp + 1][nq][1]);
                if (kp == 0) mma_step<HALF, true>(x[nq], a0, b.x, b.y);
                else mma_step<HALF, false>(x[nq], a0, b.x, b.y);
                mma_step<HALF, false>(x[nq], a1, b.z, b.w);
            }
        }
    };

    // Dot products of SB sub-blocks (the first is sub-block kb1) to scores relative to the column's reference, in
    // log2 units (8-bit: + log2 of the V scale); what a query does not see to -infinity.
    auto relative = [&](const TileDesc &dsc, int t0, int cnt, int kb1, const Scales &sc, float (&x)[C::SB][NQT][4],
                        auto fast_tag, auto half_tag) {
        constexpr bool FAST = decltype(fast_tag)::value, HALF = decltype(half_tag)::value;
#pragma unroll
        for (int nq = 0; nq < NQT; ++nq) {
            float2 qs = make_float2(0.f, 0.f);
            if (HALF) qs = *reinterpret_cast<const float2 *>(&qscale[col0 + 8 * nq]);
            const float2 m = refs(nq);
            if constexpr (FAST && HALF && !MOD) {
                const float2 f = make_float2(qs.x * sc.ks, qs.y * sc.ks);
                const float2 off = make_float2(sc.lv - m.x, sc.lv - m.y);
#pragma unroll
                for (int sb = 0; sb < C::SB; ++sb)
#pragma unroll
                    for (int h = 0; h < 4; h += 2) {
                        const float2 y = fma2(make_float2(x[sb][nq][h], x[sb][nq][h + 1]), f, off);
                        x[sb][nq][h] = y.x;
                        x[sb][nq][h + 1] = y.y;
                    }
            }
#pragma unroll
            for (int e = 0; e < (FAST && HALF && !MOD ? 0 : 2); ++e) {
                const int col = col0 + 8 * nq + e;
                const int jq = FAST && !MOD ? 0 : qpos[col];
                const float f = HALF ? sc.ks * (e ? qs.y : qs.x) : a.sx;
                const float off = HALF ? sc.lv - (e ? m.y : m.x) : -(e ? m.y : m.x);
                // distance of this lane's first key from the query (exact below 2^24), and its visible range
                const int first = t0 + 16 * kb1 + g4;
                const float slope = MOD ? qslope[col] : 0.f;
                const float dist = MOD ? static_cast<float>(first - (dsc.T + jq)) : 0.f;
                int lo = 0, hi = 0, sink = 0, win = 0;
                if (!FAST) {
                    const int4 r = qsees[col];
                    if (dsc.kind == kRing) {
                        lo = r.x;
                        hi = r.w == dsc.plane ? r.y : 0;
                    } else {
                        hi = dsc.kind == kDual ? r.z : dsc.T;
                    }
                    hi = min(hi, t0 + cnt) - first;
                    lo -= first;
                    if (pa.dwin >= 0) {
                        sink = pa.sink - first;
                        win = dsc.T + jq - pa.dwin - first;
                    }
                }
#pragma unroll
                for (int sb = 0; sb < C::SB; ++sb)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int kk = 16 * sb + 8 * h;
                        float &v = x[sb][nq][e + 2 * h];
                        if (MOD == 2)
                            v = capped(v * f, a.cap, a.rcap) + off;
                        else if (MOD && a.cap != 0.f)
                            v = fmaf(-2.f * a.cap, __fdividef(1.f, 1.f + exp2f(v * f)), a.cap + off);
                        else
                            v = fmaf(v, f, off);
                        if (MOD) v = fmaf(slope, dist + static_cast<float>(kk), v);
                        if (!FAST) {
                            bool vis = kk >= lo && kk < hi;
                            if (pa.dwin >= 0) vis = vis && (kk < sink || kk >= win);
                            v = vis ? v : -INFINITY;
                        }
                    }
            }
        }
    };

    // P of 16 keys, rounded (rows g4 and g4 + 8, columns 2 c4 and 2 c4 + 1); adds to the columns' sums
    auto weigh = [&](const float (&x)[4], float (&tl)[2], float (&tr)[2], uint32_t &lo, uint32_t &hi, auto half_tag) {
        constexpr bool HALF = decltype(half_tag)::value;
        const float2 p = make_float2(exp2f(x[0]), exp2f(x[1])), r = make_float2(exp2f(x[2]), exp2f(x[3]));
        const float2 t = add2(make_float2(tl[0], tl[1]), add2(p, r));
        tl[0] = t.x;
        tl[1] = t.y;
        if constexpr (HALF) {
            const __half2 l2 = __floats2half2_rn(p.x, p.y), h2 = __floats2half2_rn(r.x, r.y);
            lo = *reinterpret_cast<const uint32_t *>(&l2);
            hi = *reinterpret_cast<const uint32_t *>(&h2);
        } else {
            const __nv_bfloat162 l2 = __floats2bfloat162_rn(p.x, p.y), h2 = __floats2bfloat162_rn(r.x, r.y);
            tr[0] += __low2float(l2) + __low2float(h2);
            tr[1] += __high2float(l2) + __high2float(h2);
            lo = *reinterpret_cast<const uint32_t *>(&l2);
            hi = *reinterpret_cast<const uint32_t *>(&h2);
        }
    };

    // O^T += V^T P^T over the 16 keys of sub-block kb, for MT column tiles of head_dim from tile mt0 on
    auto accumulate = [&](const TileDesc &dsc, uint32_t kb0, int t0, int cnt, int kb, int mt0, const uint32_t (&pb)[NQT][2],
                          auto fast_tag, auto half_tag) {
        constexpr bool FAST = decltype(fast_tag)::value, HALF = decltype(half_tag)::value;
        if constexpr (HALF) {
            const uint32_t v0 = kb0 + 64 * D + kb * 16 * D + lane * 16;
            if constexpr (C::MT == 1) {
                const uint2 w = lds64(v0 + (mt0 >> 1) * 512 + (mt0 & 1) * 8);
                uint32_t af[4];
                q8_to_f16(w.x, af[0], af[2]);
                q8_to_f16(w.y, af[1], af[3]);
#pragma unroll
                for (int nq = 0; nq < NQT; ++nq) mma_step<true, false>(o[0][nq], af, pb[nq][0], pb[nq][1]);
            } else {
#pragma unroll
                for (int mp = 0; mp < C::MT / 2; ++mp) {
                    const uint4 w = lds128(v0 + (mt0 / 2 + mp) * 512);
                    uint32_t af[4];
                    q8_to_f16(w.x, af[0], af[2]);
                    q8_to_f16(w.y, af[1], af[3]);
#pragma unroll
                    for (int nq = 0; nq < NQT; ++nq) mma_step<true, false>(o[2 * mp][nq], af, pb[nq][0], pb[nq][1]);
                    q8_to_f16(w.z, af[0], af[2]);
                    q8_to_f16(w.w, af[1], af[3]);
#pragma unroll
                    for (int nq = 0; nq < NQT; ++nq) mma_step<true, false>(o[2 * mp + 1][nq], af, pb[nq][0], pb[nq][1]);
                }
            }
        } else {
            const uint32_t v0 = kb0 + C::RING_BYTES / 2 + (static_cast<uint32_t>(16 * kb) + vrow_off) * 64;
            auto v_frag = [&](int mt, uint32_t (&af)[4]) {
                const uint32_t col16 = static_cast<uint32_t>(2 * (mt & 1)) + vcol_sel;
                ldsm_x4_t(v0 + (mt >> 1) * kBox + ((col16 ^ swz) << 4), af[0], af[1], af[2], af[3]);
            };
            bool odd = false;  // a masked tile holding infinities or NaN (stale rows and unwritten ones included)
            if constexpr (!FAST) {
                for (int mt = 0; mt < C::MT; ++mt) {
                    uint32_t af[4];
                    v_frag(mt0 + mt, af);
                    odd = odd || bf16x2_nonfinite(af[0]) || bf16x2_nonfinite(af[1]) || bf16x2_nonfinite(af[2]) ||
                          bf16x2_nonfinite(af[3]);
                }
                odd = __any_sync(0xffffffffu, odd);
            }
            if (!odd) {
#pragma unroll
                for (int mt = 0; mt < C::MT; ++mt) {
                    uint32_t af[4];
                    v_frag(mt0 + mt, af);
#pragma unroll
                    for (int nq = 0; nq < NQT; ++nq) mma_step<false, false>(o[mt][nq], af, pb[nq][0], pb[nq][1]);
                }
            } else {
                // 0 * NaN would reach queries that do not see the row: one block position at a time, with
                // the rows that it does not see taken out of V
                for (int j = pa.j0; j < pa.j0 + a.qB; ++j) {
                    uint32_t m01 = 0, m23 = 0;  // this thread's keys 2 c4, 2 c4 + 1, and 8 more
#pragma unroll 1
                    for (int u = 0; u < 4; ++u) {
                        const int kk = 16 * kb + 2 * c4 + (u & 1) + 4 * (u & 2);
                        if (kk < cnt && score_sees(pa, dsc.T, dsc.kind, dsc.plane, t0 + kk, j, pa.jloop[j])) {
                            const uint32_t m = 0xFFFFu << (16 * (u & 1));
                            m01 |= u < 2 ? m : 0u;
                            m23 |= u < 2 ? 0u : m;
                        }
                    }
#pragma unroll
                    for (int mt = 0; mt < C::MT; ++mt) {
                        uint32_t af[4];
                        v_frag(mt0 + mt, af);
                        af[0] &= m01; af[1] &= m01; af[2] &= m23; af[3] &= m23;
#pragma unroll
                        for (int nq = 0; nq < NQT; ++nq) {
                            float t4[4];
                            mma_step<false, true>(t4, af, pb[nq][0], pb[nq][1]);
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                if (qpos[col0 + 8 * nq + (e & 1)] == j) o[mt][nq][e] += t4[e];
                        }
                    }
                }
            }
        }
    };

    // the block's sums into the columns' (8-bit: over the V scale).  0 * NaN: a column that sees none of a block
    // that reads as NaN takes nothing from it
    auto add_sums = [&](const float (&tl)[NQT][2], const float (&tr)[NQT][2], float iv, auto fast_tag, auto half_tag) {
        constexpr bool FAST = decltype(fast_tag)::value, HALF = decltype(half_tag)::value;
        if constexpr (FAST && HALF) {
#pragma unroll
            for (int nq = 0; nq < NQT; ++nq) {
                const float2 l = fma2(make_float2(tl[nq][0], tl[nq][1]), make_float2(iv, iv),
                                      make_float2(l_lse[nq][0], l_lse[nq][1]));
                l_lse[nq][0] = l.x;
                l_lse[nq][1] = l.y;
            }
        } else {
#pragma unroll
            for (int nq = 0; nq < NQT; ++nq)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float s = !HALF ? tl[nq][e] : !FAST && tl[nq][e] == 0.f ? 0.f : tl[nq][e] * iv;
                    l_lse[nq][e] += s;
                    if constexpr (!HALF) {
                        float fix = tr[nq][e] - tl[nq][e];
                        if constexpr (C::WIDE) {
#pragma unroll
                            for (int x = 4; x < 32; x <<= 1) fix += __shfl_xor_sync(0xffffffffu, fix, x);
                            if (g4 == 0) gfix[warp * C::NQ + 8 * nq + 2 * c4 + e] += fix;
                        } else {
                            l_fix[nq][e] += fix;
                        }
                    }
                }
        }
    };

    // moves a column's reference up by `up`; its sums are worth 2^lg of what they were then
    auto move_ref = [&](int nq, int e, float up, float lg, float (&x)[C::SB][NQT][4]) {
        const bool far = lg < -100.f;  // what O holds is 2^-100 of what comes then; the normaliser may still hold more
        const float al = far ? 0.f : exp2f(lg);
        l_lse[nq][e] *= far ? exp2f(0.5f * lg) : al;
        if (far) l_lse[nq][e] *= exp2f(0.5f * lg);
        if constexpr (C::WIDE) {
            const int col = 8 * nq + 2 * c4 + e;
            if (g4 == 0) gfix[warp * C::NQ + col] *= al;
            if (g4 == 0 && kg == 0) gref[tg * C::NQ + col] += up;
        } else {
            m_ref[nq][e] += up;
            l_fix[nq][e] *= al;
        }
#pragma unroll
        for (int sb = 0; sb < C::SB; ++sb) {
            x[sb][nq][e] -= up;
            x[sb][nq][e + 2] -= up;
        }
#pragma unroll
        for (int mt = 0; mt < C::MT; ++mt) {
            o[mt][nq][e] *= al;
            o[mt][nq][e + 2] *= al;
        }
    };
    // a block with a tiny V scale: its keys' weights to the normaliser, in place of the sums that add_sums adds
    auto sum_tiny = [&](const float (&x)[C::SB][NQT][4], const Scales &sc) {
#pragma unroll
        for (int nq = 0; nq < NQT; ++nq)
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int sb = 0; sb < C::SB; ++sb)
                    l_lse[nq][e] += exp2f(x[sb][nq][e] - sc.lv) + exp2f(x[sb][nq][e + 2] - sc.lv);
    };
    auto column_max = [&](const float (&x)[C::SB][NQT][4], int nq, int e) {
        float m = -INFINITY;
#pragma unroll
        for (int sb = 0; sb < C::SB; ++sb) m = fmaxf(m, fmaxf(x[sb][nq][e], x[sb][nq][e + 2]));
        return m;
    };

    // ---------------------------------------------------------------- a block, each warp on its own keys
    auto compute = [&](const TileDesc &dsc, uint32_t kb0, int t0, int cnt, auto fast_tag, auto half_tag) {
        constexpr bool FAST = decltype(fast_tag)::value, HALF = decltype(half_tag)::value;
        float x[C::SB][NQT][4];
        Scales sc = {1.f, 0.f, 1.f};
        if constexpr (HALF) sc = scales_of(kb0);
#pragma unroll
        for (int sb = 0; sb < C::SB; ++sb) {
            const int kb = kg * C::SB + sb;
            if (!FAST && 16 * kb >= cnt) {
#pragma unroll
                for (int nq = 0; nq < NQT; ++nq) x[sb][nq][0] = x[sb][nq][1] = x[sb][nq][2] = x[sb][nq][3] = 0.f;
            } else {
                scores(kb0, kb, x[sb], half_tag);
            }
        }
        relative(dsc, t0, cnt, kg * C::SB, sc, x, fast_tag, half_tag);
        // The reference moves when a score exceeds it by more than kScoreHi, or when the column has no sum
        // yet; the warp looks at a column's maximum over all lanes only if one lane calls for it (blocks of tiny
        // values, as rare, are dealt with there too).
        bool over = HALF && sc.lv < kTinyScale;
#pragma unroll
        for (int nq = 0; nq < NQT; ++nq)
#pragma unroll
            for (int e = 0; e < 2; ++e)
                over = over || column_max(x, nq, e) > (l_lse[nq][e] == 0.f ? -INFINITY : kScoreHi);
        if (__any_sync(0xffffffffu, over)) {
#pragma unroll
            for (int nq = 0; nq < NQT; ++nq)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float mt = column_max(x, nq, e), l = l_lse[nq][e];
#pragma unroll
                    for (int s = 4; s < 32; s <<= 1) {
                        mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, s));
                        l = fmaxf(l, __shfl_xor_sync(0xffffffffu, l, s));
                    }
                    if (mt > (l == 0.f ? -INFINITY : kScoreHi))
                        move_ref(nq, e, mt - kScoreLo, l == 0.f ? 0.f : kScoreLo - mt, x);
                }
            if (HALF && sc.lv < kTinyScale) sum_tiny(x, sc);
        }
        float tl[NQT][2], tr[NQT][2];
#pragma unroll
        for (int nq = 0; nq < NQT; ++nq) tl[nq][0] = tl[nq][1] = tr[nq][0] = tr[nq][1] = 0.f;
#pragma unroll
        for (int sb = 0; sb < C::SB; ++sb) {
            const int kb = kg * C::SB + sb;
            if (!FAST && 16 * kb >= cnt) continue;
            uint32_t pb[NQT][2];
#pragma unroll
            for (int nq = 0; nq < NQT; ++nq) {
                uint32_t lo, hi;
                weigh(x[sb][nq], tl[nq], tr[nq], lo, hi, half_tag);
                pb[nq][0] = movmatrix_t(lo);  // to the B operand's layout
                pb[nq][1] = movmatrix_t(hi);
            }
            accumulate(dsc, kb0, t0, cnt, kb, 0, pb, fast_tag, half_tag);
        }
        add_sums(tl, tr, HALF && sc.lv < kTinyScale ? 0.f : sc.iv, fast_tag, half_tag);
    };

    // ---------------------------------------------------------------- a block, by the four warps of a wide group
    // Warp kg forms P of sub-block kg and leaves it in shared memory; then it adds all sub-blocks to its quarter
    // of O.  All four keep the same references: a block that has to move one says so before the barrier, and
    // is weighed again after its warps have compared their maxima.  P is double-buffered: a warp that writes the
    // buffer of block n + 2 has passed the barrier of block n + 1, which its readers reach after block n.
    int nblk = 0;
    const uint32_t pbuf0 = smem_addr(qf) + C::Q_BYTES + tg * (C::P_BYTES / TG);
    auto compute_wide = [&](const TileDesc &dsc, uint32_t kb0, int t0, int cnt, auto fast_tag, auto half_tag) {
        constexpr bool FAST = decltype(fast_tag)::value, HALF = decltype(half_tag)::value;
        constexpr int PT = (NQT / 2) * 512;  // bytes of P of a sub-block
        const uint32_t pbuf = pbuf0 + (nblk & 1) * 4 * PT;
        const bool mine = FAST || 16 * kg < cnt;
        float x[C::SB][NQT][4], tl[NQT][2], tr[NQT][2];
        Scales sc = {1.f, 0.f, 1.f};
        if constexpr (HALF) sc = scales_of(kb0);
        // P as 8 x 8 matrices of 128 bytes, rows keys, columns queries: [row tile][keys 0..7, 8..15], which ldmatrix
        // transposes into B fragments.  Returns whether a probability exceeds 2^kScoreHi.
        auto put = [&]() -> bool {
            uint32_t most = 0;
#pragma unroll
            for (int nq = 0; nq < NQT; ++nq) {
                tl[nq][0] = tl[nq][1] = tr[nq][0] = tr[nq][1] = 0.f;
                uint32_t lo, hi;
                weigh(x[0][nq], tl[nq], tr[nq], lo, hi, half_tag);
                const uint32_t at = pbuf + kg * PT + nq * 256 + lane * 4;
                sts32(at, lo);
                sts32(at + 128, hi);
                most = __vmaxu2(most, __vmaxu2(lo, hi));  // probabilities have no sign: ordered as their bits
            }
            const uint32_t bound = HALF ? 0x7800u : 0x4700u;  // 2^15 as f16, as bf16 (NaN is above both: harmless)
            return (most & 0xFFFFu) > bound || (most >> 16) > bound;
        };
        if (mine) {
            scores(kb0, kg, x[0], half_tag);
            relative(dsc, t0, cnt, kg, sc, x, fast_tag, half_tag);
            bool over = put();
            if (seen != (1u << (2 * NQT)) - 1) {  // some column has no reference yet: any score of it calls for one
#pragma unroll
                for (int nq = 0; nq < NQT; ++nq)
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        over = over || (!(seen >> (2 * nq + e) & 1) && column_max(x, nq, e) > -INFINITY);
            }
            if (__any_sync(0xffffffffu, over) && lane == 0) gflag[4 * tg + (nblk & 1)] = nblk;
        } else {
#pragma unroll
            for (int nq = 0; nq < NQT; ++nq) {
                tl[nq][0] = tl[nq][1] = tr[nq][0] = tr[nq][1] = 0.f;
                x[0][nq][0] = x[0][nq][1] = x[0][nq][2] = x[0][nq][3] = -INFINITY;
            }
        }
        named_bar_sync(2 + tg, 128);
        const uint4 flags = lds128(smem_addr(gflag + 4 * tg));
        if (flags.z != ~0u) {  // a warp of the group gave up waiting for this tile
            aborted = true;
            return;
        }
        if (static_cast<int>(nblk & 1 ? flags.y : flags.x) == nblk || (HALF && scales_of(kb0).lv < kTinyScale)) {
            float *gm = gmax + tg * 4 * C::NQ;
#pragma unroll
            for (int nq = 0; nq < NQT; ++nq)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float mt = column_max(x, nq, e);
#pragma unroll
                    for (int s = 4; s < 32; s <<= 1) mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, s));
                    if (g4 == 0) gm[kg * C::NQ + 8 * nq + 2 * c4 + e] = mt;
                }
            named_bar_sync(2 + tg, 128);
#pragma unroll
            for (int nq = 0; nq < NQT; ++nq)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float *g = gm + 8 * nq + 2 * c4 + e;
                    const float mt = fmaxf(fmaxf(g[0], g[C::NQ]), fmaxf(g[2 * C::NQ], g[3 * C::NQ]));
                    const bool has = seen >> (2 * nq + e) & 1;
                    if (mt > (has ? kScoreHi : -INFINITY)) {
                        move_ref(nq, e, mt - kScoreLo, has ? kScoreLo - mt : 0.f, x);
                        seen |= 1u << (2 * nq + e);
                    }
                }
            if (mine) put();
            if (HALF && scales_of(kb0).lv < kTinyScale) {
                sum_tiny(x, scales_of(kb0));
#pragma unroll
                for (int nq = 0; nq < NQT; ++nq) tl[nq][0] = tl[nq][1] = 0.f;
            }
            named_bar_sync(2 + tg, 128);
        }
        if (16 * C::MT * kg < D) {
#pragma unroll
            for (int kb = 0; kb < 4; ++kb) {
                if (!FAST && 16 * kb >= cnt) continue;
                uint32_t pb[NQT][2];
#pragma unroll
                for (int i = 0; i < NQT / 2; ++i)
                    ldsm_x4_t(pbuf + kb * PT + i * 512 + lane * 16, pb[2 * i][0], pb[2 * i][1], pb[2 * i + 1][0],
                              pb[2 * i + 1][1]);
                accumulate(dsc, kb0, t0, cnt, kb, C::MT * kg, pb, fast_tag, half_tag);
            }
        }
        add_sums(tl, tr, sc.iv, fast_tag, half_tag);
        ++nblk;
    };
    auto block = [&](const TileDesc &dsc, uint32_t kb0, int t0, int cnt, auto fast_tag, auto half_tag) {
        if constexpr (C::WIDE) compute_wide(dsc, kb0, t0, cnt, fast_tag, half_tag);
        else compute(dsc, kb0, t0, cnt, fast_tag, half_tag);
    };

    // Every consumer warp takes the CTA's pairs in order (finalize and stage_q synchronise all of them) and its
    // group's tiles, each in its pair.
    const bool ring_all_visible = pa.nloops == 1 && pa.dwin < 0;
    int i = tg;
    bool here = false;  // tile i has landed
    if (a.early) pdl_wait();  // the caller may be writing the queries
    fetch_q(P_first);
    if (tid == 32) {
#pragma unroll 1
        for (int k = 0; k < 2; ++k) {
            const int2 f = score_parts(a, cp, cum, Ts, kvH, k ? P_last : P_first);
            sflag[8 + 2 * k] = f.x;
            sflag[9 + 2 * k] = f.y;
        }
    }
    for (int p = P_first; p <= P_last; ++p) {
        reset_state();
        stage_q(p);
        while (i < ntiles) {
            const int s = i % NS;
            if (!here) {
                if (!mbar_wait_bounded(full0 + 8 * s, (i / NS) & 1)) {
                    aborted = true;
                    atomicOr(a.err, RIPE_DEVERR_WAIT_TIMEOUT);
                    *reinterpret_cast<volatile int *>(&sflag[1]) = 1;
                    if constexpr (C::WIDE) {  // the group's other warps may be waiting for this one's P: all stop here
                        if (lane == 0) gflag[4 * tg + 2] = 1;
                        __syncwarp();
                        named_bar_sync(2 + tg, 128);
                    }
                    i = ntiles;
                    break;
                }
                here = true;
            }
            const TileDesc dsc = sdesc[s];
            if (dsc.pair != p) break;
            const bool half = Q8 && dsc.kind == kDeep;
            if (!C::WIDE && st_half != (half ? 1 : 0)) load_q(half);
            const uint32_t base = stage0 + s * C::STAGE_BYTES;
            // mask-free: deepest-plane rows outside a draft window, or a full ring tile that every query of
            // the call sees whole (one loop; every key before the first query and in the last one's window)
            const int last = dsc.T + pa.j0 + a.qB - 1;
            const bool whole =
                dsc.kind == kDeep ? pa.dwin < 0
                                  : dsc.kind == kRing && ring_all_visible && dsc.t0 + kTileRows - 1 <= dsc.T + pa.j0 &&
                                        (pa.all_deepest || pa.crel || dsc.t0 >= last - pa.W);
            if constexpr (Q8) {
                if (half) {
                    for (int b = 0; b < (dsc.cnt >> 6); ++b) {
                        const uint32_t rb = base + b * q8_record_bytes(D);
                        if (whole)
                            block(dsc, rb, dsc.t0 + 64 * b, 64, std::true_type(), std::true_type());
                        else
                            block(dsc, rb, dsc.t0 + 64 * b, 64, std::false_type(), std::true_type());
                    }
                }
            }
            if (!half) {
                if (!Q8 && whole && dsc.cnt == kTileRows)
                    block(dsc, base, dsc.t0, dsc.cnt, std::true_type(), std::false_type());
                else
                    block(dsc, base, dsc.t0, dsc.cnt, std::false_type(), std::false_type());
            }
            if (C::WIDE && aborted) {
                i = ntiles;
                break;
            }
            publish();
            __syncwarp();
            if (lane == 0) mbar_arrive(empty0 + 8 * s);
            here = false;
            i += TG;
        }
        if (p < P_last) fetch_q(p + 1);
        finalize(p);
    }
    publish();
    named_bar_sync(1, nct);
    if (*reinterpret_cast<volatile int *>(&sflag[1]) == 0) {
        const int nm = sflag[3];
        for (int k = 0; k < nm; ++k) merge_pair(sflag[4 + k]);
    }
}

// ---------------------------------------------------------------- host side
template <int D, int NQT, int WR, int WK, int TG, bool Q8, int MOD>
struct ScoreInst {
    using C = SCfg<D, NQT, WR, WK, TG, Q8>;
    static constexpr auto kernel = ripe_score_kernel<D, NQT, WR, WK, TG, Q8, MOD>;
    static cudaError_t set_attr() {
        if constexpr (C::SPLIT) {
            // with fewer registers at launch the consumers' setmaxnreg.inc could never be satisfied
            cudaFuncAttributes fa;
            const cudaError_t e = cudaFuncGetAttributes(&fa, kernel);
            if (e != cudaSuccess) return e;
            if (fa.numRegs * C::THREADS < C::NCW * 32 * C::REG_CONSUMER + 4 * 32 * C::REG_PRODUCER)
                return cudaErrorInvalidConfiguration;
        }
        return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::smem_bytes(kMaxBatch));
    }
    static cudaError_t launch(const LaunchTarget &t, int grid, const ScoreArgs &a, cudaStream_t s) {
        if (grid > C::MAX_PARTS) grid = C::MAX_PARTS;
        return launch_pdl(kernel, dim3(grid), dim3(C::THREADS), C::smem_bytes(t.N), s, *t.tmKd, *t.tmVd, *t.tmKw,
                          *t.tmVw, a);
    }
};

// Query-side configuration by the query rows of a row group.
template <int D, bool Q8, int MOD>
struct ScoreSet {
    using R8 = ScoreInst<D, 1, 1, 4, 2, Q8, MOD>;
    using R16 = ScoreInst<D, 2, 1, 4, 2, Q8, MOD>;
    using Wide = ScoreInst<D, 4, 1, 4, 3, Q8, MOD>;
    using Narrow = ScoreInst<D, 2, 2, 2, 2, Q8, MOD>;
    using R32 = std::conditional_t<Q8, Wide, Narrow>;
    static cudaError_t set_attr() {
        cudaError_t e = R8::set_attr();
        if (e == cudaSuccess) e = R16::set_attr();
        if (e == cudaSuccess) e = R32::set_attr();
        return e;
    }
    static cudaError_t launch(const LaunchTarget &t, int grid, const ScoreArgs &a, cudaStream_t s) {
        if (a.grows <= 8) return R8::launch(t, grid, a, s);
        if (a.grows <= 16) return R16::launch(t, grid, a, s);
        return R32::launch(t, grid, a, s);
    }
};

}  // namespace ripe
