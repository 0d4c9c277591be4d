// Attention over a RIPE cache whose deepest-plane region is held in 8 bits (Q8), or with capped or
// distance-biased scores (MOD); included by the translation units that instantiate it.
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
//     down to 2^-18 of the row's largest; P is rounded to f16 (2^-11 relative).
//   * The K scale enters with the softmax scale; the V scale enters the exponent: p' = 2^(x + log2 s -
//     m), O sums p' u, and the normaliser sums p' / s.  So a block costs no multiply of its own per
//     element, and the reference m follows the size of p' u, which is what O accumulates.
//   * tanh y = 1 - 2 / (1 + e^2y): one exponential and one reciprocal, absolute error 2^-22 of the cap
//     (the hardware's tanh is 2^-11 relative: 0.02 at a cap of 50).
//   * A masked value never reaches a sum: stale ring rows or later draft rows may hold NaN or infinity.
#pragma once

#include <cuda_fp16.h>

#include <mutex>
#include <type_traits>

#include "ripe_score.cuh"

namespace ripe {

// softmax reference: moved when a score exceeds it by more than kHi, and then to kLo below the maximum, so
// that the probabilities lie in (0, 2^15], within f16's range, and are exact down to 2^-(14 + 10 + kLo)
constexpr float kScoreHi = 15.f, kScoreLo = 7.f;

// Query-side shapes as VCfg (ripe_verify.cu): NQT 8-query tiles per warp, WR row groups, WK key groups
// per 64-key block, TG tile groups consuming alternate tiles.
template <int D, int NQT, int WR, int WK, int TG, bool Q8>
struct SCfg {
    static constexpr int NQ = 8 * NQT;
    static constexpr int ROWS = NQ * WR;
    static constexpr int GW = WR * WK;
    static constexpr int NCW = GW * TG;
    // with two query tiles per warp the producer warp heads a warpgroup that gives registers up
    static constexpr bool SPLIT = NQT >= 2;
    static constexpr int THREADS = SPLIT ? (NCW + 4) * 32 : (NCW + 1) * 32;
    static constexpr int LAUNCH_REGS = (65536 / THREADS) / 8 * 8 > 255 ? 248 : (65536 / THREADS) / 8 * 8;
    static constexpr int REG_PRODUCER = 72;
    static constexpr int REG_FREE = ((LAUNCH_REGS * (NCW + 4) - 4 * REG_PRODUCER) / NCW) / 8 * 8;
    static constexpr int REG_CONSUMER = REG_FREE > 248 ? 248 : REG_FREE;
    static_assert(NCW % 4 == 0, "consumer warps form whole warpgroups");
    static_assert(NCW * REG_CONSUMER + 4 * REG_PRODUCER <= (NCW + 4) * LAUNCH_REGS, "register split");
    static constexpr int SB = 4 / WK;  // 16-key sub-blocks per warp and block
    static constexpr int NBOX = D / kBoxCols;
    static constexpr int STAGE_BYTES = Q8 ? (2 * q8_record_bytes(D) + 1023) / 1024 * 1024 : 2 * NBOX * kBoxBytes;
    static_assert(STAGE_BYTES >= 2 * NBOX * kBoxBytes, "a stage holds a bf16 tile too");
    static constexpr int DP = D + 4;
    static constexpr int MERGE_FLOATS = NCW * NQ * DP;
    static constexpr int MLF = NCW * NQ * 4 + ROWS * (TG * WK + 4);
    static constexpr int MISC = 1024 + 1024;
    static constexpr int AVAIL = kSmemLimit - MISC - 4 * (MERGE_FLOATS + MLF) - 4 * (2 * kMaxBatch + 2);
    static constexpr int NS_RAW = AVAIL / STAGE_BYTES > 8 ? 8 : AVAIL / STAGE_BYTES;
    static constexpr int NS = NS_RAW - NS_RAW % TG;  // a stage always serves the same tile group
    static_assert(NS >= 2, "not enough shared memory for the pipeline");
    static constexpr int SMEM_FIXED = MISC + NS * STAGE_BYTES + 4 * (MERGE_FLOATS + MLF);
    static_assert(SMEM_FIXED + 4 * (2 * kMaxBatch + 2) <= kSmemLimit, "shared memory");
    static constexpr int MAX_PARTS =
        (NS * STAGE_BYTES) / (2 * ROWS * 4) < 256 ? (NS * STAGE_BYTES) / (2 * ROWS * 4) : 256;
    static_assert(MAX_PARTS >= 148, "stage buffers too small for the end-of-CTA merge");
    static constexpr int smem_bytes(int N) { return SMEM_FIXED + (2 * N + 2) * 4; }
};

__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(bar)
                 : "memory");
}

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

__device__ __forceinline__ void mma_16816_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
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

// The chunk of the concatenated tile lists that this CTA streams (as plan_chunks in ripe_verify.cuh).
struct ScoreChunk {
    int total, chunk, pieces, tot_head, head, g_begin, g_end;
};

__device__ __forceinline__ ScoreChunk score_chunks(const ScoreArgs &a, int *cum, int *Ts, int *sflag, int tid, int warp,
                                                   int lane) {
    const int N = a.N, kvH = a.kvH;
    ScoreChunk c;
    for (int n = tid; n < N; n += blockDim.x) {
        const int T = a.T[n];
        Ts[n] = T;
        cum[n + 1] = score_geom(T, a.plan).total * kvH;
    }
    if (tid == 0) cum[0] = 0;
    __syncthreads();
    pdl_trigger();  // the next kernel may be scheduled; it waits for this one to finish
    if (warp == 0) {
        int carry = 0;
        bool same = true;
        const int first = cum[1];
        for (int b = 0; b < N; b += 32) {
            const int own = (b + lane < N) ? cum[b + lane + 1] : 0;
            same = same && __all_sync(0xffffffffu, b + lane >= N || own == first);
            int v = own;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int u = __shfl_up_sync(0xffffffffu, v, o);
                if (lane >= o) v += u;
            }
            if (b + lane < N) cum[b + lane + 1] = v + carry;
            carry += __shfl_sync(0xffffffffu, v, 31);
        }
        if (lane == 0) {
            int ch, pc;
            choose_chunk(carry, first / kvH, same, static_cast<int>(gridDim.x), N, kvH, a.min_chunk, ch, pc);
            sflag[6] = ch;
            sflag[7] = pc;
        }
    }
    __syncthreads();
    c.total = cum[N];
    c.chunk = sflag[6];
    c.pieces = sflag[7];
    c.tot_head = c.pieces ? cum[1] / kvH : 0;
    c.head = 0;
    if (c.pieces) {
        c.head = blockIdx.x / c.pieces;
        c.g_begin = c.head * c.tot_head + (blockIdx.x - c.head * c.pieces) * c.chunk;
        c.g_end = min(min(c.g_begin + c.chunk, (c.head + 1) * c.tot_head), c.total);
    } else {
        c.g_begin = blockIdx.x * c.chunk;
        c.g_end = min(c.total, c.g_begin + c.chunk);
    }
    return c;
}

template <int D, int NQT, int WR, int WK, int TG, bool Q8, bool MOD>
__global__ void __launch_bounds__(SCfg<D, NQT, WR, WK, TG, Q8>::THREADS, 1)
ripe_score_kernel(const __grid_constant__ CUtensorMap tmKd, const __grid_constant__ CUtensorMap tmVd,
                  const __grid_constant__ CUtensorMap tmKw, const __grid_constant__ CUtensorMap tmVw,
                  const __grid_constant__ ScoreArgs a) {
    using C = SCfg<D, NQT, WR, WK, TG, Q8>;
    constexpr int NS = C::NS;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *stages = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                  ~static_cast<uintptr_t>(1023));
    float *mo = reinterpret_cast<float *>(stages + NS * C::STAGE_BYTES);  // [NCW][NQ][DP]
    float *mml = mo + C::MERGE_FLOATS;                                    // [NCW][NQ][4] m, l_out, l_lse
    float *wq = mml + C::NCW * C::NQ * 4;                                 // [ROWS][TG*WK] weights
    float *fin = wq + C::ROWS * TG * WK;                                  // [ROWS][4] final m, l_out, l_lse
    uint64_t *bars = reinterpret_cast<uint64_t *>(mml + C::MLF);          // full[NS], empty[NS]
    TileDesc *sdesc = reinterpret_cast<TileDesc *>(bars + 2 * NS);        // [NS]
    int *sflag = reinterpret_cast<int *>(sdesc + NS);                     // [16]
    int *cum = sflag + 16;                                                // [N + 1]
    int *Ts = cum + a.N + 1;                                              // [N]

    const int tid = threadIdx.x;
    const int warp = tid >> 5;
    const int lane = tid & 31;
    const ScorePlan &pa = a.plan;
    const int N = a.N, kvH = a.kvH;

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
    // rows past a short box are never written by TMA: keep them finite
    if (pa.deep_box < kTileRows || pa.ring_box < kTileRows) {
        uint4 *z = reinterpret_cast<uint4 *>(stages);
        for (int i = tid; i < NS * C::STAGE_BYTES / 16; i += blockDim.x) z[i] = make_uint4(0, 0, 0, 0);
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    if (!a.early) pdl_wait();
    const ScoreChunk cp = score_chunks(a, cum, Ts, sflag, tid, warp, lane);
    const int chunk = cp.chunk, pieces = cp.pieces;
    const int g_begin = cp.g_begin, g_end = cp.g_end;
    if (g_begin >= g_end) {
        if (a.early) pdl_wait();  // the launch completes only after its predecessor
        return;
    }
    const int ntiles = g_end - g_begin;
    const int P_first = pieces ? cp.head : pair_of(cum, N, kvH, g_begin);
    const int P_last = pieces ? cp.head : pair_of(cum, N, kvH, g_end - 1);
    const uint32_t full0 = smem_addr(&bars[0]);
    const uint32_t empty0 = smem_addr(&bars[NS]);
    const uint32_t stage0 = smem_addr(stages);

    if (warp >= C::NCW) {
        // ================================================================ producer (one thread)
        if constexpr (C::SPLIT) setmaxnreg_dec<C::REG_PRODUCER>();
        if (warp != C::NCW || lane != 0) return;
        int n = P_first / kvH, kh = P_first - (P_first / kvH) * kvH;
        ScoreGeom sg = score_geom(Ts[n], pa);
        int lt = g_begin - (cum[n] + kh * sg.total);
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
                const size_t r = (static_cast<size_t>(a.layer) * N + n) * kvH + kh;
                mbar_expect_tx(fb, bytes);
                bulk_load(kdst, a.rec + (r * a.rec_blocks + (t.t0 >> 6)) * q8_record_bytes(D), bytes, fb);
            } else {
                const int rows = deep ? pa.deep_box : pa.ring_box;
                const CUtensorMap *mk = deep ? &tmKd : &tmKw;
                const CUtensorMap *mv = deep ? &tmVd : &tmVw;
                const int z = deep ? ((a.layer * N + n) * kvH + kh) : (((a.layer * N + n) * pa.R + t.plane) * kvH + kh);
                const uint32_t vdst = kdst + C::NBOX * kBoxBytes;
                mbar_expect_tx(fb, 2 * C::NBOX * rows * 64);
#pragma unroll
                for (int b = 0; b < C::NBOX; ++b) {
                    tma_load_3d(kdst + b * kBoxBytes, mk, fb, b * kBoxCols, t.y, z);
                    tma_load_3d(vdst + b * kBoxBytes, mv, fb, b * kBoxCols, t.y, z);
                }
            }
            if (++lt == sg.total) {
                lt = 0;
                if (++kh == kvH) {
                    kh = 0;
                    if (++n < N) sg = score_geom(Ts[n], pa);
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

    // query columns held by this thread: NQ*rg + 8*nq + 2*c4 + e
    int jq[NQT][2];
#pragma unroll
    for (int nq = 0; nq < NQT; ++nq)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int i = C::NQ * rg + 8 * nq + 2 * c4 + e;
            jq[nq][e] = i < a.Mq ? pa.j0 + i / a.g : -1;
        }
    // ldmatrix lane geometry of the bf16 tiles (64-byte swizzle: 16-byte chunk ^= (row >> 1) & 3)
    const int mi = lane >> 3, r8 = lane & 7;
    const uint32_t swz = static_cast<uint32_t>(r8 >> 1);
    const uint32_t krow_off = static_cast<uint32_t>((mi & 1) * 8 + r8);
    const uint32_t kcol_sel = static_cast<uint32_t>(mi >> 1);
    const uint32_t vrow_off = static_cast<uint32_t>((mi >> 1) * 8 + r8);
    const uint32_t vcol_sel = static_cast<uint32_t>(mi & 1);

    float o[D / 16][NQT][4];
    // l_lse sums the probabilities in fp32, l_out as the P V product of a bf16 tile sees them (rounded)
    float m_ref[NQT][2], l_lse[NQT][2], l_out[NQT][2];
    uint32_t qb[D / 16][NQT][2];  // Q as B fragments: bf16, or f16 in the column order of 8-bit tiles
    float fcol[NQT][2];           // 8-bit tiles: sx over the power of two that scaled the row
    float slope[NQT][2];          // distance bias of the column's head

    int fin_next = P_first;
    int st_pair = -1;
    bool st_half = false;  // qb holds the f16 form
    bool aborted = false;

    auto reset_state = [&]() {
#pragma unroll
        for (int mt = 0; mt < D / 16; ++mt)
#pragma unroll
            for (int nq = 0; nq < NQT; ++nq) o[mt][nq][0] = o[mt][nq][1] = o[mt][nq][2] = o[mt][nq][3] = 0.f;
#pragma unroll
        for (int nq = 0; nq < NQT; ++nq) {
            m_ref[nq][0] = m_ref[nq][1] = -INFINITY;
            l_lse[nq][0] = l_lse[nq][1] = 0.f;
            l_out[nq][0] = l_out[nq][1] = 0.f;
        }
    };

    auto load_q = [&](int n, int kh, bool half) {
        st_half = half;
#pragma unroll
        for (int nq = 0; nq < NQT; ++nq) {
            const int i = C::NQ * rg + 8 * nq + g4;  // B-operand column = query g4 of the tile
            const uint32_t *qp = nullptr;
            if (i < a.Mq) {
                const int j = i / a.g, hg = i - j * a.g;
                qp = reinterpret_cast<const uint32_t *>(
                    a.q + ((static_cast<size_t>(n) * a.qB + j) * a.Hq + kh * a.g + hg) * D);
            }
            if (Q8 && half) {
                uint32_t most = 0;  // largest magnitude of the row, as bf16 bits
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks) {
                    uint2 w = make_uint2(0, 0);
                    if (qp) w = __ldg(reinterpret_cast<const uint2 *>(qp + 8 * ks + 2 * c4));
                    qb[ks][nq][0] = w.x;
                    qb[ks][nq][1] = w.y;
                    most = max(most, max(max(w.x & 0x7FFFu, (w.x >> 16) & 0x7FFFu),
                                         max(w.y & 0x7FFFu, (w.y >> 16) & 0x7FFFu)));
                }
                most = max(most, __shfl_xor_sync(0xffffffffu, most, 1));
                most = max(most, __shfl_xor_sync(0xffffffffu, most, 2));
                // 2^k that brings the row's largest element into [16, 32); 1 for a row with infinities or NaN
                const int ex = static_cast<int>(most >> 7);
                const int k = ex == 255 ? 0 : min(131 - ex, 126);
                const float up = __uint_as_float(static_cast<uint32_t>(127 + k) << 23);
                const float down = __uint_as_float(static_cast<uint32_t>(127 - k) << 23);
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const uint32_t w = qb[ks][nq][x];
                        const __half2 h = __floats2half2_rn(__uint_as_float(w << 16) * up,
                                                            __uint_as_float(w & 0xFFFF0000u) * up);
                        qb[ks][nq][x] = *reinterpret_cast<const uint32_t *>(&h);
                    }
#pragma unroll
                for (int e = 0; e < 2; ++e) fcol[nq][e] = a.sx * __shfl_sync(0xffffffffu, down, (2 * c4 + e) * 4);
            } else {
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks) {
                    qb[ks][nq][0] = qp ? __ldg(qp + 8 * ks + c4) : 0u;
                    qb[ks][nq][1] = qp ? __ldg(qp + 8 * ks + 4 + c4) : 0u;
                }
            }
            if (MOD) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int ic = C::NQ * rg + 8 * nq + 2 * c4 + e;
                    slope[nq][e] = a.slopes && ic < a.Mq ? __ldg(a.slopes + kh * a.g + ic % a.g) * 1.4426950408889634f : 0.f;
                }
            }
        }
    };

    // the CTAs holding tiles of pair p: c_first .. c_first + nparts - 1 (returns nparts)
    auto parts_of = [&](int p, int &c_first) -> int {
        const int n = p / kvH, kh = p - (p / kvH) * kvH;
        const int tot_n = (cum[n + 1] - cum[n]) / kvH;
        if (pieces) {
            c_first = p * pieces;
            return cdiv(tot_n, chunk);
        }
        const int start = cum[n] + kh * tot_n;
        c_first = start / chunk;
        return (start + tot_n - 1) / chunk - c_first + 1;
    };

    // four columns of the output of row i (block position, head) of pair p, and its log-sum-exp
    auto write_row = [&](int p, int i, int c0, float4 acc, float m, float lo, float ll) {
        const int n = p / kvH, kh = p - (p / kvH) * kvH;
        const float inv = 1.f / lo;
        const int j = i / a.g, h = kh * a.g + (i - j * a.g);
        const size_t orow = (static_cast<size_t>(n) * a.qB + j) * a.Hq + h;
        __nv_bfloat162 *op = reinterpret_cast<__nv_bfloat162 *>(&a.out[orow * D + c0]);
        op[0] = __floats2bfloat162_rn(acc.x * inv, acc.y * inv);
        op[1] = __floats2bfloat162_rn(acc.z * inv, acc.w * inv);
        if (c0 == 0 && a.lse) a.lse[orow] = (m + __log2f(ll)) * 0.69314718055994531f;
    };

    // ---------------------------------------------------------------- finalize one pair
    auto finalize = [&](int p, bool have) {
        float *mw = mo + warp * C::NQ * C::DP;
        if (have) {
#pragma unroll
            for (int nq = 0; nq < NQT; ++nq)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float l = l_lse[nq][e], lb = l_out[nq][e];
#pragma unroll
                    for (int x = 4; x < 32; x <<= 1) {
                        l += __shfl_xor_sync(0xffffffffu, l, x);
                        lb += __shfl_xor_sync(0xffffffffu, lb, x);
                    }
                    l_lse[nq][e] = l;
                    l_out[nq][e] = lb;
                }
#pragma unroll
            for (int mt = 0; mt < D / 16; ++mt)
#pragma unroll
                for (int nq = 0; nq < NQT; ++nq) {
                    const int q0 = 8 * nq + 2 * c4;
                    mw[q0 * C::DP + 16 * mt + g4] = o[mt][nq][0];
                    mw[(q0 + 1) * C::DP + 16 * mt + g4] = o[mt][nq][1];
                    mw[q0 * C::DP + 16 * mt + 8 + g4] = o[mt][nq][2];
                    mw[(q0 + 1) * C::DP + 16 * mt + 8 + g4] = o[mt][nq][3];
                }
            if (g4 == 0) {
#pragma unroll
                for (int nq = 0; nq < NQT; ++nq)
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        *reinterpret_cast<float4 *>(&mml[(warp * C::NQ + 8 * nq + 2 * c4 + e) * 4]) =
                            make_float4(m_ref[nq][e], l_out[nq][e], l_lse[nq][e], 0.f);
            }
        } else {
            for (int q = lane; q < C::NQ; q += 32)
                *reinterpret_cast<float4 *>(&mml[(warp * C::NQ + q) * 4]) = make_float4(-INFINITY, 0.f, 0.f, 0.f);
        }
        named_bar_sync(1, nct);
        const bool abort_now = *reinterpret_cast<volatile int *>(&sflag[1]) != 0;
        int c_first;
        const int nparts = parts_of(p, c_first);
        const bool sole = nparts == 1;
        for (int i = tid; i < C::ROWS; i += nct) {
            const int rgi = i / C::NQ, q = i - rgi * C::NQ;
            float M = -INFINITY;
#pragma unroll
            for (int w = 0; w < TG * WK; ++w)
                M = fmaxf(M, mml[(((w / WK) * C::GW + rgi * WK + w % WK) * C::NQ + q) * 4]);
            float L = 0.f, Ll = 0.f;
#pragma unroll
            for (int w = 0; w < TG * WK; ++w) {
                const float4 ml = *reinterpret_cast<const float4 *>(
                    &mml[(((w / WK) * C::GW + rgi * WK + w % WK) * C::NQ + q) * 4]);
                // a partial without a reference has no sums, or NaN of a block that reads as NaN
                const float f = ml.x == -INFINITY ? (ml.z == 0.f ? 0.f : ml.z) : exp2f(ml.x - M);
                wq[i * (TG * WK) + w] = f;
                L += f * ml.y;
                Ll += f * ml.z;
            }
            *reinterpret_cast<float4 *>(&fin[i * 4]) = make_float4(M, L, Ll, 0.f);
        }
        named_bar_sync(1, nct);
        constexpr int D4 = D / 4;
        const int rows = sole ? a.Mq : C::ROWS;
        for (int e = tid; e < rows * D4 && !abort_now; e += nct) {
            const int i = e / D4, c0 = 4 * (e - i * D4);
            const int rgi = i / C::NQ, q = i - rgi * C::NQ;
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < TG * WK; ++w) {
                const float f = wq[i * (TG * WK) + w];
                if (f != 0.f) {
                    const float4 v = *reinterpret_cast<const float4 *>(
                        &mo[(((w / WK) * C::GW + rgi * WK + w % WK) * C::NQ + q) * C::DP + c0]);
                    acc.x += f * v.x; acc.y += f * v.y; acc.z += f * v.z; acc.w += f * v.w;
                }
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
        if (!sole && !abort_now && tid == 0) {
            // publish this CTA's partial (bar.sync + one fence covers every thread's writes)
            __threadfence();
            if (arrive_last(&a.counters[p], nparts, 0)) {
                __threadfence();
                sflag[4 + sflag[3]] = p;  // merged at the end of this CTA's tiles
                sflag[3] += 1;
            }
        }
    };

    // ---------------------------------------------------------------- merge the partials of one pair
    // Runs in the CTA that arrived last, after all of its own tiles (the stage buffers are free).
    auto merge_pair = [&](int p) {
        int c_first;
        const int nparts = parts_of(p, c_first);
        float *pw = reinterpret_cast<float *>(stages);  // [nparts][ROWS] m, then weights
        float *pl = pw + nparts * C::ROWS;              // [nparts][ROWS] l
        for (int e = tid; e < nparts * a.Mq; e += nct) {
            const int c = e / a.Mq, i = e - (e / a.Mq) * a.Mq;
            const size_t prow = (static_cast<size_t>(c_first + c) + p) * C::ROWS + i;
            const float2 ml = __ldcg(reinterpret_cast<const float2 *>(&a.part_ml[prow * 4]));
            pw[c * C::ROWS + i] = ml.x;
            pl[c * C::ROWS + i] = ml.y;
        }
        named_bar_sync(1, nct);
        for (int i = tid; i < a.Mq; i += nct) {
            float M = -INFINITY;
            for (int c = 0; c < nparts; ++c) M = fmaxf(M, pw[c * C::ROWS + i]);
            float L = 0.f, Ll = 0.f;
            for (int c = 0; c < nparts; ++c) {
                const float mk = pw[c * C::ROWS + i];
                const size_t prow = (static_cast<size_t>(c_first + c) + p) * C::ROWS + i;
                const float ll = __ldcg(&a.part_ml[prow * 4 + 2]);
                const float w = mk == -INFINITY ? (ll == 0.f ? 0.f : ll) : exp2f(mk - M);
                pw[c * C::ROWS + i] = w;
                L += w * pl[c * C::ROWS + i];
                Ll += w * ll;
            }
            fin[i * 4] = M;
            fin[i * 4 + 1] = L;
            fin[i * 4 + 2] = Ll;
        }
        named_bar_sync(1, nct);
        for (int e = tid; e < a.Mq * (D / 4); e += nct) {
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

    // ---------------------------------------------------------------- 64 keys of one tile
    // kb0: shared-memory address of the keys (a bf16 tile or an 8-bit record); t0, cnt: first key, keys
    auto compute = [&](const TileDesc &dsc, uint32_t kb0, int t0, int cnt, auto fast_tag, auto half_tag) {
        constexpr bool FAST = decltype(fast_tag)::value;   // every query sees all 64 keys
        constexpr bool HALF = decltype(half_tag)::value;   // an 8-bit block
        const uint32_t vb0 = kb0 + (HALF ? 64 * D : C::NBOX * kBoxBytes);
        float x[C::SB][NQT][4];
        bool act[C::SB];
        float ks = 1.f, lv = 0.f, iv = 1.f;
        if constexpr (HALF) {
            const uint4 sc = lds128(kb0 + 128 * D);
            ks = __uint_as_float(sc.x);
            lv = __uint_as_float(sc.y);
            iv = __uint_as_float(sc.z);
        }
#pragma unroll
        for (int sb = 0; sb < C::SB; ++sb) {
            const int kb = kg * C::SB + sb;
            act[sb] = FAST || 16 * kb < cnt;
            float se[NQT][4], so[NQT][4];
#pragma unroll
            for (int nq = 0; nq < NQT; ++nq)
#pragma unroll
                for (int e = 0; e < 4; ++e) se[nq][e] = so[nq][e] = 0.f;
            if (act[sb]) {
                if constexpr (HALF) {
#pragma unroll
                    for (int kp = 0; kp < D / 32; ++kp) {
                        const uint4 w = lds128(kb0 + kb * 16 * D + (kp * 32 + lane) * 16);
                        uint32_t af[4];
                        q8_to_f16(w.x, af[0], af[2]);
                        q8_to_f16(w.y, af[1], af[3]);
#pragma unroll
                        for (int nq = 0; nq < NQT; ++nq) mma_16816_f16(se[nq], af, qb[2 * kp][nq][0], qb[2 * kp][nq][1]);
                        q8_to_f16(w.z, af[0], af[2]);
                        q8_to_f16(w.w, af[1], af[3]);
#pragma unroll
                        for (int nq = 0; nq < NQT; ++nq)
                            mma_16816_f16(so[nq], af, qb[2 * kp + 1][nq][0], qb[2 * kp + 1][nq][1]);
                    }
                } else {
                    const uint32_t krow = static_cast<uint32_t>(16 * kb) + krow_off;
#pragma unroll
                    for (int ks2 = 0; ks2 < D / 16; ++ks2) {
                        const uint32_t col16 = static_cast<uint32_t>(2 * (ks2 & 1)) + kcol_sel;
                        uint32_t af[4];
                        ldsm_x4(kb0 + (ks2 >> 1) * kBoxBytes + krow * 64 + ((col16 ^ swz) << 4), af[0], af[1], af[2], af[3]);
#pragma unroll
                        for (int nq = 0; nq < NQT; ++nq) {
                            if (ks2 & 1) mma_16816(so[nq], af, qb[ks2][nq][0], qb[ks2][nq][1]);
                            else mma_16816(se[nq], af, qb[ks2][nq][0], qb[ks2][nq][1]);
                        }
                    }
                }
            }
#pragma unroll
            for (int nq = 0; nq < NQT; ++nq)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float f = HALF ? ks * fcol[nq][e & 1] : a.sx;
                    float v = se[nq][e] + so[nq][e];
                    const int kk = 16 * kb + g4 + 8 * (e >> 1);
                    if (MOD && a.cap != 0.f)
                        v = fmaf(-2.f * a.cap, __fdividef(1.f, 1.f + exp2f(v * f)), a.cap + lv);
                    else
                        v = HALF ? fmaf(v, f, lv) : v * f;
                    if (MOD) v = fmaf(slope[nq][e & 1], static_cast<float>(t0 + kk - (dsc.T + jq[nq][e & 1])), v);
                    if (!FAST) {
                        const int j = jq[nq][e & 1];
                        const bool vis = j >= 0 && act[sb] && kk < cnt &&
                                         score_sees(pa, dsc.T, dsc.kind, dsc.plane, t0 + kk, j, pa.jloop[j < 0 ? 0 : j]);
                        v = vis ? v : -INFINITY;
                    }
                    x[sb][nq][e] = v;
                }
        }
        // the reference of a column moves when the warp's maximum exceeds it by more than kScoreHi, which
        // is so exactly when one lane's own maximum does
        bool over = false;
        float mloc[NQT][2];
#pragma unroll
        for (int nq = 0; nq < NQT; ++nq)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float mt = -INFINITY;
#pragma unroll
                for (int sb = 0; sb < C::SB; ++sb) mt = fmaxf(mt, fmaxf(x[sb][nq][e], x[sb][nq][e + 2]));
                mloc[nq][e] = mt;
                over = over || mt > m_ref[nq][e] + kScoreHi;
            }
        if (__any_sync(0xffffffffu, over)) {
#pragma unroll
            for (int nq = 0; nq < NQT; ++nq) {
                float al[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float mt = mloc[nq][e];
                    mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, 4));
                    mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, 8));
                    mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, 16));
                    al[e] = 1.f;
                    if (mt > m_ref[nq][e] + kScoreHi) {
                        al[e] = exp2f(m_ref[nq][e] - (mt - kScoreLo));
                        m_ref[nq][e] = mt - kScoreLo;
                    }
                    l_lse[nq][e] *= al[e];
                    l_out[nq][e] *= al[e];
                }
#pragma unroll
                for (int mt = 0; mt < D / 16; ++mt) {
                    o[mt][nq][0] *= al[0]; o[mt][nq][1] *= al[1];
                    o[mt][nq][2] *= al[0]; o[mt][nq][3] *= al[1];
                }
            }
        }
        float tl[NQT][2];
#pragma unroll
        for (int nq = 0; nq < NQT; ++nq) tl[nq][0] = tl[nq][1] = 0.f;
#pragma unroll
        for (int sb = 0; sb < C::SB; ++sb) {
            if (!act[sb]) continue;
            const int kb = kg * C::SB + sb;
            uint32_t pb[NQT][2];
#pragma unroll
            for (int nq = 0; nq < NQT; ++nq) {
                // no reference yet: every score so far is -inf, or NaN
                const float r0 = m_ref[nq][0] == -INFINITY ? 0.f : m_ref[nq][0];
                const float r1 = m_ref[nq][1] == -INFINITY ? 0.f : m_ref[nq][1];
                const float p0 = exp2f(x[sb][nq][0] - r0), p1 = exp2f(x[sb][nq][1] - r1);
                const float p2 = exp2f(x[sb][nq][2] - r0), p3 = exp2f(x[sb][nq][3] - r1);
                tl[nq][0] += p0 + p2;
                tl[nq][1] += p1 + p3;
                uint32_t lo, hi;
                if constexpr (HALF) {
                    const __half2 l2 = __floats2half2_rn(p0, p1), h2 = __floats2half2_rn(p2, p3);
                    lo = *reinterpret_cast<const uint32_t *>(&l2);
                    hi = *reinterpret_cast<const uint32_t *>(&h2);
                } else {
                    // bf16 rounds to 2^-9: normalise by the rounded values, which is what O sums
                    const __nv_bfloat162 l2 = __floats2bfloat162_rn(p0, p1), h2 = __floats2bfloat162_rn(p2, p3);
                    l_out[nq][0] += __low2float(l2) + __low2float(h2);
                    l_out[nq][1] += __high2float(l2) + __high2float(h2);
                    lo = *reinterpret_cast<const uint32_t *>(&l2);
                    hi = *reinterpret_cast<const uint32_t *>(&h2);
                }
                pb[nq][0] = movmatrix_t(lo);
                pb[nq][1] = movmatrix_t(hi);
            }
            if constexpr (HALF) {
#pragma unroll
                for (int mp = 0; mp < D / 32; ++mp) {
                    const uint4 w = lds128(vb0 + kb * 16 * D + (mp * 32 + lane) * 16);
                    uint32_t af[4];
                    q8_to_f16(w.x, af[0], af[2]);
                    q8_to_f16(w.y, af[1], af[3]);
#pragma unroll
                    for (int nq = 0; nq < NQT; ++nq) mma_16816_f16(o[2 * mp][nq], af, pb[nq][0], pb[nq][1]);
                    q8_to_f16(w.z, af[0], af[2]);
                    q8_to_f16(w.w, af[1], af[3]);
#pragma unroll
                    for (int nq = 0; nq < NQT; ++nq) mma_16816_f16(o[2 * mp + 1][nq], af, pb[nq][0], pb[nq][1]);
                }
            } else {
                const uint32_t vrow = static_cast<uint32_t>(16 * kb) + vrow_off;
                auto v_frag = [&](int mt, uint32_t (&af)[4]) {
                    const uint32_t col16 = static_cast<uint32_t>(2 * (mt & 1)) + vcol_sel;
                    ldsm_x4_t(vb0 + (mt >> 1) * kBoxBytes + vrow * 64 + ((col16 ^ swz) << 4), af[0], af[1], af[2], af[3]);
                };
                bool odd = false;  // a masked tile holding infinities or NaN
                if constexpr (!FAST) {
                    for (int mt = 0; mt < D / 16; ++mt) {
                        uint32_t af[4];
                        v_frag(mt, af);
                        odd = odd || bf16x2_nonfinite(af[0]) || bf16x2_nonfinite(af[1]) || bf16x2_nonfinite(af[2]) ||
                              bf16x2_nonfinite(af[3]);
                    }
                    odd = __any_sync(0xffffffffu, odd);
                }
                if (!odd) {
#pragma unroll
                    for (int mt = 0; mt < D / 16; ++mt) {
                        uint32_t af[4];
                        v_frag(mt, af);
#pragma unroll
                        for (int nq = 0; nq < NQT; ++nq) mma_16816(o[mt][nq], af, pb[nq][0], pb[nq][1]);
                    }
                } else {
                    // 0 * NaN would reach queries that do not see the row: one column at a time, with the
                    // rows that it does not see taken out of V
#pragma unroll
                    for (int nq = 0; nq < NQT; ++nq)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const uint32_t lo = __ballot_sync(0xffffffffu, x[sb][nq][e] != -INFINITY);
                            const uint32_t hi = __ballot_sync(0xffffffffu, x[sb][nq][e + 2] != -INFINITY);
                            for (int cc = 0; cc < 4; ++cc) {  // column 8 nq + 2 cc + e
                                const uint32_t b0 = (lo >> (8 * c4 + cc)) & 1u, b1 = (lo >> (8 * c4 + 4 + cc)) & 1u;
                                const uint32_t b2 = (hi >> (8 * c4 + cc)) & 1u, b3 = (hi >> (8 * c4 + 4 + cc)) & 1u;
                                const uint32_t m01 = b0 * 0xFFFFu + b1 * 0xFFFF0000u;  // keys 2 c4, 2 c4 + 1
                                const uint32_t m23 = b2 * 0xFFFFu + b3 * 0xFFFF0000u;  // and 8 more
#pragma unroll
                                for (int mt = 0; mt < D / 16; ++mt) {
                                    uint32_t af[4];
                                    v_frag(mt, af);
                                    af[0] &= m01; af[1] &= m01; af[2] &= m23; af[3] &= m23;
                                    float t4[4] = {0.f, 0.f, 0.f, 0.f};
                                    mma_16816(t4, af, pb[nq][0], pb[nq][1]);
                                    if (c4 == cc) {
                                        o[mt][nq][e] += t4[e];
                                        o[mt][nq][e + 2] += t4[e + 2];
                                    }
                                }
                            }
                        }
                }
            }
        }
#pragma unroll
        for (int nq = 0; nq < NQT; ++nq)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                if constexpr (HALF) {
                    // 0 * NaN: a column that sees none of a block that reads as NaN takes nothing from it
                    const float s = !FAST && tl[nq][e] == 0.f ? 0.f : tl[nq][e] * iv;
                    l_lse[nq][e] += s;
                    l_out[nq][e] += s;
                } else {
                    l_lse[nq][e] += tl[nq][e];
                }
            }
    };

    const bool ring_all_visible = pa.nloops == 1 && pa.dwin < 0;
    reset_state();
    if (a.early) pdl_wait();  // the caller may be writing the queries
    for (int i = tg; i < ntiles; i += TG) {
        const int s = i % NS;
        if (!mbar_wait_bounded(full0 + 8 * s, (i / NS) & 1)) {
            aborted = true;
            atomicOr(a.err, RIPE_DEVERR_WAIT_TIMEOUT);
            *reinterpret_cast<volatile int *>(&sflag[1]) = 1;
            break;
        }
        const TileDesc dsc = sdesc[s];
        const bool half = Q8 && dsc.kind == kDeep;
        if (dsc.pair != st_pair) {
            if (st_pair >= 0 || fin_next < dsc.pair) {
                while (fin_next < dsc.pair) {
                    finalize(fin_next, st_pair == fin_next);
                    ++fin_next;
                }
                reset_state();
            }
            st_pair = dsc.pair;
            load_q(dsc.n, dsc.kh, half);
        } else if (Q8 && half != st_half) {
            load_q(dsc.n, dsc.kh, half);
        }
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
                        compute(dsc, rb, dsc.t0 + 64 * b, 64, std::true_type(), std::true_type());
                    else
                        compute(dsc, rb, dsc.t0 + 64 * b, 64, std::false_type(), std::true_type());
                }
            }
        }
        if (!half) {
            if (whole && dsc.cnt == kTileRows)
                compute(dsc, base, dsc.t0, dsc.cnt, std::true_type(), std::false_type());
            else
                compute(dsc, base, dsc.t0, dsc.cnt, std::false_type(), std::false_type());
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(empty0 + 8 * s);
    }
    while (fin_next <= P_last) {
        finalize(fin_next, !aborted && st_pair == fin_next);
        ++fin_next;
    }
    named_bar_sync(1, nct);
    if (*reinterpret_cast<volatile int *>(&sflag[1]) == 0) {
        const int nm = sflag[3];
        for (int k = 0; k < nm; ++k) merge_pair(sflag[4 + k]);
    }
}

// ---------------------------------------------------------------- host side
template <int D, int NQT, int WR, int WK, int TG, bool Q8, bool MOD>
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

// Query-side configuration by the query rows per kv head: the one that ripe_verify.cu measured best
// for its tiles (RIPE_QCFG_LIST).
template <int D, bool Q8, bool MOD>
struct ScoreSet {
    using R8 = ScoreInst<D, 1, 1, 4, 2, Q8, MOD>;
    using R16 = ScoreInst<D, 2, 1, 4, 2, Q8, MOD>;
    using R32 = ScoreInst<D, 2, 2, 2, 2, Q8, MOD>;
    using R64 = ScoreInst<D, 2, 4, 2, 1, Q8, MOD>;
    static cudaError_t set_attr() {
        cudaError_t e = R8::set_attr();
        if (e == cudaSuccess) e = R16::set_attr();
        if (e == cudaSuccess) e = R32::set_attr();
        if (e == cudaSuccess) e = R64::set_attr();
        return e;
    }
    static cudaError_t launch(const LaunchTarget &t, int grid, const ScoreArgs &a, cudaStream_t s) {
        if (a.Mq <= 8) return R8::launch(t, grid, a, s);
        if (a.Mq <= 16) return R16::launch(t, grid, a, s);
        if (a.Mq <= 32) return R32::launch(t, grid, a, s);
        return R64::launch(t, grid, a, s);
    }
};

}  // namespace ripe
