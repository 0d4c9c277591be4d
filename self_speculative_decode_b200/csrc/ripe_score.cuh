// Internal definitions of the attention over caches with an 8-bit deepest-plane region, or with
// capped or distance-biased scores (ripe_score.cu, ripe_score_q8.cu), and of that region's layout
// (ripe_q8.cu): the tile plan and the argument block.
#pragma once

#include "ripe_verify.cuh"

namespace ripe {

// ---------------------------------------------------------------- 8-bit deepest-plane region
// 64 tokens of one (layer, sequence, kv head) form a block: K and V as signed 8-bit values with one
// scale each, x = u * s with s = max|x| * (1 / 127).  A block is stored as one record of
// q8_record_bytes(d), copied to shared memory by one bulk copy:
//   K bytes [64 d], V bytes [64 d], {K scale, log2 of the V scale, 1 / V scale, V scale}, 16 bytes pad.
// Bytes hold u + 128 and lie in the order in which the mma.sync m16n8k16 A fragments want them, so a
// lane reads the bytes of two fragments with one conflict-free 16-byte load and no transpose:
//   K  (A = K: rows keys, k = head_dim): per 16 keys and 32 columns, lane (g4, c4) holds for each 16
//      columns the four columns 4 c4 .. 4 c4 + 3 of key g4, then of key g4 + 8 (the order of the
//      columns inside a k-step is free as long as Q follows it);
//   V  (A = V^T: rows head_dim, k = keys): per 16 keys and 32 columns, lane (g4, c4) holds for each 16
//      columns the keys 2 c4, 2 c4 + 1, 2 c4 + 8, 2 c4 + 9 of column g4, then of column g4 + 8.
constexpr int kQ8Block = 64;
constexpr float kQ8MinScale = 8.271806125530277e-25f;  // 2^-80: the smallest scale
constexpr float kQ8MaxScale = 1.2089258196146292e24f;  // 2^80: above it the block reads as NaN

__host__ __device__ constexpr int q8_record_bytes(int d) { return 128 * d + 32; }

// offset of key t (0..63), column e inside the K (or V) half of a record
__host__ __device__ __forceinline__ int q8_k_offset(int t, int e, int d) {
    const int kb = t >> 4, r = t & 15, ks = e >> 4;
    const int lane = (r & 7) * 4 + ((e & 15) >> 2);
    return kb * 16 * d + ((ks >> 1) * 32 + lane) * 16 + (ks & 1) * 8 + (r >> 3) * 4 + (e & 3);
}
__host__ __device__ __forceinline__ int q8_v_offset(int t, int e, int d) {
    const int kb = t >> 4, kk = t & 15, mt = e >> 4, r = e & 15;
    const int lane = (r & 7) * 4 + ((kk & 7) >> 1);
    return kb * 16 * d + ((mt >> 1) * 32 + lane) * 16 + (mt & 1) * 8 + (r >> 3) * 4 + (kk & 1) + 2 * (kk >> 3);
}

// ---------------------------------------------------------------- tile plan
// As in ripe_common.cuh, with a deepest-plane region that ends at a multiple of `unit` positions (1,
// or 64 in the 8-bit region: whole blocks), so that up to unit - 1 positions older than the window
// are still in the ring:
//   DEEP  [0, D), D = floor(max(0, T - W) / unit) * unit, in tiles of deep_tile rows
//   RING  plane r, [lo, T + B) with lo the first key that a query sees at plane r; the only loop
//         being the deepest, [D, T + B), as every key is then read at plane R-1
//   DUAL  plane R-1, [D, hi): keys older than the window of some query of the call
struct ScorePlan {
    int W, B, R, S, unit;
    int deep_box, ring_box;
    int deep_tile;    // rows of a DEEP tile: 64, or 128 (two 8-bit blocks)
    int ring_cost;    // what a RING or DUAL tile costs, in DEEP tiles
    int head_cost;    // what a head costs beside its tiles
    int crel;         // cache-relative window
    int all_deepest;  // a single loop, the deepest one
    int sink, dwin;   // windowed draft (dwin >= 0), as PlanArgs
    int j0;           // first query's block position
    int nloops;
    uint8_t loop[kMaxQueryRows];
    uint8_t jloop[kMaxQueryRows];
};

struct ScoreSeg {  // a range of positions in the ring, cut where the ring wraps
    int p0, len, slot0, first, n1, n;
};

struct ScoreGeom {
    int T, D;
    int e1, b2, nd1, nd;  // DEEP rows [0, e1) in nd1 tiles, then [b2, D)
    ScoreSeg ring, dual;
    int total;
    int cost;  // of the whole list, in DEEP tiles
};

// A masked tile takes about as long as two deepest-plane tiles, and the end of a head (merging the warps' partials, the
// next head's queries) as long as 4 or more, growing with the rows.  Measured on 32 sequences of 10 .. 9000 keys, 8 kv
// heads x 128, at 4 / 16 / 32 / 64 rows a kv head, us:
//   8 bits        59 /  81 / 155 / 295; heads at 4: 59 / 80 / 191 / 383, at 12: 59 /  83 / 134 / 247; masked tiles at 1:
//                 59 /  79 / 173 / 330, at 3: 60 / 82 / 144 / 278
//   bf16, capped  95 / 123 / 165 / 293; heads at 2: 106 / 143 / 191 / 336, at 8: 97 / 107 / 128 / 239; masked tiles at
//                 1: 99 / 143 / 189 / 358, at 3: 96 / 109 / 149 / 247
// (so that from 16 rows over bf16 and from 32 over 8 bits larger values would serve uneven batches better still)
__host__ __device__ constexpr int score_ring_cost() { return 2; }
__host__ __device__ constexpr int score_head_cost(bool q8, int rows) { return q8 && rows > 8 ? 8 : 4; }

// tiles of a box of 32 or 64 rows (ring) by shifts
__host__ __device__ __forceinline__ int score_tiles(int rows, int box) {
    return box == 64 ? (rows + 63) >> 6 : box == 32 ? (rows + 31) >> 5 : cdiv(rows, box);
}

__host__ __device__ __forceinline__ ScoreSeg score_seg(int p0, int len, const ScorePlan &a) {
    ScoreSeg s;
    s.p0 = p0;
    s.len = len > 0 ? len : 0;
    s.slot0 = p0 % a.S;
    s.first = s.len < a.S - s.slot0 ? s.len : a.S - s.slot0;
    s.n1 = score_tiles(s.first, a.ring_box);
    s.n = s.n1 + score_tiles(s.len - s.first, a.ring_box);
    return s;
}

__host__ __device__ __forceinline__ ScoreGeom score_geom(int T, const ScorePlan &a) {
    ScoreGeom s;
    const int A = T - a.W > 0 ? T - a.W : 0;
    const int tr = a.deep_tile;
    s.T = T;
    s.D = a.unit > 1 ? A & ~(kQ8Block - 1) : A;
    s.e1 = s.b2 = 0;
    if (a.dwin >= 0) {
        const int se = a.sink < s.D ? (a.sink + 63) & ~63 : s.D;
        s.e1 = se < s.D ? se : s.D;
        int ws = T + a.j0 - a.dwin;
        ws = ws < 0 ? 0 : ws > s.D ? s.D : ws;
        s.b2 = (ws & ~63) > s.e1 ? ws & ~63 : s.e1;
    }
    s.nd1 = tr == 64 ? (s.e1 + 63) >> 6 : (s.e1 + 127) >> 7;
    s.nd = s.nd1 + (tr == 64 ? (s.D - s.b2 + 63) >> 6 : (s.D - s.b2 + 127) >> 7);
    if (a.all_deepest) {
        s.ring = score_seg(s.D, T + a.B - s.D, a);
        s.dual = score_seg(s.D, 0, a);
    } else {
        int lo = a.crel ? A : T + a.j0 - a.W;
        lo = lo < 0 ? 0 : lo > T ? T : lo;
        int hi = a.crel ? A : T + a.B - 1 - a.W;
        hi = hi < T ? hi : T;
        s.ring = score_seg(lo, T + a.B - lo, a);
        s.dual = score_seg(s.D, hi - s.D, a);
    }
    const int masked = a.nloops * s.ring.n + s.dual.n;
    s.total = s.nd + masked;
    s.cost = s.nd + a.ring_cost * masked + a.head_cost;
    return s;
}

// The lists of all heads are laid end to end on a line of costs and cut into equal chunks; a tile belongs to the
// chunk in which it begins.  score_begin: where tile lt of a head begins; score_first: the first tile of a head that
// begins at or behind offset c (total: none).
__host__ __device__ __forceinline__ int score_begin(const ScoreGeom &s, int lt, const ScorePlan &a) {
    return lt < s.nd ? lt : s.nd + a.ring_cost * (lt - s.nd);
}
__host__ __device__ __forceinline__ int score_first(const ScoreGeom &s, int c, const ScorePlan &a) {
    if (c <= s.nd) return c < 0 ? 0 : c;
    const int lt = s.nd + (c - s.nd + a.ring_cost - 1) / a.ring_cost;
    return lt < s.total ? lt : s.total;
}

__host__ __device__ __forceinline__ Tile score_tile(const ScoreGeom &s, int lt, const ScorePlan &a) {
    Tile t;
    if (lt < s.nd) {
        const int tr = a.deep_tile;
        const bool head = lt < s.nd1;
        t.kind = kDeep;
        t.plane = a.R - 1;
        t.t0 = head ? lt * tr : s.b2 + (lt - s.nd1) * tr;
        const int end = head ? s.e1 : s.D;
        t.cnt = end - t.t0 < tr ? end - t.t0 : tr;
        t.y = t.t0;
        return t;
    }
    lt -= s.nd;
    const ScoreSeg *g = &s.dual;
    t.kind = kDual;
    t.plane = a.R - 1;
    if (lt < a.nloops * s.ring.n) {
        int k = 0;
        while (lt >= s.ring.n) { lt -= s.ring.n; ++k; }
        g = &s.ring;
        t.kind = kRing;
        t.plane = a.loop[k];
    } else {
        lt -= a.nloops * s.ring.n;
    }
    int off, end;
    if (lt < g->n1) {
        off = lt * a.ring_box;
        end = g->first;
        t.y = g->slot0 + off;
    } else {
        off = g->first + (lt - g->n1) * a.ring_box;
        end = g->len;
        t.y = off - g->first;
    }
    t.t0 = g->p0 + off;
    t.cnt = end - off < a.ring_box ? end - off : a.ring_box;
    return t;
}

// The keys [lo, hi) of a tile of this kind and plane that the query of block position jq (loop lq) sees, before
// the tile's own end and a draft window.
__host__ __device__ __forceinline__ void score_range(const ScorePlan &a, int T, int kind, int plane, int jq, int lq,
                                                     int &lo, int &hi) {
    const int p = T + jq;
    lo = 0;
    hi = T;  // deepest-plane rows are all older than every query's window
    if (kind == kRing) {
        hi = lq == plane ? p + 1 : 0;
        if (!a.all_deepest && !a.crel) lo = p - a.W < T ? p - a.W : T;
    } else if (kind == kDual && !a.crel) {
        hi = p - a.W;
    }
}

__host__ __device__ __forceinline__ bool score_sees(const ScorePlan &a, int T, int kind, int plane, int t, int jq,
                                                    int lq) {
    int lo, hi;
    score_range(a, T, kind, plane, jq, lq, lo, hi);
    return t >= lo && t < hi && (a.dwin < 0 || t < a.sink || t >= T + jq - a.dwin);
}

// ---------------------------------------------------------------- arguments of one launch
constexpr int kGroupRows = 32;
// Caps from here on take `capped` (ripe_score_kernel.cuh): below, the exponential form is off by at most 2^-16 (2^-22
// of the cap) and faster (8 sequences x 32768 keys, 32 rows: 194 us against 209, in 8 bits 199 against 212).
constexpr float kCapSeries = 64.f;
constexpr float kCapMost = 1e36f;   // above it 1 / cap nears the end of fp32
constexpr int kWideRingRows = 32;  // ring tile of an 8-bit cache with more than 16 rows: as many bytes as a block

struct ScoreArgs {
    const __nv_bfloat16 *q;
    __nv_bfloat16 *out;
    float *lse;
    const int32_t *T;
    float *part_o, *part_ml;
    int32_t *counters;
    uint32_t *err;
    const uint8_t *rec;   // 8-bit records [L][N][kvH][rec_blocks]
    int rec_blocks;
    const float *slopes;  // [Hq] distance bias per key; nullptr: none
    ScorePlan plan;
    int N, kvH, g, Hq, layer, Mq, min_chunk, qB;
    int groups, grows;    // a kv head's Mq query rows in row groups of grows <= kGroupRows
    int has_deep, early;  // as VerifyArgs
    float sx;             // factor of the dot product: scale * log2(e), or 2 scale log2(e) / cap with a cap below kCapSeries
    float cap;            // cap * log2(e), 0: no cap
    float rcap;           // 1 / cap for a cap from kCapSeries on, else 0
    int dbg_deep_rows, dbg_part_slots;
};

cudaError_t launch_score_q8(int d, const LaunchTarget &t, int grid, const ScoreArgs &a, cudaStream_t s);
cudaError_t launch_score_q8_mod(int d, const LaunchTarget &t, int grid, const ScoreArgs &a, cudaStream_t s);
cudaError_t launch_score_q8_cap(int d, const LaunchTarget &t, int grid, const ScoreArgs &a, cudaStream_t s);
cudaError_t launch_score_cap(int d, const LaunchTarget &t, int grid, const ScoreArgs &a, cudaStream_t s);
cudaError_t launch_score_bf16(int d, const LaunchTarget &t, int grid, const ScoreArgs &a, cudaStream_t s);
cudaError_t set_score_q8_attributes();
cudaError_t set_score_q8_mod_attributes();
cudaError_t set_score_q8_cap_attributes();
cudaError_t set_score_cap_attributes();
cudaError_t set_score_bf16_attributes();

}  // namespace ripe
