// Host-only dump of how the attention over 8-bit caches and with capped or biased scores cuts the heads' tile lists into
// CTAs (ripe_score_kernel.cuh).  tests/test_score_chunks.py compiles it with nvcc; nothing here runs on a GPU.
//
// Input, one case per line: q8 wide rows kvH groups grid W B R max_T max_B loop sink window N T_0 .. T_{N-1}
// (rows: query rows of a row group; loop -1: a loop per position, 0, 1, .. in turn; window >= 0: a draft's last position)
// Output per case: "H total_0 .. total_{N-1}" (tiles of a head), a line "C p_first lt p_last ntiles" per CTA, a line
// "P first count" per head with the CTAs that the kernel takes to hold its tiles, then "E".
#include <cstdio>
#include <vector>

#include "ripe_score_kernel.cuh"

using namespace ripe;

int main() {
    int q8, wide, rows, kvH, groups, grid, W, B, R, max_T, max_B, loop, sink, window, N;
    while (std::scanf("%d %d %d %d %d %d %d %d %d %d %d %d %d %d %d", &q8, &wide, &rows, &kvH, &groups, &grid, &W, &B, &R, &max_T,
                      &max_B, &loop, &sink, &window, &N) == 15) {
        std::vector<int> T(N), cum(N + 1, 0), real(N, 0);
        for (int &t : T)
            if (std::scanf("%d", &t) != 1) return 2;
        ScoreArgs a = {};  // as launch_score fills it
        ScorePlan &p = a.plan;
        const int unit = q8 ? kQ8Block : 1;
        p.W = W < max_T ? W : max_T;
        p.B = B;
        p.R = R;
        p.S = p.W + max_B + unit - 1 < max_T ? p.W + max_B + unit - 1 : max_T;
        p.unit = unit;
        const int deep_rows = (max_T - p.W) / unit * unit;
        p.deep_box = deep_rows == 0 || deep_rows >= kTileRows ? kTileRows : deep_rows;
        p.deep_tile = q8 && !wide ? 2 * kQ8Block : kTileRows;
        p.ring_box = p.S < kTileRows ? p.S : kTileRows;
        if (wide && p.ring_box > kWideRingRows) p.ring_box = kWideRingRows;
        p.ring_cost = score_ring_cost();
        p.head_cost = score_head_cost(q8, rows);
        p.sink = sink;
        p.dwin = window;
        p.j0 = window >= 0 ? B - 1 : 0;
        bool used[kMaxLoops] = {false};
        for (int j = 0; j < kMaxQueryRows; ++j) {
            const int r = loop >= 0 ? loop : (j < B ? j : 0) % R;
            p.jloop[j] = static_cast<uint8_t>(r);
            used[r] = true;
        }
        for (int r = 0; r < R; ++r)
            if (used[r]) p.loop[p.nloops++] = static_cast<uint8_t>(r);
        p.all_deepest = p.nloops == 1 && p.loop[0] == R - 1 ? 1 : 0;
        a.N = N;
        a.kvH = kvH;
        a.groups = groups;
        a.min_chunk = RIPE_MIN_CHUNK;
        const int heads = kvH * groups;
        bool same = true;
        std::printf("H");
        for (int n = 0; n < N; ++n) {
            const ScoreGeom g = score_geom(T[n], p);
            cum[n + 1] = cum[n] + g.cost * heads;
            real[n] = n ? real[n - 1] + score_geom(T[n - 1], p).total * heads : 0;
            same = same && g.cost * heads == cum[1];
            std::printf(" %d", g.total);
        }
        std::printf("\n");
        // fewer CTAs where there is less work, as launch_score
        const int need = (cum[N] + a.min_chunk - 1) / a.min_chunk;
        const int ctas = need < grid ? need : grid;
        const int2 cut = score_cut(a, ctas, cum[N], cum[1] / heads, same, heads);
        ScoreChunk c = {};
        for (int cta = 0; cta < ctas; ++cta) {
            c = ScoreChunk();
            c.chunk = cut.x;
            c.pieces = cut.y;
            if (c.pieces) {
                c.p_first = c.p_last = cta / c.pieces;
                if (c.p_first < N * heads) score_piece(a, score_geom(T[c.p_first / heads], p), cta, c);
            } else {
                score_line(a, cum.data(), real.data(), T.data(), heads, cta, c);
            }
            std::printf("C %d %d %d %d\n", c.p_first, c.lt, c.p_last, c.ntiles);
        }
        for (int h = 0; h < N * heads; ++h) {
            const int2 f = score_parts(a, c, cum.data(), T.data(), heads, h);
            std::printf("P %d %d\n", f.x, f.y);
        }
        std::printf("E\n");
    }
    return 0;
}
