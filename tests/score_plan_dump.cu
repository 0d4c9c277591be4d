// Host-only dump of the tile list that the kernels of ripe_score.cu walk for one (sequence, kv head), with the
// plan set up as launch_score sets it up, and of the keys that each query sees in each tile.
// tests/test_score_plan.py compiles it with nvcc; nothing here runs on a GPU.
//
// Input, one case per line:
//   T W R max_T max_B mode unit wide B j0 qB sink window nloops loop_0 .. loop_{nloops-1}
//     queries at block positions j0 .. j0 + qB - 1, position j at loop_{j mod nloops}
// Output per case: "S deep_rows", one line "kind t0 cnt y plane bits_0 .. bits_{qB-1}" per tile (bit i of
// bits_q: query q sees key t0 + i), then "E total".
#include <cstdio>
#include <string>

#include "ripe_score.cuh"

using namespace ripe;

int main(int argc, char **) {
    if (argc > 1) {  // byte offsets inside a record: "d t e k v" lines
        for (int d : {64, 96, 128})
            for (int t = 0; t < 64; ++t)
                for (int e = 0; e < d; ++e)
                    std::printf("%d %d %d %d %d\n", d, t, e, q8_k_offset(t, e, d), q8_v_offset(t, e, d));
        return 0;
    }
    int T, W, R, max_T, max_B, mode, unit, wide, B, j0, qB, sink, window, nloops, loops[kMaxQueryRows];
    while (std::scanf("%d %d %d %d %d %d %d %d %d %d %d %d %d %d", &T, &W, &R, &max_T, &max_B, &mode, &unit, &wide, &B, &j0, &qB,
                      &sink, &window, &nloops) == 14) {
        for (int k = 0; k < nloops; ++k)
            if (std::scanf("%d", &loops[k]) != 1) return 2;
        // cache geometry (ripe_cache_alloc, ripe_cache_alloc_q8)
        const int Wc = W > max_T ? max_T : W;
        const int S = Wc + max_B + unit - 1 < max_T ? Wc + max_B + unit - 1 : max_T;
        const int deep_rows = (max_T - Wc) / unit * unit;
        ScorePlan p = {};
        p.W = Wc;
        p.B = B;
        p.R = R;
        p.S = S;
        p.unit = unit;
        p.deep_box = (deep_rows == 0 || deep_rows >= kTileRows) ? kTileRows : deep_rows;
        p.ring_box = S < kTileRows ? S : kTileRows;
        if (wide && p.ring_box > kWideRingRows) p.ring_box = kWideRingRows;
        p.deep_tile = unit > 1 && !wide ? 2 * kQ8Block : kTileRows;
        p.ring_cost = 2;
        p.head_cost = 2;
        p.crel = mode;
        p.sink = sink;
        p.dwin = window;
        p.j0 = j0;
        bool used[kMaxLoops] = {false};
        for (int j = 0; j < kMaxQueryRows; ++j) {
            const int r = loops[j < B ? j % nloops : 0];
            p.jloop[j] = static_cast<uint8_t>(r);
            used[r] = true;
        }
        for (int r = 0; r < R; ++r)
            if (used[r]) p.loop[p.nloops++] = static_cast<uint8_t>(r);
        p.all_deepest = p.nloops == 1 && p.loop[0] == R - 1 ? 1 : 0;
        const ScoreGeom g = score_geom(T, p);
        std::printf("%d %d\n", S, deep_rows);
        for (int lt = 0; lt < g.total; ++lt) {
            const Tile t = score_tile(g, lt, p);
            std::printf("%d %d %d %d %d", t.kind, t.t0, t.cnt, t.y, t.plane);
            for (int q = 0; q < qB; ++q) {
                std::string bits;
                for (int i = 0; i < t.cnt; ++i)
                    bits += score_sees(p, T, t.kind, t.plane, t.t0 + i, j0 + q, p.jloop[j0 + q]) ? '1' : '0';
                std::printf(" %s", bits.c_str());
            }
            std::printf("\n");
        }
        std::printf("E %d\n", g.total);
    }
    return 0;
}
