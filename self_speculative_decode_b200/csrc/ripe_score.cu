// Launch of the attention over 8-bit caches or with capped or biased scores, and its instances over bf16
// caches.
#include <cfloat>
#include <cmath>

#include "ripe_score_kernel.cuh"

namespace ripe {

constexpr float kLog2e = 1.4426950408889634f;

cudaError_t launch_score_bf16(int d, const LaunchTarget &t, int grid, const ScoreArgs &a, cudaStream_t s) {
    switch (d) {
        case 64: return ScoreSet<64, false, 1>::launch(t, grid, a, s);
        case 96: return ScoreSet<96, false, 1>::launch(t, grid, a, s);
        case 128: return ScoreSet<128, false, 1>::launch(t, grid, a, s);
        default: return cudaErrorInvalidValue;
    }
}

cudaError_t set_score_bf16_attributes() {
    cudaError_t e = ScoreSet<64, false, 1>::set_attr();
    if (e == cudaSuccess) e = ScoreSet<96, false, 1>::set_attr();
    if (e == cudaSuccess) e = ScoreSet<128, false, 1>::set_attr();
    return e;
}

int ensure_score_attributes(int device) {
    if (device < 0 || device >= kMaxDevices) return RIPE_EINVAL;
    static bool done[kMaxDevices] = {};
    static std::mutex mu;
    std::lock_guard<std::mutex> lock(mu);
    if (done[device]) return RIPE_OK;
    cudaError_t e = set_score_q8_attributes();  // the caller makes the device current
    if (e == cudaSuccess) e = set_score_q8_mod_attributes();
    if (e == cudaSuccess) e = set_score_q8_cap_attributes();
    if (e == cudaSuccess) e = set_score_bf16_attributes();
    if (e == cudaSuccess) e = set_score_cap_attributes();
    if (e != cudaSuccess) {
        cudaGetLastError();
        return RIPE_ECUDA;
    }
    done[device] = true;
    return RIPE_OK;
}

float score_factor(const ripe_cache *c, float scale) {
    if (c->softcap > 0.f && c->softcap < FLT_MIN) return NAN;  // the kernels take subnormals for 0
    return c->softcap > 0.f && c->softcap < kCapSeries ? 2.f * scale * kLog2e / c->softcap : scale * kLog2e;
}

int launch_score(ripe_cache *c, const ScoreCall &call, cudaStream_t s) {
    const bool q8 = c->kv_bits == 8;
    ScoreArgs a = {};
    a.q = static_cast<const __nv_bfloat16 *>(call.q);
    a.out = static_cast<__nv_bfloat16 *>(call.out);
    a.lse = call.lse;
    a.T = c->T_dev;
    a.part_o = c->part_o;
    a.part_ml = c->part_ml;
    a.counters = c->counters;
    a.err = c->err_dev;
    a.rec = c->rec8;
    a.rec_blocks = c->rec_blocks;
    a.slopes = c->has_bias ? c->slopes_dev : nullptr;
    ScorePlan &p = a.plan;
    p.W = c->W;
    p.B = call.B;
    p.R = c->R;
    p.S = c->ring_slots;
    p.unit = q8 ? kQ8Block : 1;
    a.Mq = call.qB * c->g;
    a.groups = cdiv(a.Mq, kGroupRows);
    a.grows = cdiv(a.Mq, a.groups);
    const bool wide = q8 && a.grows > 16;
    p.deep_box = c->deep_box;
    p.deep_tile = q8 && !wide ? 2 * kQ8Block : kTileRows;
    p.ring_box = wide && c->ring_box > kWideRingRows ? kWideRingRows : c->ring_box;
    p.ring_cost = score_ring_cost();
    p.head_cost = score_head_cost(q8, a.grows);
    p.crel = c->mode == RIPE_WINDOW_CACHE_RELATIVE ? 1 : 0;
    p.sink = call.sink;
    p.dwin = call.window;
    p.j0 = call.j0;
    bool used[kMaxLoops] = {false};
    for (int j = 0; j < kMaxQueryRows; ++j) {
        const int r = call.loops ? call.loops[j < call.B ? j : 0] : call.r;
        p.jloop[j] = static_cast<uint8_t>(r);
        used[r] = true;
    }
    for (int r = 0; r < c->R; ++r)
        if (used[r]) p.loop[p.nloops++] = static_cast<uint8_t>(r);
    p.all_deepest = p.nloops == 1 && p.loop[0] == c->R - 1 ? 1 : 0;
    a.N = c->N;
    a.kvH = c->kvH;
    a.g = c->g;
    a.Hq = c->Hq;
    a.layer = call.layer;
    a.qB = call.qB;
    a.min_chunk = RIPE_MIN_CHUNK;
    a.has_deep = !q8 && c->deep_rows > 0 ? 1 : 0;
    a.early = c->lengths_dirty ? 0 : 1;
    a.cap = c->softcap * kLog2e;
    a.rcap = c->softcap >= kCapSeries ? 1.f / a.cap : 0.f;
    a.sx = score_factor(c, call.scale);  // finite: checked by the caller
    a.dbg_deep_rows = c->deep_rows;
    // partials of two groups of 32 rows take the room of one of 64 (ripe_cache_alloc's scratch)
    a.dbg_part_slots = c->num_sms + c->N * c->kvH * a.groups;

    // grid: one CTA per SM, fewer when the host copy of T says there is less work
    int grid = c->num_sms < 256 ? c->num_sms : 256;
    if (c->synced) {
        long total = 0;
        for (int n = 0; n < c->N; ++n) total += static_cast<long>(score_geom(c->T[n], p).cost) * c->kvH * a.groups;
        const long need = (total + a.min_chunk - 1) / a.min_chunk;
        if (need < grid) grid = static_cast<int>(need);
    }
    if (grid < 1) grid = 1;
    const LaunchTarget t = {&c->tm_Kd, &c->tm_Vd, wide ? &c->tm_Kw32 : &c->tm_Kw, wide ? &c->tm_Vw32 : &c->tm_Vw,
                            c->device, c->num_sms, c->N};
    const auto launch = a.rcap != 0.f   ? (q8 ? launch_score_q8_cap : launch_score_cap)
                        : !q8           ? launch_score_bf16
                        : c->scored()   ? launch_score_q8_mod
                                        : launch_score_q8;
    const cudaError_t e = launch(c->d, t, grid, a, s);
    c->launches += 1;
    c->lengths_dirty = false;
    return e == cudaSuccess ? RIPE_OK : RIPE_ECUDA;
}

}  // namespace ripe
