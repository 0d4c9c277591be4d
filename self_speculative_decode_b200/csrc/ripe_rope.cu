// Appending draft-block rows with the position rotation applied on the way, and the entry point over
// caller-owned buffers (declared in include/ripe.h).
//
// Each pair (a, b) of the first rotary_dim elements of a key or query head at position p becomes
// (a cos - b sin, b cos + a sin), with cos and sin of row p of the caller's fp32 tables; products and sums
// in fp32, one rounding to bf16.  Keys go straight to their ring slot (T_n + j) mod S with the values beside
// them, queries to q_out: every element is read once and written once, where a separate rotation would write
// the keys and read them again.  The position comes from the device's length, so that the call works after a
// device-side commit and inside a captured graph.
//
// Bytes bound large calls and launch latency small ones.  A thread holds two vectors of VEC elements (the two
// halves of VEC pairs, or 2 VEC neighbouring elements), which need the same VEC table entries in either
// pairing; one row of a block (a token of a sequence) belongs to one CTA row, whose heads share its table row
// through L1.  Measured: 19.8 us for 512 sequences x 8 tokens of 32 query / 8 kv heads x 128 (103 MB, 0.81 of the
// measured copy bandwidth); blocks of 256 or 384 threads 23.2 us, three items a thread in flight 21.2 us.
#include <cstring>

#include "ripe_common.cuh"

namespace ripe {
namespace {

constexpr int kRopeThreads = 128;

struct RopeArgs {
    const __nv_bfloat16 *k, *v, *q;  // token rows ld_kv / ld_q elements apart; q may be null, or k and v
    __nv_bfloat16 *k_out, *v_out, *q_out;
    const int32_t *T;
    uint32_t *err;
    const float *cos, *sin;  // [positions][rot / 2]
    long long ld_kv, ld_q;
    int positions, rot, interleaved;
    int N, B, j0, Hq, kvH, R, S, layer, r, max_T;
    int ring;   // k_out, v_out are the window ring; otherwise k_out is packed [N][B][kvH][d]
    int early;  // the previous launch on the cache leaves the lengths alone: the next one may start at once
};

template <int VEC>
struct Vec;
template <>
struct Vec<8> { typedef uint4 type; };
template <>
struct Vec<4> { typedef uint2 type; };

template <int VEC>
__device__ __forceinline__ void unpack(const typename Vec<VEC>::type &w, float (&f)[VEC]) {
    const uint32_t *u = reinterpret_cast<const uint32_t *>(&w);
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) {
        f[2 * i] = __uint_as_float(u[i] << 16);
        f[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
    }
}

template <int VEC>
__device__ __forceinline__ typename Vec<VEC>::type pack(const float (&f)[VEC]) {
    typename Vec<VEC>::type w;
    uint32_t *u = reinterpret_cast<uint32_t *>(&w);
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) {
        const __nv_bfloat162 p = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
        u[i] = *reinterpret_cast<const uint32_t *>(&p);
    }
    return w;
}

// grid (N * B, y): CTA row x holds token x % B of sequence x / B, its items spread over y CTAs
template <int D, int VEC>
__global__ void __launch_bounds__(kRopeThreads) ripe_append_rope_kernel(const RopeArgs a) {
    typedef typename Vec<VEC>::type V;
    constexpr int PER = D / (2 * VEC);  // items (pairs of vectors) of a head
    // a verify launch reads nothing this kernel writes before its own wait, but it may read the lengths: it
    // may start at once unless the launch before this one writes them
    if (a.early) pdl_trigger();
    pdl_wait();
    if (!a.early) pdl_trigger();
    const int n = blockIdx.x / a.B, j = blockIdx.x - n * a.B;
    const int Tn = a.T[n], pos = Tn + a.j0 + j;
    // the whole block of a sequence that does not fit is skipped, as in ripe_append_block
    const int most = (a.rot > 0 && a.positions < a.max_T ? a.positions : a.max_T) - a.j0 - a.B;
    if (Tn < 0 || Tn > most) {
        if (threadIdx.x == 0 && blockIdx.y == 0) atomicOr(a.err, RIPE_DEVERR_CAPACITY);
        return;
    }
    const int kheads = a.k ? a.kvH : 0, vheads = a.v ? a.kvH : 0, qheads = a.q ? a.Hq : 0;
    const int items = (kheads + vheads + qheads) * PER;
    const size_t tok = blockIdx.x;
    const size_t half = a.rot / 2;
    for (int it = blockIdx.y * kRopeThreads + threadIdx.x; it < items; it += gridDim.y * kRopeThreads) {
        int h = it / PER;
        const int i = it - h * PER;
        const __nv_bfloat16 *src;
        __nv_bfloat16 *dst;
        bool turn = a.rot > 0;
        if (h < qheads) {
            src = a.q + tok * a.ld_q + static_cast<size_t>(h) * D;
            dst = a.q_out + (tok * a.Hq + h) * D;
        } else {
            h -= qheads;
            const bool is_v = h >= kheads;
            h -= is_v ? kheads : 0;
            turn = turn && !is_v;
            src = (is_v ? a.v : a.k) + tok * a.ld_kv + static_cast<size_t>(h) * D;
            const size_t row = a.ring ? (((static_cast<size_t>(a.layer) * a.N + n) * a.R + a.r) * a.kvH + h) * a.S + pos % a.S
                                      : tok * a.kvH + h;
            dst = (is_v ? a.v_out : a.k_out) + row * D;
        }
        // element offsets of the item's two vectors
        const int pairs = a.rot / (2 * VEC);
        int e0 = 2 * i * VEC, e1 = e0 + VEC;
        turn = turn && i < pairs;
        if (turn && !a.interleaved) {
            e0 = i * VEC;
            e1 = static_cast<int>(half) + e0;
        }
        V x = *reinterpret_cast<const V *>(src + e0), y = *reinterpret_cast<const V *>(src + e1);
        if (turn) {
            float f[VEC], g[VEC], c[VEC], s[VEC];
            unpack<VEC>(x, f);
            unpack<VEC>(y, g);
            const float4 *cp = reinterpret_cast<const float4 *>(a.cos + pos * half + i * VEC);
            const float4 *sp = reinterpret_cast<const float4 *>(a.sin + pos * half + i * VEC);
#pragma unroll
            for (int u = 0; u < VEC / 4; ++u) {
                *reinterpret_cast<float4 *>(&c[4 * u]) = __ldg(cp + u);
                *reinterpret_cast<float4 *>(&s[4 * u]) = __ldg(sp + u);
            }
            if (a.interleaved) {
#pragma unroll
                for (int u = 0; u < VEC / 2; ++u) {
                    const float p = f[2 * u], q = f[2 * u + 1], w = g[2 * u], z = g[2 * u + 1];
                    f[2 * u] = p * c[u] - q * s[u];
                    f[2 * u + 1] = q * c[u] + p * s[u];
                    g[2 * u] = w * c[VEC / 2 + u] - z * s[VEC / 2 + u];
                    g[2 * u + 1] = z * c[VEC / 2 + u] + w * s[VEC / 2 + u];
                }
            } else {
#pragma unroll
                for (int u = 0; u < VEC; ++u) {
                    const float p = f[u], q = g[u];
                    f[u] = p * c[u] - q * s[u];
                    g[u] = q * c[u] + p * s[u];
                }
            }
            x = pack<VEC>(f);
            y = pack<VEC>(g);
        }
        *reinterpret_cast<V *>(dst + e0) = x;
        *reinterpret_cast<V *>(dst + e1) = y;
    }
}

template <int D>
cudaError_t launch_rope_d(const RopeArgs &a, int num_sms, cudaStream_t s) {
    const bool wide = a.rot % 16 == 0;
    const int items = ((a.k ? a.kvH : 0) + (a.v ? a.kvH : 0) + (a.q ? a.Hq : 0)) * (D / (wide ? 16 : 8));
    const int rows = a.N * a.B;
    // few rows: spread each over CTAs until every SM has some
    int y = cdiv(items, kRopeThreads);
    const int most = cdiv(8 * num_sms, rows);
    if (y > most) y = most;
    const dim3 grid(rows, y);
    return wide ? launch_pdl(ripe_append_rope_kernel<D, 8>, grid, dim3(kRopeThreads), 0, s, a)
                : launch_pdl(ripe_append_rope_kernel<D, 4>, grid, dim3(kRopeThreads), 0, s, a);
}

cudaError_t launch_rope_any(int d, const RopeArgs &a, int num_sms, cudaStream_t s) {
    switch (d) {
        case 64: return launch_rope_d<64>(a, num_sms, s);
        case 96: return launch_rope_d<96>(a, num_sms, s);
        case 128: return launch_rope_d<128>(a, num_sms, s);
        default: return cudaErrorInvalidValue;
    }
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

void set_rope(RopeArgs &a, const ripe_rope *rope) {
    a.cos = rope ? rope->cos : nullptr;
    a.sin = rope ? rope->sin : nullptr;
    a.positions = rope ? rope->positions : 0;
    a.rot = rope ? rope->rotary_dim : 0;
    a.interleaved = rope && rope->interleaved ? 1 : 0;
}

}  // namespace

// Everything about the tensors that the host can see; RIPE_OK or RIPE_EINVAL.
int check_rope(const ripe_rope *rope, int d, int Hq, int kvH, int64_t rows, const void *k, const void *v,
               int64_t ld_kv, const void *q, int64_t ld_q, const void *k_out, const void *q_out) {
    if (rope) {
        if (!rope->cos || !rope->sin || rope->positions < 1 || rope->rotary_dim < 8 || rope->rotary_dim > d ||
            rope->rotary_dim % 8 || rope->interleaved < 0 || rope->interleaved > 1 || !aligned16(rope->cos) ||
            !aligned16(rope->sin))
            return RIPE_EINVAL;
    }
    if ((q == nullptr) != (q_out == nullptr)) return RIPE_EINVAL;
    const void *ptrs[] = {k, v, q, k_out, q_out};
    for (const void *p : ptrs)
        if (!aligned16(p)) return RIPE_EINVAL;
    if ((k && (ld_kv < static_cast<int64_t>(kvH) * d || ld_kv % 8)) || (q && (ld_q < static_cast<int64_t>(Hq) * d || ld_q % 8)))
        return RIPE_EINVAL;
    // in place only whole: q_out (k_out) is q (k) itself, packed, or does not touch it
    auto overlaps = [](const void *x, int64_t nx, const void *y, int64_t ny) {
        const char *p = static_cast<const char *>(x), *r = static_cast<const char *>(y);
        return p < r + 2 * ny && r < p + 2 * nx;
    };
    const int64_t span_q = (rows - 1) * ld_q + static_cast<int64_t>(Hq) * d, full_q = rows * Hq * d;
    const int64_t span_k = (rows - 1) * ld_kv + static_cast<int64_t>(kvH) * d, full_k = rows * kvH * d;
    if (q && !(q == q_out && ld_q == static_cast<int64_t>(Hq) * d) && overlaps(q, span_q, q_out, full_q)) return RIPE_EINVAL;
    if (k && k_out && !(k == k_out && ld_kv == static_cast<int64_t>(kvH) * d) && overlaps(k, span_k, k_out, full_k))
        return RIPE_EINVAL;
    if (q && k && overlaps(k, span_k, q_out, full_q)) return RIPE_EINVAL;
    if (q && v && overlaps(v, span_k, q_out, full_q)) return RIPE_EINVAL;
    if (q && k_out && (overlaps(q, span_q, k_out, full_k) || overlaps(q_out, full_q, k_out, full_k))) return RIPE_EINVAL;
    if (rope) {  // the tables are inputs too: fp32, so twice as many elements of two bytes
        const int64_t table = static_cast<int64_t>(rope->positions) * rope->rotary_dim;
        for (const float *t : {rope->cos, rope->sin})
            if ((q && overlaps(t, table, q_out, full_q)) || (k_out && overlaps(t, table, k_out, full_k))) return RIPE_EINVAL;
    }
    return RIPE_OK;
}

// Rows of block positions j0 .. j0 + B - 1 into ring plane r, rotated when rope is given.
int launch_append_rope(ripe_cache *c, int layer, int r, int j0, int B, const void *k, const void *v, int64_t ld_kv,
                       const void *q, int64_t ld_q, void *q_out, const ripe_rope *rope, cudaStream_t s) {
    RopeArgs a = {};
    a.k = static_cast<const __nv_bfloat16 *>(k);
    a.v = static_cast<const __nv_bfloat16 *>(v);
    a.q = static_cast<const __nv_bfloat16 *>(q);
    a.k_out = c->Kw;
    a.v_out = c->Vw;
    a.q_out = static_cast<__nv_bfloat16 *>(q_out);
    a.ring = 1;
    a.ld_kv = ld_kv;
    a.ld_q = ld_q;
    set_rope(a, rope);
    a.T = c->T_dev;
    a.err = c->err_dev;
    a.N = c->N;
    a.B = B;
    a.j0 = j0;
    a.Hq = c->Hq;
    a.kvH = c->kvH;
    a.R = c->R;
    a.S = c->ring_slots;
    a.layer = layer;
    a.r = r;
    a.max_T = c->max_T;
    a.early = c->lengths_dirty ? 0 : 1;
    const cudaError_t e = launch_rope_any(c->d, a, c->num_sms, s);
    c->launches += 1;
    c->lengths_dirty = false;
    return e == cudaSuccess ? RIPE_OK : RIPE_ECUDA;
}

// Rows of block positions j0 .. j0 + B - 1 rotated into k_out and q_out (either may be left out).
int launch_rotate(ripe_cache *c, int j0, int B, const void *k, int64_t ld_k, void *k_out, const void *q, int64_t ld_q,
                  void *q_out, const ripe_rope *rope, cudaStream_t s) {
    RopeArgs a = {};
    a.k = static_cast<const __nv_bfloat16 *>(k);
    a.q = static_cast<const __nv_bfloat16 *>(q);
    a.k_out = static_cast<__nv_bfloat16 *>(k_out);
    a.q_out = static_cast<__nv_bfloat16 *>(q_out);
    a.ld_kv = ld_k;
    a.ld_q = ld_q;
    set_rope(a, rope);
    a.T = c->T_dev;
    a.err = c->err_dev;
    a.N = c->N;
    a.B = B;
    a.j0 = j0;
    a.Hq = c->Hq;
    a.kvH = c->kvH;
    a.S = 1;
    a.max_T = c->max_T;
    // the launch after this one may read what this one writes before waiting only if it is a verify launch,
    // which reads the rotated rows after its wait
    a.early = c->lengths_dirty ? 0 : 1;
    const cudaError_t e = launch_rope_any(c->d, a, c->num_sms, s);
    c->launches += 1;
    c->lengths_dirty = false;
    return e == cudaSuccess ? RIPE_OK : RIPE_ECUDA;
}

}  // namespace ripe

extern "C" int ripe_append_rope_static(const ripe_cache_view *view, int layer, int r, const void *k, const void *v,
                                       int64_t ld_kv, const void *q, int64_t ld_q, void *q_out, const ripe_rope *rope,
                                       uint32_t *device_error, void *stream) {
    using namespace ripe;
    const NvtxRange nvtx_range("ripe_append_rope_static");
    if (!view || !k || !v || !device_error) return RIPE_EINVAL;
    const ripe_cache_view &c = *view;
    const int d = c.head_dim;
    if (c.batch < 1 || c.batch > kMaxBatch || c.layers < 1 || c.q_heads < 1 || c.kv_heads < 1 ||
        c.q_heads % c.kv_heads || (d != 64 && d != 96 && d != 128) || c.loops < 1 || c.loops > kMaxLoops ||
        c.window < 0 || c.max_T < 1 || c.max_B < 1 || c.max_B > kMaxQueryRows || c.max_B > c.max_T ||
        c.max_B * (c.q_heads / c.kv_heads) > kMaxQueryRows || c.block_len < 1 || c.block_len > c.max_B ||
        layer < 0 || layer >= c.layers || r < 0 || r >= c.loops || !c.k_ring || !c.v_ring || !c.lengths || !aligned_to(4, c.lengths, device_error) ||
        !aligned16(c.k_ring) || !aligned16(c.v_ring))
        return RIPE_EINVAL;
    const int64_t rows = static_cast<int64_t>(c.batch) * c.block_len;
    const int st = check_rope(rope, d, c.q_heads, c.kv_heads, rows, k, v, ld_kv, q, ld_q, nullptr, q_out);
    if (st != RIPE_OK) return st;
    int dev = -1, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return RIPE_ECUDA;
    const int W = c.window > c.max_T ? c.max_T : c.window;
    RopeArgs a = {};
    a.k = static_cast<const __nv_bfloat16 *>(k);
    a.v = static_cast<const __nv_bfloat16 *>(v);
    a.q = static_cast<const __nv_bfloat16 *>(q);
    a.k_out = static_cast<__nv_bfloat16 *>(const_cast<void *>(c.k_ring));
    a.v_out = static_cast<__nv_bfloat16 *>(const_cast<void *>(c.v_ring));
    a.q_out = static_cast<__nv_bfloat16 *>(q_out);
    a.ring = 1;
    a.ld_kv = ld_kv;
    a.ld_q = ld_q;
    set_rope(a, rope);
    a.T = c.lengths;
    a.err = device_error;
    a.N = c.batch;
    a.B = c.block_len;
    a.Hq = c.q_heads;
    a.kvH = c.kv_heads;
    a.R = c.loops;
    a.S = static_cast<int64_t>(W) + c.max_B < c.max_T ? W + c.max_B : c.max_T;
    a.layer = layer;
    a.r = r;
    a.max_T = c.max_T;
    a.early = 0;  // the caller's own kernels may write the lengths and buffers
    if (launch_rope_any(d, a, sms, static_cast<cudaStream_t>(stream)) != cudaSuccess) return RIPE_ECUDA;
    return cudaGetLastError() == cudaSuccess ? RIPE_OK : RIPE_ECUDA;
}
