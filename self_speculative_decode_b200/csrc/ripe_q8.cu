// The 8-bit deepest-plane region: quantising blocks of 64 tokens at prefix load and at eviction, and
// reading them back (layout and rule: ripe_score.cuh, include/ripe.h).
//
// A block is quantised once, when its 64 positions have all left the window, from the bf16 rows that
// the ring holds until then: the region's contents depend on the committed positions alone, not on how
// they were split into draft blocks.  Bytes moved bound these kernels (256 d bf16 in, 128 d out per
// block); eviction finds a whole block in one commit of 64 accepted tokens per sequence and head.
// Measured: the prefix of 8 sequences x 32768 positions, 8 heads x 128, with the ring's share 333 us (4.8 TB/s);
// dividing every element and storing bytes took 580 us, four CTAs an SM instead of five 350 us.  A commit that evicts
// a block from each of 14080 heads x 96 178 us (2.9 TB/s), with three CTAs an SM 195 us.
#include "ripe_score.cuh"

namespace ripe {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ size_t ring_row(int layer, int n, int plane, int kh, int slot, int N, int R, int kvH,
                                           int S) {
    return (((static_cast<size_t>(layer) * N + n) * R + plane) * kvH + kh) * S + slot;
}

__device__ __forceinline__ int q8_end(int T, int W) {  // D: positions held in 8 bits
    const int A = T - W > 0 ? T - W : 0;
    return A & ~(kQ8Block - 1);
}

__device__ __forceinline__ float low_bf16(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float high_bf16(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// Bytes u + 128 of four values, u = x / s (rounded to fp32) rounded to nearest even; r = 1 / s.
// x r lies within 2^-16 of x / s (|x / s| < 128, r off by half a step of fp32), so the integer next to x r is
// the wanted one unless x r is within 2^-14 of halfway between two: those are divided.
__device__ __forceinline__ uint32_t quantise4(float x0, float x1, float x2, float x3, float s, float r) {
    constexpr float kMagic = 12582912.f;  // 1.5 * 2^23: x r + kMagic holds the integer in its low bits
    const float x[4] = {x0, x1, x2, x3};
    uint32_t u[4];
    float far = 0.f;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        const float m = __fmaf_rn(x[c], r, kMagic);
        u[c] = __float_as_uint(m);
        far = fmaxf(far, fabsf(__fmaf_rn(x[c], r, kMagic - m)));
    }
    if (far > 0.5f - 0x1p-14f) {
#pragma unroll
        for (int c = 0; c < 4; ++c) u[c] = static_cast<uint32_t>(__float2int_rn(__fdiv_rn(x[c], s)));
    }
    return __byte_perm(__byte_perm(u[0], u[1], 0x0040), __byte_perm(u[2], u[3], 0x0040), 0x5410) ^ 0x80808080u;
}

// One block: row(t) is the row index of its token t in k and v (rows of d bf16); rec its record.
// Scale s = max|x| * (1 / 127) in fp32, at least 2^-80; u = x / s rounded to nearest even.  A block holding an infinity
// or a NaN, or a scale above 2^80, gets a NaN scale: everything that sees it reads NaN.
// A thread holds eight columns of NV rows of K, and of the four rows of V whose bytes share a word of the record: every
// store to buf is a word.
// The whole CTA calls it; buf holds 128 d bytes, red 16 words.
template <int D, class Row>
__device__ __forceinline__ void quantise_block(const uint4 *__restrict__ k, const uint4 *__restrict__ v, Row row,
                                               uint8_t *rec, uint8_t *buf, uint32_t *red) {
    constexpr int D8 = D / 8, NV = 64 * D8 / kThreads;
    static_assert(16 * D8 <= kThreads && NV * kThreads == 64 * D8);
    const int tid = threadIdx.x;
    const bool has_v = tid < 16 * D8;
    const int vg = tid / D8, v8 = tid - vg * D8, vt = 16 * (vg >> 2) + 2 * (vg & 3);  // rows vt, vt + 1, vt + 8, vt + 9
    uint4 xk[NV], xv[4];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int e = tid + i * kThreads, t = e / D8;
        xk[i] = __ldcg(k + row(t) * D8 + (e - t * D8));
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) xv[i] = has_v ? __ldcg(v + row(vt + (i & 1) + 8 * (i >> 1)) * D8 + v8) : make_uint4(0, 0, 0, 0);
    const auto most_of = [](uint32_t m, const uint4 &x) {
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int c = 0; c < 4; ++c) m = max(m, max(w[c] & 0x7FFFu, (w[c] >> 16) & 0x7FFFu));
        return m;
    };
    uint32_t most[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < NV; ++i) most[0] = most_of(most[0], xk[i]);
#pragma unroll
    for (int i = 0; i < 4; ++i) most[1] = most_of(most[1], xv[i]);
#pragma unroll
    for (int h = 0; h < 2; ++h) most[h] = __reduce_max_sync(0xffffffffu, most[h]);
    if ((tid & 31) == 0) {
        red[tid >> 5] = most[0];
        red[8 + (tid >> 5)] = most[1];
    }
    __syncthreads();
    float s[2], r[2];
    bool ok[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = max(m, red[8 * h + i]);
        s[h] = fmaxf(__fmul_rn(__uint_as_float(m << 16), 1.f / 127.f), kQ8MinScale);
        ok[h] = !(m >= 0x7F80u || s[h] > kQ8MaxScale);
        if (!ok[h]) s[h] = __uint_as_float(0x7FC00000u);
        r[h] = __frcp_rn(s[h]);
    }
    if (tid == kThreads - 32) {
        // the kernels weigh V by 2^lv and the normaliser by its reciprocal: taken from the rounded lv, so
        // that the two cancel
        const float lv = static_cast<float>(log2(static_cast<double>(s[1])));
        float4 *tail = reinterpret_cast<float4 *>(rec + 128 * D);
        tail[0] = make_float4(s[0], lv, static_cast<float>(exp2(-static_cast<double>(lv))), s[1]);
        tail[1] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int e = tid + i * kThreads, t = e / D8, c0 = 8 * (e - t * D8);
        const uint32_t w[4] = {xk[i].x, xk[i].y, xk[i].z, xk[i].w};
#pragma unroll
        for (int c = 0; c < 4; c += 2) {
            const uint32_t u = ok[0] ? quantise4(low_bf16(w[c]), high_bf16(w[c]), low_bf16(w[c + 1]),
                                                 high_bf16(w[c + 1]), s[0], r[0])
                                     : 0x80808080u;
            *reinterpret_cast<uint32_t *>(buf + q8_k_offset(t, c0 + 2 * c, D)) = u;
        }
    }
    if (has_v) {
        uint32_t w[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            w[i][0] = xv[i].x;
            w[i][1] = xv[i].y;
            w[i][2] = xv[i].z;
            w[i][3] = xv[i].w;
        }
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            const int p = c >> 1;
            const auto at = [&](int i) { return c & 1 ? high_bf16(w[i][p]) : low_bf16(w[i][p]); };
            const uint32_t u = ok[1] ? quantise4(at(0), at(1), at(2), at(3), s[1], r[1]) : 0x80808080u;
            *reinterpret_cast<uint32_t *>(buf + 64 * D + q8_v_offset(vt, 8 * v8 + c, D)) = u;
        }
    }
    __syncthreads();
    for (int i = tid; i < 128 * D / 16; i += kThreads)
        reinterpret_cast<uint4 *>(rec)[i] = reinterpret_cast<const uint4 *>(buf)[i];
}

template <int D>
__global__ void __launch_bounds__(kThreads, 5)
ripe_q8_load_kernel(uint8_t *__restrict__ rec, const uint4 *__restrict__ k, const uint4 *__restrict__ v,
                    const HostIntArray T, int N, int kvH, int rec_blocks, int W, int layer, int most_blocks,
                    long long ld_t) {
    __shared__ __align__(16) uint8_t buf[128 * D];
    __shared__ uint32_t red[16];
    const int b = blockIdx.x % most_blocks, pair = blockIdx.x / most_blocks;
    const int n = pair / kvH;
    if (b * kQ8Block >= q8_end(T.v[n], W)) return;
    const size_t first = static_cast<size_t>(pair) * ld_t + static_cast<size_t>(b) * kQ8Block;
    quantise_block<D>(k, v, [&](int t) { return first + t; },
                      rec + ((static_cast<size_t>(layer) * N * kvH + pair) * rec_blocks + b) * q8_record_bytes(D), buf,
                      red);
}

// The ring's share of a prefix plane: the deepest plane from D on, the others from T - W on.
__global__ void ripe_q8_load_ring_kernel(uint4 *__restrict__ Kw, uint4 *__restrict__ Vw, const uint4 *__restrict__ k,
                                         const uint4 *__restrict__ v, int32_t *T_dev, const HostIntArray T, int N,
                                         int kvH, int d8, int R, int S, int W, int layer, int plane, int rows,
                                         long long ld_t) {
    if (blockIdx.x == 0)
        for (int n = threadIdx.x; n < N; n += blockDim.x) T_dev[n] = T.v[n];
    const size_t total = static_cast<size_t>(N) * kvH * rows * d8;
    for (size_t idx = blockIdx.x * static_cast<size_t>(blockDim.x) + threadIdx.x; idx < total;
         idx += static_cast<size_t>(gridDim.x) * blockDim.x) {
        const int c8 = static_cast<int>(idx % d8);
        size_t rest = idx / d8;
        const int i = static_cast<int>(rest % rows);
        rest /= rows;
        const int kh = static_cast<int>(rest % kvH), n = static_cast<int>(rest / kvH);
        const int Tn = T.v[n];
        const int A = Tn - W > 0 ? Tn - W : 0;
        const int t = (plane == R - 1 ? A & ~(kQ8Block - 1) : A) + i;
        if (t >= Tn) continue;
        const size_t src = ((static_cast<size_t>(n) * kvH + kh) * ld_t + t) * d8 + c8;
        const size_t dst = ring_row(layer, n, plane, kh, t % S, N, R, kvH, S) * d8 + c8;
        Kw[dst] = k[src];
        Vw[dst] = v[src];
    }
}

// At a commit: the block whose last position leaves the window, if any (an accepted length of at most 64
// completes at most one), from ring plane R-1.
template <int D>
__global__ void __launch_bounds__(kThreads, 4)
ripe_q8_evict_kernel(uint8_t *__restrict__ rec, const uint4 *__restrict__ Kw, const uint4 *__restrict__ Vw,
                     const int32_t *T, const HostIntArray acc_h, const int32_t *acc_d, int L, int N,
                     int B, int kvH, int R, int S, int W, int rec_blocks, int max_T) {
    __shared__ __align__(16) uint8_t buf[128 * D];
    __shared__ uint32_t red[16];
    pdl_wait();
    pdl_trigger();
    const int items = L * N * kvH;
    for (int it = blockIdx.x; it < items; it += gridDim.x) {
        const int kh = it % kvH, n = (it / kvH) % N, layer = it / kvH / N;
        const int Tn = T[n], p0 = q8_end(Tn, W);
        const int a = accepted(acc_h, acc_d, n, B, Tn, max_T, nullptr);  // (the length update reports)
        if (q8_end(Tn + a, W) == p0 || p0 / kQ8Block >= rec_blocks) continue;
        const size_t row0 = ring_row(layer, n, R - 1, kh, 0, N, R, kvH, S);
        quantise_block<D>(Kw, Vw, [&](int t) { return row0 + (p0 + t) % S; },
                          rec + (static_cast<size_t>(it) * rec_blocks + p0 / kQ8Block) * q8_record_bytes(D), buf, red);
        __syncthreads();  // buf and red are used again
    }
}

// One sequence's blocks as 8-bit values [kvH][D][d] and scales [kvH][D / 64].
__global__ void ripe_q8_export_kernel(const uint8_t *__restrict__ rec, int8_t *__restrict__ k, int8_t *__restrict__ v,
                                      float *__restrict__ ks, float *__restrict__ vs, size_t pair0, int kvH,
                                      int rec_blocks, int blocks, int d) {
    const int kh = blockIdx.x / blocks, b = blockIdx.x % blocks;
    const uint8_t *r = rec + ((pair0 + kh) * rec_blocks + b) * q8_record_bytes(d);
    const size_t out = static_cast<size_t>(blockIdx.x) * 64 * d;
    for (int i = threadIdx.x; i < 64 * d; i += blockDim.x) {
        const int t = i / d, e = i - t * d;
        k[out + i] = static_cast<int8_t>(r[q8_k_offset(t, e, d)] - 128);
        v[out + i] = static_cast<int8_t>(r[64 * d + q8_v_offset(t, e, d)] - 128);
    }
    if (threadIdx.x == 0) {
        const float4 s = *reinterpret_cast<const float4 *>(r + 128 * d);
        ks[blockIdx.x] = s.x;
        vs[blockIdx.x] = s.w;
    }
}

struct PlaneMask8 {
    uint8_t v[kMaxLoops];
};

// The logical view (ripe_cache_export): positions of the 8-bit region as u * s rounded to bf16.
__global__ void ripe_q8_view_kernel(const uint8_t *__restrict__ rec, const __nv_bfloat16 *__restrict__ Kw,
                                    const __nv_bfloat16 *__restrict__ Vw, const int32_t *__restrict__ T_dev,
                                    __nv_bfloat16 *__restrict__ ko, __nv_bfloat16 *__restrict__ vo, uint8_t *present,
                                    const PlaneMask8 app, int n, int layer, int Tv, int Bcur, int N, int kvH, int d,
                                    int R, int S, int W, int rec_blocks) {
    const int Tn = T_dev[n], Dn = q8_end(Tn, W);
    const size_t total = static_cast<size_t>(R) * kvH * Tv * d;
    for (size_t idx = blockIdx.x * static_cast<size_t>(blockDim.x) + threadIdx.x; idx < total;
         idx += static_cast<size_t>(gridDim.x) * blockDim.x) {
        const int e = static_cast<int>(idx % d);
        size_t rest = idx / d;
        const int t = static_cast<int>(rest % Tv);
        rest /= Tv;
        const int kh = static_cast<int>(rest % kvH), plane = static_cast<int>(rest / kvH);
        const bool pres = t < Tn ? plane == R - 1 || t >= Tn - W : t < Tn + Bcur && app.v[plane];
        __nv_bfloat16 kx = __float2bfloat16(0.f), vx = kx;
        if (pres && t < Dn && t < Tn - W) {
            const uint8_t *r = rec + (((static_cast<size_t>(layer) * N + n) * kvH + kh) * rec_blocks + t / kQ8Block) *
                                         q8_record_bytes(d);
            const float4 s = *reinterpret_cast<const float4 *>(r + 128 * d);
            kx = __float2bfloat16((r[q8_k_offset(t % kQ8Block, e, d)] - 128) * s.x);
            vx = __float2bfloat16((r[64 * d + q8_v_offset(t % kQ8Block, e, d)] - 128) * s.w);
        } else if (pres) {
            const size_t src = ring_row(layer, n, plane, kh, t % S, N, R, kvH, S) * d + e;
            kx = Kw[src];
            vx = Vw[src];
        }
        ko[idx] = kx;
        vo[idx] = vx;
        if (kh == 0 && e == 0) present[static_cast<size_t>(plane) * Tv + t] = pres ? 1 : 0;
    }
}

// Debug builds, after a commit: ring slots without a live position get the largest finite bf16, blocks that
// are not filled yet NaN scales.
__global__ void ripe_q8_poison_kernel(uint8_t *__restrict__ rec, uint4 *__restrict__ Kw, uint4 *__restrict__ Vw,
                                      const int32_t *__restrict__ T, int L, int N, int R, int kvH, int d8, int S, int W,
                                      int rec_blocks) {
    const uint32_t pw = kPoisonByte * 0x01010101u;
    const uint4 poison = make_uint4(pw, pw, pw, pw), ones = make_uint4(~0u, ~0u, ~0u, ~0u);
    const size_t ring_vecs = static_cast<size_t>(L) * N * R * kvH * S * d8;
    const size_t rec_vecs = static_cast<size_t>(q8_record_bytes(8 * d8)) / 16;
    const size_t all = ring_vecs + static_cast<size_t>(L) * N * kvH * rec_blocks * rec_vecs;
    for (size_t idx = blockIdx.x * static_cast<size_t>(blockDim.x) + threadIdx.x; idx < all;
         idx += static_cast<size_t>(gridDim.x) * blockDim.x) {
        if (idx < ring_vecs) {
            const size_t row = idx / d8;
            const int slot = static_cast<int>(row % S), plane = static_cast<int>(row / S / kvH % R);
            const int Tn = T[row / S / kvH / R % N];
            const int lo = plane == R - 1 ? q8_end(Tn, W) : (Tn - W > 0 ? Tn - W : 0);
            const int off = ((slot - lo % S) + S) % S;  // slot of position lo + off
            if (off < Tn - lo) continue;
            Kw[idx] = poison;
            Vw[idx] = poison;
        } else {
            const size_t b = (idx - ring_vecs) / rec_vecs;
            const int n = static_cast<int>(b / rec_blocks / kvH % N);
            if (static_cast<int>(b % rec_blocks) < q8_end(T[n], W) / kQ8Block) continue;
            reinterpret_cast<uint4 *>(rec)[idx - ring_vecs] = ones;
        }
    }
}

template <class F>
int by_head_dim(int d, F f) {
    switch (d) {
        case 64: f(std::integral_constant<int, 64>()); break;
        case 96: f(std::integral_constant<int, 96>()); break;
        case 128: f(std::integral_constant<int, 128>()); break;
        default: return RIPE_EINVAL;
    }
    return cudaGetLastError() == cudaSuccess ? RIPE_OK : RIPE_ECUDA;
}

int blocks_for(size_t work, int cap) {
    const size_t b = (work + 255) / 256;
    return b < 1 ? 1 : b > static_cast<size_t>(cap) ? cap : static_cast<int>(b);
}

}  // namespace

int launch_q8_load_prefix(ripe_cache *c, int layer, int plane, const int32_t *T, const void *k, const void *v,
                          int64_t ld_t, cudaStream_t s) {
    HostIntArray th;
    int most = 0, rows = 1;
    for (int n = 0; n < c->N; ++n) {
        th.v[n] = T[n];
        const int A = T[n] > c->W ? T[n] - c->W : 0, D = A & ~(kQ8Block - 1);
        most = D / kQ8Block > most ? D / kQ8Block : most;
        rows = T[n] - D > rows ? T[n] - D : rows;
    }
    const int d8 = c->d / 8;
    ripe_q8_load_ring_kernel<<<blocks_for(static_cast<size_t>(c->N) * c->kvH * rows * d8, 8 * c->num_sms), 256, 0, s>>>(
        reinterpret_cast<uint4 *>(c->Kw), reinterpret_cast<uint4 *>(c->Vw), static_cast<const uint4 *>(k),
        static_cast<const uint4 *>(v), c->T_dev, th, c->N, c->kvH, d8, c->R, c->ring_slots, c->W, layer, plane, rows,
        static_cast<long long>(ld_t));
    c->launches += 1;
    c->lengths_dirty = true;
    if (cudaGetLastError() != cudaSuccess) return RIPE_ECUDA;
    if (plane != c->R - 1 || most == 0) return RIPE_OK;
    c->launches += 1;
    return by_head_dim(c->d, [&](auto d) {
        ripe_q8_load_kernel<decltype(d)::value><<<c->N * c->kvH * most, kThreads, 0, s>>>(
            c->rec8, static_cast<const uint4 *>(k), static_cast<const uint4 *>(v), th, c->N, c->kvH, c->rec_blocks,
            c->W, layer, most, static_cast<long long>(ld_t));
    });
}

int launch_q8_evict(ripe_cache *c, const HostIntArray &acc_host, const int32_t *acc_dev, cudaStream_t s) {
    if (c->rec_blocks == 0) return RIPE_OK;
    const int items = c->L * c->N * c->kvH;
    const int grid = items < 4 * c->num_sms ? items : 4 * c->num_sms;
    c->launches += 1;
    return by_head_dim(c->d, [&](auto d) {
        launch_pdl(ripe_q8_evict_kernel<decltype(d)::value>, dim3(grid), dim3(kThreads), 0, s, c->rec8,
                   reinterpret_cast<const uint4 *>(c->Kw), reinterpret_cast<const uint4 *>(c->Vw),
                   static_cast<const int32_t *>(c->T_dev), acc_host, acc_dev, c->L, c->N, c->B_cur, c->kvH, c->R,
                   c->ring_slots, c->W, c->rec_blocks, c->max_T);
    });
}

int launch_q8_export(ripe_cache *c, int n, int layer, int8_t *k, int8_t *v, float *ks, float *vs, cudaStream_t s) {
    const int A = c->T[n] > c->W ? c->T[n] - c->W : 0, blocks = A / kQ8Block;
    if (blocks == 0) return RIPE_OK;
    ripe_q8_export_kernel<<<c->kvH * blocks, 256, 0, s>>>(
        c->rec8, k, v, ks, vs, (static_cast<size_t>(layer) * c->N + n) * c->kvH, c->kvH, c->rec_blocks, blocks, c->d);
    c->launches += 1;
    return cudaGetLastError() == cudaSuccess ? RIPE_OK : RIPE_ECUDA;
}

int launch_q8_view(ripe_cache *c, int n, int layer, void *k_out, void *v_out, uint8_t *present, cudaStream_t s) {
    PlaneMask8 app;
    for (int p = 0; p < kMaxLoops; ++p) app.v[p] = p < c->R ? c->appended[static_cast<size_t>(layer) * c->R + p] : 0;
    const int Tv = c->T[n] + c->B_cur;
    if (Tv == 0) return RIPE_OK;
    ripe_q8_view_kernel<<<blocks_for(static_cast<size_t>(c->R) * c->kvH * Tv * c->d, 8 * c->num_sms), 256, 0, s>>>(
        c->rec8, c->Kw, c->Vw, c->T_dev, static_cast<__nv_bfloat16 *>(k_out), static_cast<__nv_bfloat16 *>(v_out),
        present, app, n, layer, Tv, c->B_cur, c->N, c->kvH, c->d, c->R, c->ring_slots, c->W, c->rec_blocks);
    c->launches += 1;
    return cudaGetLastError() == cudaSuccess ? RIPE_OK : RIPE_ECUDA;
}

int launch_q8_poison(ripe_cache *c, cudaStream_t s) {
    const size_t vecs = static_cast<size_t>(c->L) * c->N * c->kvH *
                        (static_cast<size_t>(c->R) * c->ring_slots * (c->d / 8) +
                         static_cast<size_t>(c->rec_blocks) * q8_record_bytes(c->d) / 16);
    ripe_q8_poison_kernel<<<blocks_for(vecs, 8 * c->num_sms), 256, 0, s>>>(
        c->rec8, reinterpret_cast<uint4 *>(c->Kw), reinterpret_cast<uint4 *>(c->Vw), c->T_dev, c->L, c->N, c->R,
        c->kvH, c->d / 8, c->ring_slots, c->W, c->rec_blocks);
    c->launches += 1;
    return cudaGetLastError() == cudaSuccess ? RIPE_OK : RIPE_ECUDA;
}

}  // namespace ripe
