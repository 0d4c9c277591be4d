"""Attention over 8-bit caches and with capped or biased scores at the ends of its range, against 64 bits."""
import numpy as np
import pytest
import torch

from self_speculative_decode_b200 import ripe, synth
from score_ref import Pair, bits_dev, quantised

pytestmark = pytest.mark.gpu


def dense(p, q, n, j, cap=0.0, slopes=None):
    """out [Hq][d], its tolerance, lse [Hq], its own, of query row q [Hq][d] (bf16 bits) at position T_n + j, over a cache
    with one plane (R = 1), the deepest one for every key.

    Tolerances as score_ref's: eps is the error of a score, and what the cap adds to it 2^-21 of a cap below 64, 2^-19 of
    the score from 64 on (csrc/ripe_score_kernel.cuh).  The largest p' (a weight times its block's V
    scale) is at least 2^7, the reference being 2^-7 of the maximum, and f16 holds each of them to 2^-25 absolute: a
    key's p' u is off by up to 2^-32 of the largest value."""
    end, D = p.T[n] + j + 1, p.D(n)
    kv = []
    for w in range(2):
        x = synth.bf16_bits_to_f32(p.planes[0][0][w][n][:, :end]).astype(np.float64)
        if p.bits == 8 and D:
            u, s = quantised(x[:, :D])
            x[:, :D] = u.astype(np.float64) * np.repeat(s.astype(np.float64), 64, 1)[:, :, None]
        kv.append(np.repeat(x, p.g, 0))
    qf = synth.bf16_bits_to_f32(q).astype(np.float64)
    x = p.scale * np.einsum("hd,htd->ht", qf, kv[0])
    eps = p.d * 2.0 ** -23 * abs(p.scale) * np.einsum("hd,htd->ht", abs(qf), abs(kv[0])).max(1)
    if cap:
        x = cap * np.tanh(x / cap)
        eps = eps + (2.0 ** -21 * cap if cap < 64 else 2.0 ** -19 * abs(x).max(1))
    if slopes is not None:
        x = x - np.asarray(slopes, np.float64)[:, None] * (end - 1 - np.arange(end))
    eps = eps + 2.0 ** -21 * abs(x).max(1)
    m = x.max(1, keepdims=True)
    w = np.exp(x - m)
    lse = m[:, 0] + np.log(w.sum(1))
    w /= w.sum(1, keepdims=True)
    out = np.einsum("ht,htd->hd", w, kv[1])
    A, B = np.einsum("ht,htd->hd", w, abs(kv[1] - out[:, None])), np.einsum("ht,htd->hd", w, abs(kv[1]))
    tol = 2.0 ** -8 * (abs(out) + A) + (2.0 ** -11 + 2 * eps[:, None] + 2.0 ** -18) * B \
        + 2.0 ** -32 * end * abs(kv[1]).max()
    return out, tol, lse, eps + 2.0 ** -18 + 2.0 ** -22 * abs(lse)


def check(p, out, lse, q, **kw):
    got, gl = out.double().cpu().numpy(), lse.double().cpu().numpy()
    for n in range(p.N):
        for j in range(q.shape[1]):
            eo, to, el, tl = dense(p, q[n, j], n, j, **kw)
            assert (abs(got[n, j] - eo) <= to).all(), (n, j, float((abs(got[n, j] - eo) / to).max()))
            assert (abs(gl[n, j] - el) <= tl).all(), (n, j, float((abs(gl[n, j] - el) / tl).max()))


@pytest.mark.parametrize("bits", [8, 16])
def test_first_slopes_set_on_a_side_stream(cuda_device, bits):
    """Work queued on the default stream comes between the allocation of the slopes and their use on another one."""
    p = Pair(2, 4, 2, 64, 2, 8, [200, 131], 3, bits=bits, seed=5).load().append(3)
    p.slopes = [0.5, 0.125, 0.3, 1.0]
    q, lse = p.queries(3), p.lse(3)
    qd = bits_dev(q)
    out = torch.empty_like(qd)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)  # about a tenth of a second
    p.gpu.set_scores(0.0, p.slopes, stream=s)
    p.gpu.verify_attn(0, 0, qd, out=out, lse=lse, stream=s)
    s.synchronize()
    p.check(out, lse, q, 0)
    torch.cuda.synchronize()  # the default stream has run dry
    out.zero_()
    torch.cuda.synchronize()
    p.gpu.verify_attn(0, 0, qd, out=out, lse=lse, stream=s)
    s.synchronize()
    p.check(out, lse, q, 0)
    p.close()


@pytest.mark.parametrize("bits", [8, 16])
def test_a_step_replayed_past_the_capacity(cuda_device, bits):
    """A captured step knows no host lengths: a block that no longer fits is reported, none of it is accepted, and the
    lengths stay within the cache, whose other sequence and earlier positions are as they should be."""
    p = Pair(2, 4, 2, 64, 2, 8, [50, 150], 4, bits=bits, cap=20.0, room=6, seed=18).load()
    kv = [[torch.empty((2, 4, 2, 64), dtype=torch.bfloat16, device="cuda") for _ in range(2)] for _ in range(2)]
    q = torch.empty((2, 4, 4, 64), dtype=torch.bfloat16, device="cuda")
    out, lse = torch.empty_like(q), p.lse(4)
    acc = torch.full((2,), 4, dtype=torch.int32, device="cuda")

    def step():
        for r in range(2):
            p.gpu.append_block(0, r, *kv[r])
        p.gpu.verify_attn(0, 0, q, out=out, lse=lse)
        p.gpu.commit_device(acc)

    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for i in range(5):  # 150 -> 154 -> 158, and 158 + 4 > 160
        T = list(p.T)
        p.T = [min(t, p.max_T - 4) for t in T]
        qb = p.queries(4)
        q.copy_(bits_dev(qb))
        for r in range(2):
            for dst, src in zip(kv[r], p.rows(0, r, 0, 4)):
                dst.copy_(bits_dev(src))
        p.T = T
        g.replay()
        torch.cuda.synchronize()
        p.check(out, lse, qb, 0, rows={(0, j) for j in range(4)} | ({(1, j) for j in range(4)} if i < 2 else set()))
        p.T = [T[0] + 4, T[1] + (4 if i < 2 else 0)]
    assert p.gpu.device_error() == ripe.RIPE_DEVERR_CAPACITY
    assert p.gpu.sync_lengths() == p.T == [70, 158]
    p.append(2).verify(0, 2)
    p.verify(1, 2)
    p.close()


@pytest.mark.parametrize("bits,Hq,B", [(16, 6, 5), (16, 6, 8), (8, 6, 5), (8, 6, 8)])
def test_calls_behind_a_rotation_in_place_read_what_it_wrote(cuda_device, bits, Hq, B):
    """Rotation, append and verification of several steps queued without a pause give what they give one at a time."""
    N, kvH, d, W = 9, 2, 96, 16
    c = ripe.RipeCache(N, 1, Hq, kvH, d, 2, W, 400, B, kv_bits=bits)
    kv = torch.randn((N, kvH, 300, d), device="cuda").bfloat16()
    for r in range(2):
        c.load_prefix(0, r, [300 - 20 * n for n in range(N)], kv, kv)
    angle = torch.arange(400, device="cuda")[:, None] * 0.01 ** (torch.arange(48, device="cuda") / 48)
    t = ripe.RotaryTable(angle.cos(), angle.sin())
    steps = [[torch.randn((N, B, h, d), device="cuda").bfloat16() for h in (Hq, kvH, kvH)] for _ in range(30)]

    def run(pause):
        out = []
        for i, (q, k, v) in enumerate(steps):
            q, k = q.clone(), k.clone()
            pause()
            if i % 2:
                c.append_block_rope(0, 0, k, v, t, q, q_out=q)
            else:
                c.rotate_block(0, t, k, q, k_out=k, q_out=q)
                pause()
                c.append_block(0, 0, k, v)
            pause()
            out.append(c.verify_attn(0, 0, q))
        return out

    run(lambda: None)
    want = run(torch.cuda.synchronize)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(run(lambda: None), want))
    assert c.device_error() == 0
    c.close()


# ------------------------------------------------------------------ NaN in one part of a split head
# 1 head, 700 keys: the list of tiles is cut into two to four pieces, the first of which hold nothing but NaN.  Query rows
# 2..64 cover the kernel's shapes; with q_std 60 the other keys' maximum lies above 2^126 times the first pieces'
# reference.
@pytest.mark.parametrize("q_std,nan", [(1.0, 128), (1.0, 256), (1.0, 384), (60.0, 256), (60.0, 448)])
@pytest.mark.parametrize("bits", [8, 16])
@pytest.mark.parametrize("w", [0, 1])
@pytest.mark.parametrize("Hq,B", [(2, 1), (4, 4), (8, 3), (8, 4), (8, 8)])
def test_a_part_of_a_head_that_is_all_nan(cuda_device, q_std, nan, bits, w, Hq, B):
    p = Pair(1, Hq, 1, 64, 1, 8, 700, B, bits=bits, cap=1000.0 if bits == 16 else 0.0, seed=3, q_std=q_std)
    p.planes[0][0][w][0, :, :nan] = 0x7FC0
    p.load().append(B)
    lse = p.lse(B)
    out = p.gpu.verify_attn(0, 0, bits_dev(p.queries(B)), lse=lse)
    assert out.isnan().all()
    if w == 0:
        assert lse.isnan().all()
    elif bits == 16:  # a value moves no score
        assert lse.isfinite().all()
    p.close()


@pytest.mark.parametrize("bits", [8, 16])
@pytest.mark.parametrize("T", [20, 700, 3000])
@pytest.mark.parametrize("Hq,B", [(2, 1), (4, 4), (8, 3), (8, 8)])
def test_a_query_with_nan_has_a_nan_log_sum_exp(cuda_device, bits, T, Hq, B):
    p = Pair(1, Hq, 1, 64, 1, 8, T, B, bits=bits, cap=25.0, seed=13).load().append(B)
    qb = p.queries(B)
    qb[0, B - 1, 1, 3] = 0x7FC0
    lse = p.lse(B)
    out = p.gpu.verify_attn(0, 0, bits_dev(qb), lse=lse)
    bad = torch.zeros((1, B, Hq), dtype=torch.bool, device="cuda")
    bad[0, B - 1, 1] = True
    assert out[bad].isnan().all() and lse[bad].isnan().all()
    assert out[~bad].isfinite().all() and lse[~bad].isfinite().all()
    p.close()


# ------------------------------------------------------------------ refused calls
@pytest.mark.parametrize("bits,cap", [(8, 0.0), (8, 30.0), (16, 30.0)])
def test_a_refused_call_leaves_the_cache_as_it_was(cuda_device, bits, cap):
    """A scale that no score survives is refused before the block's or the draft's rows are written."""
    p = Pair(2, 4, 2, 64, 2, 8, [100, 200], 3, bits=bits, cap=cap, seed=17).load()
    junk = torch.full((2, 3, 2, 64), 9.0, dtype=torch.bfloat16, device="cuda")
    p.draft(0, 0)
    q1 = bits_dev(p.queries(1))
    for scale in (float("inf"), float("nan")):
        with pytest.raises(ripe.RipeError) as e:  # the drafted row again
            p.gpu.draft_attn(0, 0, 0, junk[:, :1].contiguous(), junk[:, :1].contiguous(), q1, scale=scale)
        assert e.value.status == ripe.RIPE_EINVAL
    p.draft(0, 1)  # attends to the row drafted first
    p.append(3)
    before = p.gpu.export(0, 0) + p.gpu.export(1, 0)
    launches = p.gpu.launch_count()
    q = bits_dev(p.queries(3))
    for scale in (float("inf"), float("nan")):
        for call in (lambda: p.gpu.append_verify(0, 1, junk, junk, q, scale=scale),
                     lambda: p.gpu.verify_attn(0, 1, q, scale=scale),
                     lambda: p.gpu.verify_attn_wave(0, [0, 1, 0], q, scale=scale)):
            with pytest.raises(ripe.RipeError) as e:
                call()
            assert e.value.status == ripe.RIPE_EINVAL
    assert p.gpu.launch_count() == launches
    assert all(torch.equal(a, b) for a, b in zip(before, p.gpu.export(0, 0) + p.gpu.export(1, 0)))
    p.verify(1, 3)
    p.close()


# ------------------------------------------------------------------ caps far above the scores
@pytest.mark.parametrize("bits", [8, 16])
@pytest.mark.parametrize("Hq,B", [(2, 1), (4, 4), (8, 4)])
@pytest.mark.parametrize("cap", [63.0, 64.0, 100.0, 1e3, 1e5, 1e7, 1e12, 1e30, 1e36])
def test_large_caps(cuda_device, bits, Hq, B, cap):
    p = Pair(2, Hq, 1, 64, 1, 8, [300, 90], B, bits=bits, seed=23, q_std=8.0).load().append(B)
    p.gpu.set_scores(cap)
    qb, lse = p.queries(B), p.lse(B)
    out = p.gpu.verify_attn(0, 0, bits_dev(qb), lse=lse)
    check(p, out, lse, qb, cap=cap)
    p.close()


@pytest.mark.parametrize("scale,cap", [(30.0, 2000.0), (300.0, 2000.0), (-2.0, 100.0), (0.0, 1e6)])
def test_scores_around_a_large_cap(cuda_device, scale, cap):
    """Scores on both sides of the kernel's two forms, up to far beyond the cap."""
    for bits in (8, 16):
        p = Pair(1, 4, 2, 64, 1, 8, 200, 3, bits=bits, seed=24, q_std=8.0, scale=scale).load().append(3)
        p.gpu.set_scores(cap)
        qb, lse = p.queries(3), p.lse(3)
        out = p.gpu.verify_attn(0, 0, bits_dev(qb), lse=lse, scale=scale)
        check(p, out, lse, qb, cap=cap)
        p.close()


def test_caps_that_fp32_cannot_hold_are_refused(cuda_device):
    p = Pair(1, 2, 2, 64, 1, 8, 100, 3, bits=16).load().append(3)
    for cap in (1.1e36, 1e38, 3e38):
        with pytest.raises(ripe.RipeError) as e:
            p.gpu.set_scores(cap)
        assert e.value.status == ripe.RIPE_EINVAL
    p.gpu.set_scores(1e-39)  # a subnormal cap: 0 in the kernel's arithmetic
    with pytest.raises(ripe.RipeError) as e:
        p.gpu.verify_attn(0, 0, bits_dev(p.queries(3)), scale=1e-3)
    assert e.value.status == ripe.RIPE_EINVAL
    p.close()


# ------------------------------------------------------------------ results on a side stream
@pytest.mark.parametrize("as_int", [False, True])
def test_results_of_a_side_stream_are_allocated_on_it(cuda_device, as_int):
    """While the default stream still uses memory that it has given back, and clears new memory only later."""
    p = Pair(2, 4, 2, 64, 2, 8, [200, 131], 3, bits=8, seed=5).load().append(3)
    angle = torch.arange(300, device="cuda")[:, None] * 0.01 ** (torch.arange(32, device="cuda") / 32)
    t = ripe.RotaryTable(angle.cos(), angle.sin())
    q, k = bits_dev(p.queries(3)), torch.randn((2, 3, 2, 64), device="cuda").bfloat16()
    s = torch.cuda.Stream()

    def calls(stream):
        return [p.gpu.verify_attn(0, 0, q, stream=stream), p.gpu.verify_attn_wave(0, [0, 1, 0], q, stream=stream),
                *p.gpu.rotate_block(0, t, k, q, stream=stream), *p.gpu.export(0, 0, stream=stream),
                *p.gpu.export_q8(0, 0, stream=stream), *p.gpu.export(1, 0, stream=stream)]

    want = [x.clone() for x in calls(None)]
    torch.cuda.synchronize()
    for _ in range(3):
        torch.cuda._sleep(100_000_000)
        used = [torch.empty_like(x) for x in want]
        for x in used:
            x.fill_(7)
        del used, x
        got = calls(s.cuda_stream if as_int else s)
        s.synchronize()
        torch.cuda.synchronize()  # the default stream fills its memory only now
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        del got
    p.close()


# ------------------------------------------------------------------ blocks of very different sizes
# V of six blocks; a key's weight does not depend on its value's size, and rows of zeros count as any other
@pytest.mark.parametrize("sizes", [(1e20, 0.0, 1.0, 1e-3, 0.0, 1.0), (0.0, 1e24, 0.0, 0.0, 1.0, 1e24),
                                   (1e24, 1e-25, 1e24, 0.0, 1e24, 1e-20), (1e-25, 1e24, 1.0, 0.0, 1e-24, 0.0)])
@pytest.mark.parametrize("Hq,B,T", [(2, 1, 400), (4, 4, 400), (8, 4, 400), (8, 4, 2000)])
def test_weights_of_blocks_of_zeros_beside_large_ones(cuda_device, sizes, Hq, B, T):
    p = Pair(1, Hq, 1, 64, 1, 8, T, B, seed=6)
    rng = np.random.default_rng(0)
    for b in range((T - 8) // 64):
        x = rng.standard_normal((1, 1, 64, 64)).astype(np.float32) * np.float32(sizes[b % 6])
        p.planes[0][0][1][:, :, 64 * b: 64 * b + 64] = synth.f32_to_bf16_bits(x)
    p.load().append(B)
    qb, lse = p.queries(B), p.lse(B)
    out = p.gpu.verify_attn(0, 0, bits_dev(qb), lse=lse)
    check(p, out, lse, qb)
    p.close()


# ------------------------------------------------------------------ slopes
def test_slopes_at_the_end_of_fp32(cuda_device):
    """Slopes whose bias leaves fp32 where it matters are refused; the largest accepted ones still select their keys."""
    for bits in (8, 16):
        p = Pair(1, 2, 2, 64, 1, 8, 300, 3, bits=bits, seed=15).load().append(3)
        for bad in ([3e38, 0.0], [0.0, -3e38], [-1e36, 0.0]):  # 303 * 1e36 * log2(e) is above 3.4e38
            with pytest.raises(ripe.RipeError) as e:
                p.gpu.set_scores(0.0, bad)
            assert e.value.status == ripe.RIPE_EINVAL
        slopes = [2e38, -5e35]
        p.gpu.set_scores(0.0, slopes)
        qb, lse = p.queries(3), p.lse(3)
        out = p.gpu.verify_attn(0, 0, bits_dev(qb), lse=lse)
        for j in range(3):  # head 0 reads its own key alone, head 1 the oldest one
            for h, t in ((0, 300 + j), (1, 0)):
                v = synth.bf16_bits_to_f32(p.planes[0][0][1][0, h, t])
                if bits == 8 and t == 0:
                    u, s = quantised(synth.bf16_bits_to_f32(p.planes[0][0][1][0, h:h + 1, :64]))
                    v = u[0, 0].astype(np.float32) * s[0, 0]
                got = out[0, j, h].float().cpu().numpy()
                assert (abs(got - v) <= 2.0 ** -7 * abs(v)).all()
        p.close()


def test_a_column_of_zeros_beside_values_of_other_blocks(cuda_device):
    """What a block of tiny values adds to a column that a later, large block leaves at zero is not blown up."""
    for Hq, B in ((2, 1), (4, 4), (8, 4)):
        p = Pair(1, Hq, 1, 64, 1, 8, 400, B, seed=6)
        rng = np.random.default_rng(0)
        for b, size in enumerate((1e-24, 1e-24, 1e24, 1e24, 1e-24, 1e24)):
            x = rng.standard_normal((1, 1, 64, 64)).astype(np.float32) * np.float32(size)
            if size > 1:
                x[..., ::2] = 0
            p.planes[0][0][1][:, :, 64 * b: 64 * b + 64] = synth.f32_to_bf16_bits(x)
        p.planes[0][0][1][:, :, 384:] = synth.f32_to_bf16_bits(np.zeros((1, 1, p.max_T - 384, 64), np.float32))
        p.load().append(B)
        out = p.gpu.verify_attn(0, 0, bits_dev(p.queries(B)))
        assert (out[..., ::2].abs() <= 1e-23).all() and (out[..., 1::2].abs() > 1e18).any()
        p.close()
