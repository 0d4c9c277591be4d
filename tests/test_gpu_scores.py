"""Capped scores and a bias linear in the distance, over both kinds of cache, against 64 bits."""
import numpy as np
import pytest
import torch

from self_speculative_decode_b200 import ripe
from score_ref import Pair, bits_dev

pytestmark = pytest.mark.gpu


def slopes(H):
    return [2.0 ** (-8.0 * (h + 1) / H) for h in range(H)]


@pytest.mark.parametrize("bits", [8, 16])
@pytest.mark.parametrize("cap,bias", [(5.0, False), (0.0, True), (50.0, True)])
@pytest.mark.parametrize("d,Hq,kvH,B", [(64, 2, 2, 1), (96, 3, 3, 8), (64, 4, 2, 8), (128, 8, 2, 7), (128, 8, 1, 8)])
def test_verify(cuda_device, bits, cap, bias, d, Hq, kvH, B):
    p = Pair(4, Hq, kvH, d, 3, 16, [0, 1, 80, 409], B, bits=bits, cap=cap, slopes=slopes(Hq) if bias else None,
             q_std=4.0, seed=d + B).load().append(B)
    for r in range(3):
        p.verify(r, B)
    p.wave([(j * 2) % 3 for j in range(B)])
    p.close()


@pytest.mark.parametrize("bits", [8, 16])
@pytest.mark.parametrize("W,mode", [(0, 0), (1, 1), (64, 0), (65, 1), (5000, 0)])
def test_windows(cuda_device, bits, W, mode):
    p = Pair(3, 4, 2, 64, 3, W, [63, 192, 340], 6, bits=bits, mode=mode, cap=20.0, slopes=slopes(4), q_std=3.0,
             seed=W).load().append(6)
    for r in range(3):
        p.verify(r, 6)
    p.wave([2, 0, 1, 2, 0, 0])
    p.close()


@pytest.mark.parametrize("bits", [8, 16])
@pytest.mark.parametrize("sink,window", [(None, None), (0, 0), (4, 30), (100, 10), (3, 1 << 30)])
def test_draft(cuda_device, bits, sink, window):
    p = Pair(3, 4, 2, 96, 4, 16, [0, 150, 333], 5, bits=bits, cap=30.0, slopes=slopes(4), q_std=5.0, seed=9).load()
    for j in range(5):
        p.draft(1, j, sink, window)
    p.close()


@pytest.mark.parametrize("bits", [8, 16])
def test_append_verify_then_commit(cuda_device, bits):
    p = Pair(2, 4, 4, 64, 2, 8, [70, 300], 4, bits=bits, cap=10.0, room=40, seed=4).load()
    for a in (4, 0, 3, 4, 4, 1):
        for r in range(2):
            q, lse = p.queries(4), p.lse(4)
            k, v = map(bits_dev, p.rows(0, r, 0, 4))
            out = p.gpu.append_verify(0, r, k, v, bits_dev(q), lse=lse)
            p.check(out, lse, q, r)
        p.commit([a, 4 - a])
    p.close()


@pytest.mark.parametrize("scale,cap", [(0.0, 10.0), (-1.0, 10.0), (300.0, 2.0), (1e-3, 1e4)])
def test_scales_and_caps(cuda_device, scale, cap):
    p = Pair(2, 4, 2, 64, 2, 8, [200, 131], 3, cap=cap, scale=scale, seed=5).load().append(3)
    p.verify(0, 3)
    p.close()


def test_steep_slopes_leave_the_nearest_keys(cuda_device):
    """Negative slopes too: the bias then favours the oldest keys, and the softmax reference keeps moving."""
    for bits in (8, 16):
        p = Pair(1, 4, 4, 64, 2, 8, 700, 3, bits=bits, slopes=[200.0, 0.5, -0.25, -3.0], seed=15).load().append(3)
        p.verify(0, 3)
        p.close()


def test_long_distances(cuda_device):
    """Split heads of an uneven batch."""
    p = Pair(3, 8, 1, 128, 2, 64, [6000, 65, 2500], 4, bits=16, cap=50.0, slopes=slopes(8), q_std=6.0, seed=3)
    p.load().append(4).verify(0, 4, rows={(0, 0), (0, 3), (1, 1), (2, 2)})
    p.close()


def test_scores_are_set_and_cleared(cuda_device):
    """Without a cap and slopes the calls are the plain ones again, bit for bit; scale 1 with a cap far above every score
    is within the cap's rounding of them."""
    p = Pair(2, 4, 2, 64, 2, 8, [200, 131], 3, bits=16, seed=5).load().append(3)
    q = bits_dev(p.queries(3))
    plain = p.gpu.verify_attn(0, 0, q)
    p.gpu.set_scores(3.0, slopes(4))
    assert not torch.equal(p.gpu.verify_attn(0, 0, q), plain)
    p.gpu.set_scores()
    assert torch.equal(p.gpu.verify_attn(0, 0, q), plain)
    p.close()


@pytest.mark.parametrize("bits", [8, 16])
@pytest.mark.parametrize("Hq,B", [(2, 3), (4, 4), (8, 6), (8, 8)])
def test_a_query_with_nan_spoils_its_own_row_only(cuda_device, bits, Hq, B):
    """And a log-sum-exp that is not asked for is not written."""
    p = Pair(2, Hq, 1, 64, 2, 8, [300, 20], B, bits=bits, cap=25.0, seed=13).load().append(B)
    qb = p.queries(B)
    bad = qb.copy()
    bad[0, 1, 0, 3] = 0x7FC0
    bad[1, 0, 1, 5] = 0x7F80
    out = p.gpu.verify_attn(0, 0, bits_dev(bad))
    want = p.gpu.verify_attn(0, 0, bits_dev(qb))
    spoilt = torch.zeros((2, B, Hq), dtype=torch.bool, device="cuda")
    spoilt[0, 1, 0] = spoilt[1, 0, 1] = True
    assert torch.equal(out[~spoilt], want[~spoilt])
    assert out[0, 1, 0].isnan().all() and not torch.equal(out[1, 0, 1], want[1, 0, 1])
    p.close()


def test_two_caches_and_a_second_stream(cuda_device):
    """Two caches used in turn, one of them on a stream of its own."""
    a = Pair(2, 4, 2, 64, 2, 8, [200, 131], 3, bits=8, cap=20.0, seed=5).load().append(3)
    b = Pair(2, 4, 2, 64, 2, 8, [333, 60], 3, bits=16, slopes=slopes(4), seed=6).load().append(3)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        qa, qb, la, lb = a.queries(3), b.queries(3), a.lse(3), b.lse(3)
        da, db = bits_dev(qa), bits_dev(qb)
        s.wait_stream(torch.cuda.current_stream())
        oa = a.gpu.verify_attn(0, 0, da, lse=la)
        ob = torch.empty_like(db)
        b.gpu.verify_attn(0, 0, db, out=ob, lse=lb, stream=s)
        torch.cuda.current_stream().wait_stream(s)
        a.check(oa, la, qa, 0)
        b.check(ob, lb, qb, 0)
    a.close()
    b.close()


def test_refusals(cuda_device):
    p = Pair(1, 2, 2, 64, 2, 8, 100, 3, bits=16).load().append(3)
    for cap, sl in ((-1.0, None), (float("nan"), None), (float("inf"), None), (0.0, [1.0, float("nan")]),
                    (0.0, [float("inf"), 1.0])):
        with pytest.raises(ripe.RipeError) as e:
            p.gpu.set_scores(cap, sl)
        assert e.value.status == ripe.RIPE_EINVAL
    with pytest.raises(ValueError):
        p.gpu.set_scores(0.0, [1.0])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        with pytest.raises(ripe.RipeError) as e:
            p.gpu.set_scores(1.0)
        assert e.value.status == ripe.RIPE_ESTATE
        torch.zeros(1, device="cuda")
    p.gpu.set_scores(10.0)
    q = bits_dev(p.queries(3))
    odd = torch.empty(q.numel() + 1, dtype=torch.bfloat16, device="cuda")[1:].view(q.shape)
    with pytest.raises(ripe.RipeError) as e:
        p.gpu.verify_attn(0, 0, odd)
    assert e.value.status == ripe.RIPE_EINVAL
    p.gpu.set_scores(1e-39)  # 2 log2(e) / cap = 2.9e39 is above the largest fp32, 3.4e38
    for scale in (1.0, float("nan"), float("inf")):
        with pytest.raises(ripe.RipeError) as e:
            p.gpu.verify_attn(0, 0, q, scale=scale)
        assert e.value.status == ripe.RIPE_EINVAL
    p.close()
