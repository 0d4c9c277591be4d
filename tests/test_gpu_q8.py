"""Attention over a cache whose deepest-plane region is held in 8 bits, and that region's upkeep, against 64 bits."""
import numpy as np
import pytest
import torch

from self_speculative_decode_b200 import ripe, synth
from score_ref import Pair, bits_dev, quantised

pytestmark = pytest.mark.gpu


def check_blocks(p, layer=0):
    """The stored blocks are the stated rule's, bit for bit."""
    for n in range(p.N):
        k, v, ks, vs = p.gpu.export_q8(n, layer)
        D = p.D(n)
        assert k.shape == (p.kvH, D, p.d)
        for got, gs, w in ((k, ks, 0), (v, vs, 1)):
            if D:
                u, s = quantised(synth.bf16_bits_to_f32(p.planes[layer][p.R - 1][w][n][:, :D]))
                assert np.array_equal(got.cpu().numpy(), u) and np.array_equal(gs.cpu().numpy(), s)


# query rows per kv head (B * group) 1..64 cover every kernel shape; lengths from an empty cache over ones that end
# inside, at and behind a block to several tiles
@pytest.mark.parametrize("d", [64, 96, 128])
@pytest.mark.parametrize("Hq,kvH,B", [(2, 2, 1), (3, 3, 8), (4, 2, 5), (8, 2, 7), (8, 1, 8)])
def test_verify(cuda_device, d, Hq, kvH, B):
    p = Pair(4, Hq, kvH, d, 3, 16, [0, 1, 80, 409], B, seed=d + B).load().append(B)
    check_blocks(p)
    for r in range(3):
        p.verify(r, B)
    p.wave([(j * 2) % 3 for j in range(B)])
    p.close()


@pytest.mark.parametrize("W", [0, 1, 63, 64, 65, 200, 5000])
@pytest.mark.parametrize("mode", [0, 1])
def test_windows(cuda_device, W, mode):
    p = Pair(3, 4, 2, 64, 3, W, [63, 192, 340], 6, mode=mode, seed=W).load().append(6)
    check_blocks(p)
    for r in range(3):
        p.verify(r, 6)
    p.wave([2, 0, 1, 2, 0, 0])
    p.close()


@pytest.mark.parametrize("sink,window", [(None, None), (0, 0), (4, 30), (100, 10), (64, 64), (3, 1 << 30)])
def test_draft(cuda_device, sink, window):
    p = Pair(3, 4, 2, 96, 4, 16, [0, 150, 333], 5, seed=9).load()
    for j in range(5):
        p.draft(1, j, sink, window)
    p.close()


def test_append_verify_and_layers(cuda_device):
    p = Pair(2, 4, 4, 64, 2, 8, [70, 300], 4, L=2, seed=4).load()
    for layer in range(2):
        check_blocks(p, layer)
        for r in range(2):
            q, lse = p.queries(4), p.lse(4)
            k, v = map(bits_dev, p.rows(layer, r, 0, 4))
            out = p.gpu.append_verify(layer, r, k, v, bits_dev(q), lse=lse)
            p.check(out, lse, q, r, layer=layer)
    p.close()


def test_contents_do_not_depend_on_how_positions_were_committed(cuda_device):
    """From the same lengths on, one token at a time, in uneven blocks with rollbacks, or in blocks of 64: the same
    bytes; and they are those of loading the longer prefix."""
    got = []
    for blocks in ([1] * 70, [13, 7, 1, 13, 13, 5, 9, 9], [64, 6]):
        p = Pair(2, 2, 2, 64, 2, 10, [100, 64], 64, room=80, seed=3).load()
        for i, a in enumerate(blocks):
            B = a if i % 2 else min(64, a + 3)  # some of the block is rolled back
            p.append(B)
            p.commit([a, a])
        check_blocks(p)
        p.append(4).verify(0, 4)
        got.append([x for n in range(2) for x in p.gpu.export_q8(n, 0)])
        p.close()
    for other in got[1:]:
        assert all(torch.equal(a, b) for a, b in zip(got[0], other))


def test_commit_on_the_device_and_in_a_graph(cuda_device):
    """A step (append, verify, device-side commit) captured once and replayed follows the lengths."""
    p = Pair(3, 4, 2, 64, 2, 16, [50, 127, 200], 4, room=80, seed=12).load()
    kv = [[torch.empty((3, 4, 2, 64), dtype=torch.bfloat16, device="cuda") for _ in range(2)] for _ in range(2)]
    q = torch.empty((3, 4, 4, 64), dtype=torch.bfloat16, device="cuda")
    out, lse = torch.empty_like(q), p.lse(4)
    acc = torch.zeros(3, dtype=torch.int32, device="cuda")

    def fill():
        qb = p.queries(4)
        q.copy_(bits_dev(qb))
        for r in range(2):
            for dst, src in zip(kv[r], p.rows(0, r, 0, 4)):
                dst.copy_(bits_dev(src))
        return qb

    def step():
        for r in range(2):
            p.gpu.append_block(0, r, *kv[r])
        p.gpu.verify_attn(0, 0, q, out=out, lse=lse)
        p.gpu.commit_device(acc)

    fill()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):  # the first step runs as it is (and accepts nothing), the second is captured
        step()
    torch.cuda.current_stream().wait_stream(s)
    p.gpu.sync_lengths()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for i in range(12):
        qb = fill()
        a = [(i * 2 + n) % 5 for n in range(3)]
        acc.copy_(torch.tensor(a, dtype=torch.int32))
        g.replay()
        torch.cuda.synchronize()
        p.check(out, lse, qb, 0)
        p.T = [t + x for t, x in zip(p.T, a)]
    assert p.gpu.sync_lengths() == p.T
    check_blocks(p)
    p.close()


def test_many_short_sequences(cuda_device):
    rng = np.random.default_rng(1)
    T = [int(t) for t in rng.integers(0, 150, 300)]
    p = Pair(300, 2, 1, 64, 2, 8, T, 3, seed=8).load().append(3)
    p.verify(0, 3, rows={(n, i) for n in range(0, 300, 7) for i in range(3)})
    p.close()


def test_few_long_heads_are_split_and_merged(cuda_device):
    p = Pair(1, 8, 1, 128, 2, 64, 9000, 8, seed=21).load().append(8)
    p.verify(0, 8, rows={(0, 0), (0, 7)})
    p.close()
    p = Pair(5, 4, 4, 96, 2, 64, [4000, 70, 2111, 64, 3333], 2, seed=22).load().append(2)
    p.verify(1, 2)
    p.close()


@pytest.mark.parametrize("q_std", [0.0, 1e-30, 12.0, 1e20])
def test_query_magnitudes(cuda_device, q_std):
    """Queries are brought into f16's range row by row; scale undoes what q_std did."""
    scale = 1.0 if q_std in (0.0, 12.0) else 1.0 / q_std
    p = Pair(2, 4, 2, 64, 2, 8, [200, 131], 3, seed=5, q_std=q_std, scale=scale).load().append(3)
    p.verify(0, 3)
    p.close()


def test_magnitudes_of_keys_and_values(cuda_device):
    """Blocks of zeros, tiny, large and ordinary values side by side, each with its own scale."""
    p = Pair(1, 2, 2, 64, 2, 8, 400, 3, seed=6)
    rng = np.random.default_rng(0)
    for w, sizes in ((0, (1.0, 0.0, 1e-3, 3.0, 1e-20, 1.0)), (1, (1e-25, 1e3, 0.0, 1.0, 1e20, 1e-6))):
        plane = p.planes[0][1][w]
        for b, size in enumerate(sizes):
            x = rng.standard_normal((1, 2, 64, 64)).astype(np.float32) * np.float32(size)
            plane[:, :, 64 * b: 64 * b + 64] = synth.f32_to_bf16_bits(x)
    p.load().append(3)
    check_blocks(p)
    p.verify(0, 3)
    p.close()


def test_a_block_with_a_nan_or_an_infinity_reads_as_nan(cuda_device):
    """Whoever sees the block gets NaN, and a draft that does not read or see it gets none; a block beyond the largest
    scale likewise."""
    for w, bad in ((0, 0x7FC0), (1, 0x7F80), (1, 0xFF80), (0, 0x7F00)):
        p = Pair(2, 2, 2, 64, 2, 8, [400, 390], 3, seed=7)
        p.planes[0][1][w][0, 1, 130, 5] = bad  # sequence 0, head 1, block 2 of the deepest plane
        p.load().append(3)
        q = p.queries(3)
        lse = p.lse(3)
        out = p.gpu.verify_attn(0, 0, bits_dev(q), lse=lse)
        assert out[0, :, 1].isnan().all() and lse[0, :, 1].isnan().all()
        assert out[0, :, 0].isfinite().all() and out[1].isfinite().all() and lse[1].isfinite().all()
        p.gpu.close()
        p = Pair(2, 2, 2, 64, 2, 8, [400, 390], 3, seed=7)
        p.planes[0][1][w][0, 1, 130, 5] = bad
        p.load()
        k, v = map(bits_dev, p.rows(0, 0, 0, 1))
        for sink, window, sees in ((4, 100, False), (0, 220, True), (130, 10, True), (64, 205, False)):
            q = p.queries(1)
            out = p.gpu.draft_attn(0, 0, 0, k, v, bits_dev(q), sink=sink, window=window)
            # (64, 205): p - window = 195, in block 3; block 2 is not read
            assert bool(out[0, 0, 1].isnan().any()) == sees, (w, bad, sink, window)
            assert out[1].isfinite().all()
        p.gpu.close()


def test_stale_and_later_rows_that_hold_nan_reach_no_query(cuda_device):
    """NaN in rolled-back rows, and in a later row of the block, stays out of the queries that do not attend to it."""
    for bits in (8, 16):
        p = Pair(2, 4, 2, 64, 2, 8, [100, 190], 6, bits=bits, cap=40.0, room=10, seed=2).load()
        nan = torch.full((2, 6, 2, 64), float("nan"), dtype=torch.bfloat16, device="cuda")
        for r in range(2):
            p.gpu.append_block(0, r, nan, nan)
        p.commit([0, 0])
        p.append(3).verify(0, 3)
        p.commit([3, 3])
        for r in range(2):
            k, v = map(bits_dev, p.rows(0, r, 0, 4))
            v[:, 2] = float("inf")
            k[:, 3] = float("nan")
            p.gpu.append_block(0, r, k, v)
        q, lse = p.queries(4), p.lse(4)
        out = p.gpu.verify_attn(0, 0, bits_dev(q), lse=lse)
        p.check(out, lse, q, 0, rows={(n, i) for n in range(2) for i in range(2)})
        assert (out[:, 2] == float("inf")).all() and out[:, 3].isnan().all() and lse[:, 3].isnan().all()
        p.gpu.close()


def test_export_view_and_stats(cuda_device):
    p = Pair(2, 2, 2, 64, 3, 10, [150, 40], 4, seed=1).load().append(4, loops=[0])
    st = p.gpu.stats()
    assert ripe.ripe_cache_kv_bits(p.gpu.handle) == 8
    assert st["deep_rows"] == 128 and st["ring_slots"] == 10 + 63 + 4
    for n in range(2):
        k, v, present = p.gpu.export(n, 0)
        T, D = p.T[n], p.D(n)
        for got, w in ((k, 0), (v, 1)):
            deep = synth.bf16_bits_to_f32(p.planes[0][2][w][n])
            if D:
                u, s = quantised(deep[:, :D])
                want = torch.from_numpy(u.astype(np.float32) * np.repeat(s, 64, 1)[:, :, None]).bfloat16()
                assert torch.equal(got[2, :, :D].cpu(), want)
            assert torch.equal(got[2, :, D:T].float().cpu(), torch.from_numpy(deep[:, D:T]))
            near = synth.bf16_bits_to_f32(p.planes[0][0][w][n])
            lo = max(0, T - 10)
            assert torch.equal(got[0, :, lo:].float().cpu(), torch.from_numpy(near[:, lo:T + 4]))
            assert not got[0, :, :lo].any() and not got[1, :, T:].any()
        pr = present.cpu().numpy()
        assert pr[2, :T].all() and pr[0, lo:].all() and not pr[0, :lo].any() and not pr[1, T:].any()
    p.close()


def test_refusals(cuda_device):
    p = Pair(1, 2, 2, 64, 2, 8, 100, 3, bits=16).load().append(3)
    with pytest.raises(ripe.RipeError) as e:
        p.gpu.export_q8(0, 0)  # a bf16 cache
    assert e.value.status == ripe.RIPE_EINVAL
    p.close()
    p = Pair(1, 2, 2, 64, 2, 8, 100, 3).load()
    q = bits_dev(p.queries(3))
    with pytest.raises(ripe.RipeError) as e:
        p.gpu.verify_attn(0, 0, q)  # nothing appended
    assert e.value.status == ripe.RIPE_ESTATE
    p.append(3)
    odd = torch.empty(q.numel() + 1, dtype=torch.bfloat16, device="cuda")[1:].view(q.shape)
    for a, b in ((odd, None), (q, odd)):
        with pytest.raises(ripe.RipeError) as e:
            p.gpu.verify_attn(0, 0, a, out=b)
        assert e.value.status == ripe.RIPE_EINVAL
    with pytest.raises(ValueError):
        ripe.RipeCache(1, 1, 2, 2, 64, 2, 8, 100, 3, kv_bits=4)
    p.close()
