"""Appending with the position rotation, and rotating alone, against 64 bits; and the calls together in a decoding loop."""
import numpy as np
import pytest
import torch

from self_speculative_decode_b200 import ripe, synth
from score_ref import Pair, bits_dev

pytestmark = pytest.mark.gpu


def table(positions, rot, interleaved):
    """fp32 tables of angles taken in 64 bits."""
    angle = np.arange(positions)[:, None] * 10000.0 ** (-2.0 * np.arange(rot // 2) / rot)
    c, s = (torch.from_numpy(f(angle).astype(np.float32)).cuda() for f in (np.cos, np.sin))
    return ripe.RotaryTable(c, s, interleaved)


def rotated(x, pos, t):
    """x [..., heads, d] float64 at positions pos [...]: the definition, from the fp32 tables."""
    x = x.copy()
    rot, half = t.rope.rotary_dim, t.rope.rotary_dim // 2
    a = np.arange(half) * (2 if t.rope.interleaved else 1)
    b = a + (1 if t.rope.interleaved else half)
    c, s = (y.cpu().numpy().astype(np.float64)[pos][..., None, :] for y in (t.cos, t.sin))
    u, v = x[..., a], x[..., b]
    x[..., a], x[..., b] = u * c - v * s, v * c + u * s
    # each output: two fp32 products and their sum, then one rounding to bf16
    size = np.abs(u) + np.abs(v)
    tol = np.zeros_like(x)
    tol[..., a] = tol[..., b] = 2.0 ** -22 * size
    return x, tol + 2.0 ** -8 * np.abs(x) * (np.arange(x.shape[-1]) < rot)


def f64(t):
    return t.double().cpu().numpy()


def close(got, want, tol):
    assert (np.abs(f64(got) - want) <= tol).all(), float((np.abs(f64(got) - want) / np.maximum(tol, 1e-30)).max())


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,rot", [(64, 64), (64, 8), (96, 96), (96, 24), (96, 80), (128, 128), (128, 32), (128, 120)])
@pytest.mark.parametrize("N,Hq,kvH,B", [(1, 1, 1, 1), (5, 6, 2, 7), (70, 8, 8, 8)])
def test_append(cuda_device, interleaved, d, rot, N, Hq, kvH, B):
    rng = np.random.default_rng(d + rot)
    T = [int(t) for t in rng.integers(0, 3000, N)]
    c = ripe.RipeCache(N, 1, Hq, kvH, d, 2, 16, max(T) + B, B)
    kv = torch.zeros((N, kvH, max(T) + 1, d), dtype=torch.bfloat16, device="cuda")
    c.load_prefix(0, 1, T, kv, kv)
    t = table(max(T) + B, rot, interleaved)
    k, v, q = (torch.randn((N, B, h, d), device="cuda").bfloat16() for h in (kvH, kvH, Hq))
    q_out = c.append_block_rope(0, 1, k, v, t, q)
    pos = np.array(T)[:, None] + np.arange(B)
    close(q_out, *rotated(f64(q), pos, t))
    want, tol = rotated(f64(k), pos, t)
    for n in {0, N // 2, N - 1}:
        ko, vo, _ = c.export(n, 0)
        close(ko[1, :, T[n]:].transpose(0, 1), want[n], tol[n])
        assert torch.equal(vo[1, :, T[n]:].transpose(0, 1), v[n])
    k2, q2 = c.rotate_block(0, t, k, q)
    assert torch.equal(q2, q_out)
    close(k2, want, tol)
    # in place, and the part of a block
    assert c.rotate_block(0, t, q=q, q_out=q)[1] is q and torch.equal(q, q_out)
    if B > 2:
        k3, _ = c.rotate_block(2, t, k[:, 2:].contiguous())
        assert torch.equal(k3, k2[:, 2:])
    assert c.device_error() == 0
    c.close()


def test_parts_of_one_projection(cuda_device):
    """k, v and q as strided parts of one tensor give what packed copies give."""
    N, B, Hq, kvH, d = 3, 5, 4, 2, 64
    c = ripe.RipeCache(N, 1, Hq, kvH, d, 2, 16, 400, B)
    t = table(400, 64, False)
    x = torch.randn((N, B, (Hq + 2 * kvH) * d), device="cuda").bfloat16()
    q, k, v = x[..., :Hq * d].view(N, B, Hq, d), x[..., Hq * d:(Hq + kvH) * d].view(N, B, kvH, d), \
        x[..., (Hq + kvH) * d:].view(N, B, kvH, d)
    a = c.append_block_rope(0, 0, k, v, t, q)
    ea = c.export(1, 0)
    b = c.append_block_rope(0, 0, k.contiguous(), v.contiguous(), t, q.contiguous())
    assert torch.equal(a, b) and all(torch.equal(x, y) for x, y in zip(ea, c.export(1, 0)))
    with pytest.raises(ripe.RipeError) as e:  # q_out over a part of the inputs
        c.append_block_rope(0, 0, k, v, t, q, q_out=x.view(-1)[:N * B * Hq * d].view(N, B, Hq, d))
    assert e.value.status == ripe.RIPE_EINVAL
    c.close()


def test_static_ring_wraps_and_leaves_other_rows(cuda_device):
    N, B, Hq, kvH, d, W, max_T = 4, 6, 4, 2, 96, 10, 5000
    S = W + B
    T = torch.tensor([0, 13, 4994, 4995], dtype=torch.int32, device="cuda")  # the last one does not fit
    ring = [torch.randn((2, N, 3, kvH, S, d), device="cuda").bfloat16() for _ in range(2)]
    before = [x.clone() for x in ring]
    view = ripe.CacheView(batch=N, layers=2, q_heads=Hq, kv_heads=kvH, head_dim=d, loops=3, window=W, max_T=max_T, max_B=B,
                          window_mode=0, block_len=B, k_ring=ring[0].data_ptr(), v_ring=ring[1].data_ptr(),
                          lengths=T.data_ptr())
    k, v, q = (torch.randn((N, B, h, d), device="cuda").bfloat16() for h in (kvH, kvH, Hq))
    t = table(max_T, 48, True)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    q_out = torch.full_like(q, 7.0)
    ripe.append_rope_static(view, 1, 2, k, v, q, t, q_out, err)
    assert err.item() == ripe.RIPE_DEVERR_CAPACITY
    pos = T.cpu().numpy()[:3, None] + np.arange(B)
    want, tol = rotated(f64(k[:3]), pos, t)
    close(q_out[:3], *rotated(f64(q[:3]), pos, t))
    assert (q_out[3] == 7.0).all()
    for n in range(3):
        for j in range(B):
            slot = (int(T[n]) + j) % S
            close(ring[0][1, n, 2, :, slot], want[n, j], tol[n, j])
            assert torch.equal(ring[1][1, n, 2, :, slot], v[n, j])
            for x, y in zip(ring, before):
                y[1, n, 2, :, slot] = x[1, n, 2, :, slot]
    assert all(torch.equal(x, y) for x, y in zip(ring, before))  # nothing else was touched
    # without a table the rows are copied; a negative or huge length is left out
    T.copy_(torch.tensor([-1, 2 ** 31 - 1, 20, 30]))
    err.zero_()
    before = [x.clone() for x in ring]
    assert ripe.append_rope_static(view, 0, 0, k, v, device_error=err) is None
    assert err.item() == ripe.RIPE_DEVERR_CAPACITY
    assert torch.equal(ring[0][0, 2, 0, :, 20 % S], k[2, 0]) and torch.equal(ring[0][:, :2], before[0][:, :2])


def test_a_captured_append_follows_the_lengths(cuda_device):
    N, B, d = 2, 3, 64
    T = torch.tensor([5, 40], dtype=torch.int32, device="cuda")
    ring = [torch.zeros((1, N, 1, 1, 20 + B, d), device="cuda").bfloat16() for _ in range(2)]
    view = ripe.CacheView(batch=N, layers=1, q_heads=1, kv_heads=1, head_dim=d, loops=1, window=20, max_T=500, max_B=B,
                          window_mode=0, block_len=B, k_ring=ring[0].data_ptr(), v_ring=ring[1].data_ptr(),
                          lengths=T.data_ptr())
    k, v, q = (torch.randn((N, B, 1, d), device="cuda").bfloat16() for _ in range(3))
    t, err, q_out = table(500, 64, False), torch.zeros(1, dtype=torch.int32, device="cuda"), torch.empty_like(q)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ripe.append_rope_static(view, 0, 0, k, v, q, t, q_out, err)
    for _ in range(3):
        T += 7
        g.replay()
        torch.cuda.synchronize()
        pos = T.cpu().numpy()[:, None] + np.arange(B)
        close(q_out, *rotated(f64(q), pos, t))
        want, tol = rotated(f64(k), pos, t)
        for n in range(N):
            for j in range(B):
                close(ring[0][0, n, 0, :, pos[n, j] % 23], want[n, j], tol[n, j])
    assert err.item() == 0


@pytest.mark.parametrize("bits", [8, 16])
def test_a_decoding_loop_with_rotation_cap_and_bias(cuda_device, bits):
    """Draft (windowed), rotated append, verification with a cap and a bias, device-side commit: the cache holds the
    rotated keys, and every result is that of 64 bits over them."""
    N, Hq, kvH, d, R, W, B = 2, 4, 2, 64, 2, 16, 4
    p = Pair(N, Hq, kvH, d, R, W, [90, 200], B, bits=bits, cap=30.0, slopes=[0.1, 0.02, 0.3, 0.0], room=120, seed=31, q_std=3.0)
    t = table(p.max_T, 32, False)
    # keys before rotation; the reference holds what the cache should: rotated, rounded to bf16
    raw = [p.planes[0][r][0].copy() for r in range(R)]
    cos, sin = t.cos.cpu(), t.sin.cpu()

    def turn(bits_, pos):  # [..., heads, d] as the kernel rounds: fp32 products, one rounding
        x = torch.from_numpy(synth.bf16_bits_to_f32(bits_).astype(np.float64))
        c, s = cos[pos.copy()].double()[..., None, :], sin[pos.copy()].double()[..., None, :]
        a, b = x[..., :16].clone(), x[..., 16:32].clone()
        x[..., :16], x[..., 16:32] = a * c - b * s, b * c + a * s
        return x

    for r in range(R):
        x = turn(raw[r].transpose(0, 2, 1, 3), np.broadcast_to(np.arange(p.max_T), (N, p.max_T)))
        p.planes[0][r][0][:] = synth.f32_to_bf16_bits(x.float().numpy()).transpose(0, 2, 1, 3)
    p.load()
    rng = np.random.default_rng(5)
    for step in range(6):
        T = list(p.T)

        def raw_rows(r, j, n_rows):
            k = np.stack([raw[r][n, :, T[n] + j: T[n] + j + n_rows].transpose(1, 0, 2) for n in range(N)])
            return bits_dev(k), bits_dev(p.rows(0, r, j, n_rows)[1])

        def sync_reference(r, j, n_rows):
            # the reference takes the rows that the cache holds (rounding of the rotation is tested above)
            for n in range(N):
                k = p.gpu.export(n, 0)[0] if n_rows > 1 else None
                if k is not None:
                    got = k[r, :, T[n]:T[n] + n_rows].contiguous().view(torch.int16).cpu().numpy().view(np.uint16)
                    p.planes[0][r][0][n, :, T[n]:T[n] + n_rows] = got

        for j in range(2):
            k, v = raw_rows(0, j, 1)
            qb = p.queries(1)
            kt, qt = p.gpu.rotate_block(j, t, k, bits_dev(qb))
            for n in range(N):
                p.planes[0][0][0][n, :, T[n] + j] = kt[n, 0].contiguous().view(torch.int16).cpu().numpy().view(np.uint16)
            lse = p.lse(1)
            out = p.gpu.draft_attn(0, 0, j, kt, v, qt, lse=lse, sink=4, window=64)
            qr = qt.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)
            p.check(out, lse, qr, 0, j0=j, sink=4, window=64)
        for r in range(R):
            k, v = raw_rows(r, 0, B)
            qb = p.queries(B)
            qt = p.gpu.append_block_rope(0, r, k, v, t, bits_dev(qb))
            sync_reference(r, 0, B)
            lse = p.lse(B)
            out = p.gpu.verify_attn(0, r, qt, lse=lse)
            p.check(out, lse, qt.contiguous().view(torch.int16).cpu().numpy().view(np.uint16), r)
        a = [int(x) for x in rng.integers(0, B + 1, N)]
        p.gpu.commit_device(torch.tensor(a, dtype=torch.int32, device="cuda"))
        p.T = [x + y for x, y in zip(p.T, a)]
        assert p.gpu.sync_lengths() == p.T
    p.close()


def test_refusals(cuda_device):
    N, B, Hq, kvH, d = 2, 4, 4, 2, 64
    c = ripe.RipeCache(N, 1, Hq, kvH, d, 2, 16, 100, B)
    k, v, q = (torch.zeros((N, B, h, d), dtype=torch.bfloat16, device="cuda") for h in (kvH, kvH, Hq))
    t = table(100, 64, False)

    def refused(status, f, *a, **kw):
        with pytest.raises(ripe.RipeError) as e:
            f(*a, **kw)
        assert e.value.status == status

    refused(ripe.RIPE_EINVAL, c.append_block_rope, 1, 0, k, v, t)
    refused(ripe.RIPE_EINVAL, c.append_block_rope, 0, 2, k, v, t)
    refused(ripe.RIPE_ECAPACITY, c.append_block_rope, 0, 0, k, v, table(B - 1, 64, False))
    refused(ripe.RIPE_EINVAL, c.rotate_block, 1, t, k)        # positions 1 .. B: past max_B
    refused(ripe.RIPE_EINVAL, c.rotate_block, -1, t, k)
    refused(ripe.RIPE_EINVAL, c.append_block_rope, 0, 0, k, v, table(100, 66, False))  # not a multiple of 8
    refused(ripe.RIPE_EINVAL, c.append_block_rope, 0, 0, k, v, table(100, 72, False))  # more than the head
    odd = torch.zeros(q.numel() + 1, dtype=torch.bfloat16, device="cuda")[1:].view(q.shape)
    refused(ripe.RIPE_EINVAL, c.append_block_rope, 0, 0, k, v, t, odd)
    c.append_block_rope(0, 0, k, v, t)
    refused(ripe.RIPE_EINVAL, c.append_block_rope, 0, 0, k[:, :2].contiguous(), v[:, :2].contiguous(), t)  # another length
    with pytest.raises(ValueError):
        c.append_block_rope(0, 0, k.transpose(1, 2).contiguous().transpose(1, 2), v, t)  # heads not packed
    with pytest.raises(ValueError):
        c.append_block_rope(0, 0, k.float(), v, t)
    with pytest.raises(ValueError):
        ripe.RotaryTable(torch.zeros(8, 32), torch.zeros(8, 32))
    assert c.device_error() == 0
    c.close()
