"""Misaligned pointers are refused on the host (the kernels' loads and stores are 4 or 16 bytes wide)."""
import ctypes

import pytest
import torch

from self_speculative_decode_b200 import ripe


def _static(q=1 << 24, out=1 << 25, lse=1 << 26, lengths=4 << 20, error=64):
    """A call that a host check has to refuse: its addresses are made up, and are never read."""
    view = ripe.CacheView(batch=2, layers=1, q_heads=4, kv_heads=2, head_dim=64, loops=2, window=8, max_T=8, max_B=4,
                          window_mode=0, block_len=4, k_ring=1 << 20, v_ring=2 << 20, lengths=lengths)
    vp = ctypes.c_void_p
    return ripe.lib().ripe_verify_attn_static(ctypes.byref(view), 0, 0, vp(q), vp(out), vp(lse), 1.0, vp(error), vp(0))


@pytest.mark.parametrize("call", [dict(q=(1 << 24) + 2), dict(out=(1 << 25) + 2), dict(lse=(1 << 26) + 2),
                                  dict(lengths=(4 << 20) + 2), dict(error=66)])
def test_static_verify(call):
    assert _static(**call) == ripe.RIPE_EINVAL


def shifted(x, elements):
    """A contiguous copy of x whose first element lies `elements` elements behind a 16-byte boundary."""
    buf = torch.zeros(x.numel() + 16, dtype=x.dtype, device=x.device)
    y = buf[elements: elements + x.numel()].view(x.shape)
    y.copy_(x)
    assert y.data_ptr() % 16 == elements * x.element_size() % 16
    return y


@pytest.mark.gpu
@pytest.mark.parametrize("bits,cap", [(16, 0.0), (16, 30.0), (8, 0.0)])
def test_calls_on_a_cache(cuda_device, bits, cap):
    """Odd elements are refused everywhere, q and out at any even one give what aligned tensors give."""
    N, B, Hq, kvH, d = 2, 3, 4, 2, 64
    c = ripe.RipeCache(N, 1, Hq, kvH, d, 2, 8, 300, B, kv_bits=bits)
    if cap:
        c.set_scores(cap)
    T = [200, 90]

    def rows(*shape):
        return torch.randn(shape, device="cuda").bfloat16()

    def refused(f, *a, **kw):
        with pytest.raises(ripe.RipeError) as e:
            f(*a, **kw)
        assert e.value.status == ripe.RIPE_EINVAL

    kv, k, v, q, k1, q1 = rows(N, kvH, 200, d), rows(N, B, kvH, d), rows(N, B, kvH, d), rows(N, B, Hq, d), \
        rows(N, 1, kvH, d), rows(N, 1, Hq, d)
    for off in (1, 2, 4):
        refused(c.load_prefix, 0, 0, T, shifted(kv, off), kv)
        refused(c.load_prefix, 0, 0, T, kv, shifted(kv, off))
    for r in range(2):
        c.load_prefix(0, r, T, kv, kv)
    lse1 = torch.zeros((N, 1, Hq), device="cuda")
    for off in (1, 2, 4):
        refused(c.draft_attn, 0, 0, 0, shifted(k1, off), k1, q1)
        refused(c.draft_attn, 0, 0, 0, k1, shifted(k1, off), q1)
        refused(c.append_block, 0, 0, shifted(k, off), v)
        refused(c.append_block, 0, 0, k, shifted(v, off))
        refused(c.append_verify, 0, 0, k, shifted(v, off), q)
    refused(c.draft_attn, 0, 0, 0, k1, k1, shifted(q1, 1))
    want = c.draft_attn(0, 0, 0, k1, k1, q1, lse=lse1)
    assert torch.equal(c.draft_attn(0, 0, 0, k1, k1, shifted(q1, 2), out=shifted(q1, 6)), want)
    for r in range(2):
        c.append_block(0, r, k, v)
    for call in (lambda *a, **kw: c.verify_attn(0, 0, *a, **kw), lambda *a, **kw: c.append_verify(0, 0, k, v, *a, **kw),
                 lambda *a, **kw: c.verify_attn_wave(0, [0, 1, 0], *a, **kw)):
        refused(call, shifted(q, 1))
        refused(call, q, out=shifted(q, 1))
        want = call(q)
        for off in (2, 4, 6):
            assert torch.equal(call(shifted(q, off), out=shifted(q, off)), want)
    assert c.device_error() == 0
    c.close()


@pytest.mark.gpu
def test_queries_of_the_tcgen05_consumer(cuda_device):
    c = ripe.RipeCache(1, 1, 8, 1, 64, 1, 8, 300, 4)
    kv, q = torch.randn((1, 1, 100, 64), device="cuda").bfloat16(), torch.randn((1, 4, 8, 64), device="cuda").bfloat16()
    c.load_prefix(0, 0, [100], kv, kv)
    c.append_block(0, 0, kv[:, :, :4].transpose(1, 2).contiguous(), kv[:, :, 4:8].transpose(1, 2).contiguous())
    before = ripe.ripe_set_verify_consumer(ripe.RIPE_CONSUMER_TC)
    try:
        want = c.verify_attn(0, 0, q)
        assert torch.equal(c.verify_attn(0, 0, q, out=shifted(q, 2)), want)
        with pytest.raises(ripe.RipeError) as e:
            c.verify_attn(0, 0, shifted(q, 2))
        assert e.value.status == ripe.RIPE_EINVAL
    finally:
        ripe.ripe_set_verify_consumer(before)
    c.close()


@pytest.mark.parametrize("q_out", [1 << 22, (1 << 22) + 100 * 64 * 2 - 16, (1 << 22) - 2048 * 2 + 16, (1 << 23) + 64])
def test_queries_rotated_onto_a_table(q_out):
    """q_out [2][4][4][64] over any part of a table of 100 positions x 32 fp32."""
    view = ripe.CacheView(batch=2, layers=1, q_heads=4, kv_heads=2, head_dim=64, loops=2, window=8, max_T=100, max_B=4,
                          window_mode=0, block_len=4, k_ring=1 << 20, v_ring=2 << 20, lengths=4 << 20)
    rope = ripe.Rope(cos=1 << 22, sin=1 << 23, positions=100, rotary_dim=64, interleaved=0)
    vp = ctypes.c_void_p
    assert ripe.lib().ripe_append_rope_static(ctypes.byref(view), 0, 0, vp(4096), vp(8192), 128, vp(1 << 24), 256, vp(q_out),
                                              ctypes.byref(rope), vp(64), vp(0)) == ripe.RIPE_EINVAL
