"""Refusals of the newer calls that need no GPU: they are made on the host, before any device work."""
import ctypes

import pytest

from self_speculative_decode_b200 import ripe
from test_abi import test_alloc_rejects_bad_arguments_on_the_host as _alloc_cases

BAD_ALLOCS = _alloc_cases.pytestmark[0].args[1]


@pytest.mark.parametrize("args", BAD_ALLOCS)
def test_alloc_q8_refuses_what_alloc_refuses(args):
    h = ctypes.c_void_p(123)
    assert ripe.lib().ripe_cache_alloc_q8(*args, ctypes.byref(h)) == ripe.RIPE_EINVAL
    assert h.value is None


def test_null_handles():
    L, null = ripe.lib(), ctypes.c_void_p(0)
    rope = ripe.Rope(cos=64, sin=64, positions=8, rotary_dim=64, interleaved=0)
    assert L.ripe_cache_alloc_q8(1, 1, 2, 2, 64, 4, 16, 128, 4, 0, None) == ripe.RIPE_EINVAL
    assert L.ripe_cache_kv_bits(null) == ripe.RIPE_EINVAL
    assert L.ripe_set_scores(null, 1.0, None, null) == ripe.RIPE_EINVAL
    assert L.ripe_cache_export_q8(null, 0, 0, null, null, null, null, null) == ripe.RIPE_EINVAL
    assert L.ripe_append_block_rope(null, 0, 0, 1, null, null, 64, null, 0, null, ctypes.byref(rope), null) == ripe.RIPE_EINVAL
    assert L.ripe_rotate_block(null, 0, 1, null, 0, null, null, 0, null, ctypes.byref(rope), null) == ripe.RIPE_EINVAL
    assert L.ripe_append_rope_static(None, 0, 0, null, null, 64, null, 0, null, None, null, null) == ripe.RIPE_EINVAL


def _static(view=None, rope=None, layer=0, r=0, k=4096, v=8192, ld_kv=128, q=None, ld_q=0, q_out=None, error=64):
    """A call that a host check has to refuse: its addresses are made up, and are never read."""
    w = dict(batch=2, layers=1, q_heads=4, kv_heads=2, head_dim=64, loops=2, window=8, max_T=100, max_B=4, window_mode=0,
             block_len=4, k_ring=1 << 20, v_ring=2 << 20, lengths=4 << 20)
    w.update(view or {})
    t = None
    if rope is not None:
        a = dict(cos=1 << 22, sin=1 << 23, positions=100, rotary_dim=64, interleaved=0)
        a.update(rope)
        t = ctypes.byref(ripe.Rope(**a))
    vp = ctypes.c_void_p
    return ripe.lib().ripe_append_rope_static(ctypes.byref(ripe.CacheView(**w)), layer, r, vp(k), vp(v), ld_kv, vp(q or 0),
                                              ld_q, vp(q_out or 0), t, vp(error), vp(0))


@pytest.mark.parametrize("call", [
    dict(view=dict(batch=0)), dict(view=dict(batch=1025)), dict(view=dict(head_dim=80)), dict(view=dict(q_heads=3)),
    dict(view=dict(block_len=5)), dict(view=dict(block_len=0)), dict(view=dict(k_ring=None)), dict(view=dict(lengths=None)),
    dict(view=dict(v_ring=(2 << 20) + 8)), dict(view=dict(max_B=40, q_heads=4)), dict(layer=1), dict(layer=-1), dict(r=2),
    dict(k=None), dict(v=None), dict(error=None), dict(k=4096 + 2), dict(ld_kv=120), dict(ld_kv=132), dict(ld_kv=-128),
    dict(q=1 << 24), dict(q_out=1 << 24), dict(q=1 << 24, q_out=1 << 25, ld_q=248), dict(q=(1 << 24) + 4, q_out=1 << 25, ld_q=256),
    dict(q=1 << 24, q_out=(1 << 24) + 256, ld_q=256),                 # shifted onto itself
    dict(q=1 << 24, q_out=1 << 24, ld_q=512),                         # in place, but strided
    dict(q=1 << 24, q_out=4096, ld_q=256),                            # over the keys
    dict(rope=dict(cos=None)), dict(rope=dict(sin=None)), dict(rope=dict(positions=0)), dict(rope=dict(rotary_dim=0)),
    dict(rope=dict(rotary_dim=12)), dict(rope=dict(rotary_dim=72)), dict(rope=dict(rotary_dim=-8)),
    dict(rope=dict(interleaved=2)), dict(rope=dict(cos=(1 << 22) + 4)),
])
def test_append_rope_static_refuses(call):
    assert _static(**call) == ripe.RIPE_EINVAL
