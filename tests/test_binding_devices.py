"""The binding refuses tensors on another device than the cache's before it calls the library (no GPU: tensors that claim
a device, and library calls that are only recorded)."""
import pytest
import torch

from self_speculative_decode_b200 import ripe

N, B, HQ, KVH, D = 2, 3, 4, 2, 64
CALLS = ("ripe_load_prefix", "ripe_append_block", "ripe_append_block_rope", "ripe_rotate_block", "ripe_verify_attn",
         "ripe_append_verify", "ripe_draft_attn", "ripe_draft_attn_window", "ripe_verify_attn_wave", "ripe_commit_device",
         "ripe_cache_export", "ripe_cache_export_q8")


class On(torch.Tensor):
    """A tensor that says it is on CUDA device `number`."""
    number = 0
    is_cuda = True

    def get_device(self):
        return self.number


def on(number, *shape, dtype=torch.bfloat16):
    t = torch.zeros(shape, dtype=dtype).as_subclass(On)
    t.number = number
    return t


@pytest.fixture
def cache(monkeypatch):
    calls = []
    for name in CALLS:
        monkeypatch.setattr(ripe, name, lambda *a, _name=name, **kw: calls.append((_name, a)))
    ripe._load_torch()
    c = object.__new__(ripe.RipeCache)
    c.N, c.L, c.Hq, c.kvH, c.d, c.R, c.W, c.max_T, c.max_B, c.mode = N, 1, HQ, KVH, D, 2, 8, 500, B, 0
    c.kv_bits, c.device, c.handle, c.calls = 8, 1, None, calls
    return c


def arguments():
    """Per call: its name, a function of the cache and the tensors, and the tensors' shapes and types."""
    kv, q, kv1, q1, lse = (N, B, KVH, D), (N, B, HQ, D), (N, 1, KVH, D), (N, 1, HQ, D), (N, B, HQ)
    f32 = dict(dtype=torch.float32)
    table = lambda cos, sin: ripe.RotaryTable(cos, sin)
    return [
        ("load_prefix", lambda c, k, v: c.load_prefix(0, 0, [9, 9], k, v, stream=1), [((N, KVH, 9, D), {})] * 2),
        ("append_block", lambda c, k, v: c.append_block(0, 0, k, v, stream=1), [(kv, {})] * 2),
        ("verify_attn", lambda c, q_, o, l: c.verify_attn(0, 0, q_, out=o, lse=l, stream=1), [(q, {}), (q, {}), (lse, f32)]),
        ("append_verify", lambda c, k, v, q_, o, l: c.append_verify(0, 0, k, v, q_, out=o, lse=l, stream=1),
         [(kv, {}), (kv, {}), (q, {}), (q, {}), (lse, f32)]),
        ("draft_attn", lambda c, k, v, q_, o, l: c.draft_attn(0, 0, 0, k, v, q_, out=o, lse=l, stream=1),
         [(kv1, {}), (kv1, {}), (q1, {}), (q1, {}), ((N, 1, HQ), f32)]),
        ("draft_attn window", lambda c, k, v, q_, o, l: c.draft_attn(0, 0, 0, k, v, q_, out=o, lse=l, stream=1, sink=4),
         [(kv1, {}), (kv1, {}), (q1, {}), (q1, {}), ((N, 1, HQ), f32)]),
        ("verify_attn_wave", lambda c, q_, o, l: c.verify_attn_wave(0, [0, 1, 0], q_, out=o, lse=l, stream=1),
         [(q, {}), (q, {}), (lse, f32)]),
        ("commit_device", lambda c, a: c.commit_device(a, stream=1), [((N,), dict(dtype=torch.int32))]),
        ("append_block_rope", lambda c, k, v, q_, o, a, b: c.append_block_rope(0, 0, k, v, table(a, b), q_, o, stream=1),
         [(kv, {}), (kv, {}), (q, {}), (q, {}), ((500, 32), f32), ((500, 32), f32)]),
        ("rotate_block", lambda c, k, q_, ko, qo, a, b: c.rotate_block(0, table(a, b), k, q_, ko, qo, stream=1),
         [(kv, {}), (q, {}), (kv, {}), (q, {}), ((500, 32), f32), ((500, 32), f32)]),
    ]


@pytest.mark.parametrize("name,call,shapes", arguments(), ids=[a[0] for a in arguments()])
def test_tensors_of_another_device_are_refused(cache, name, call, shapes):
    call(cache, *(on(1, *s, **kw) for s, kw in shapes))
    assert len(cache.calls) == 1
    for odd in range(len(shapes)):
        with pytest.raises(ValueError):
            call(cache, *(on(0 if i == odd else 1, *s, **kw) for i, (s, kw) in enumerate(shapes)))
    assert len(cache.calls) == 1


@pytest.mark.parametrize("f", ["export", "export_q8"])
def test_exports_are_allocated_on_the_device_of_the_cache(cache, monkeypatch, f):
    """Whatever device is current."""
    made = []

    def make(shape, dtype=None, device=None):
        made.append(device)
        return torch.Tensor(0)

    monkeypatch.setattr(cache, "stats", lambda: dict(lengths_synced=1, block_len=0), raising=False)
    monkeypatch.setattr(cache, "sync_lengths", lambda stream=None: [200, 200], raising=False)
    for name in ("empty", "zeros"):
        monkeypatch.setattr(torch, name, make)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(cache, "_on", lambda stream: 1, raising=False)
    getattr(cache, f)(0, 0)
    assert len(cache.calls) == 1 and made and all(d == torch.device("cuda", 1) for d in made)
