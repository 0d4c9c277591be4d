"""What the newer operators cost: appending a draft block with the position rotation applied on the way, attention
over a cache whose deepest-plane region is held in 8 bits, and attention whose scores are capped or biased by distance.

Each case names one call as a decoder makes it. With ``own`` false ``run`` computes it in elementary torch operations
in 32 bits; with ``own`` true it calls the library (``self_speculative_decode_b200.ripe``). ``exact`` gives the same
outputs from the definitions in 64 bits.

Lengths of a ragged batch run evenly from T_lo to T_hi. Planes are N(0, 1) with plane r near the deepest one, as
looped models have them; queries are N(0, 1) * q_std / sqrt(head_dim), so that logits have a standard deviation of q_std.
"""
import math

import torch

own = False

BLOCK = 64      # tokens that share a scale in the 8-bit region
LOOPS = 4       # planes of the caches that the attention cases build
LOOP = 1        # the loop that is verified


# ------------------------------------------------------------------ cases
def _append(name, N, B, Hq, kvH, d, rot, pairs, T_lo, T_hi):
    c = dict(op="append", N=N, B=B, Hq=Hq, kvH=kvH, d=d, rot=rot, interleaved=pairs, T_lo=T_lo, T_hi=T_hi, W=64)
    return dict(c, name=name) if name else c


def _attention(name, N, B, Hq, kvH, d, W, T_lo, T_hi, bits, cap=0.0, bias=False, q_std=1.0, draft=False):
    c = dict(op="attention", N=N, B=B, Hq=Hq, kvH=kvH, d=d, W=W, T_lo=T_lo, T_hi=T_hi, bits=bits, cap=cap, bias=bias,
             q_std=q_std, draft=draft)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one token of one sequence on its way into the cache: a lone launch, where only latency counts
        _append("append, one token", 1, 1, 8, 2, 64, 64, False, 700, 700),
        # a draft block of the Huginn-shaped layer (55 heads x 96), pairs of neighbouring elements rotated
        _append("append, Huginn block", 1, 8, 55, 55, 96, 96, True, 1024, 1024),
        # an odd batch in a serving step; half of each head is rotated
        _append("append, 37 sequences", 37, 5, 32, 8, 128, 64, False, 3, 30000),
        # a full serving batch: memory bound
        _append("append, 512 sequences", 512, 8, 32, 8, 128, 128, False, 512, 8192),
        # the tiny check of the benchmark: almost everything lies in the window
        _attention("8 bits, tiny", 1, 4, 2, 2, 64, 16, 128, 128, 8),
        # the Huginn-shaped verification
        _attention("8 bits, Huginn", 1, 8, 55, 55, 96, 64, 1024, 1024, 8),
        # one drafted token for each of 16 sequences of uneven lengths
        _attention("8 bits, ragged draft step", 16, 1, 32, 8, 128, 64, 100, 8007, 8, draft=True),
        # the long-context GQA verification
        _attention("8 bits, long context", 8, 8, 32, 8, 128, 64, 32768, 32768, 8),
        # one drafted token with a distance bias: latency
        _attention("bias, draft step", 1, 1, 8, 8, 64, 16, 200, 200, 16, bias=True, draft=True),
        # the Huginn-shaped verification with capped scores
        _attention("cap, Huginn", 1, 8, 55, 55, 96, 64, 1024, 1024, 16, cap=30.0, q_std=8.0),
        # uneven lengths from an empty cache on, capped and biased at once
        _attention("cap and bias, ragged", 15, 6, 20, 4, 64, 32, 0, 5001, 16, cap=50.0, bias=True, q_std=4.0),
        # the long-context GQA verification with capped scores
        _attention("cap, long context", 8, 8, 32, 8, 128, 64, 32768, 32768, 16, cap=50.0, q_std=8.0),
    ]


def _between(rng, lo, hi):
    """A whole number in [lo, hi], spread evenly over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """More of the same: an append, an attention over the 8-bit cache or one with capped or biased scores."""
    kvH, g = rng.choice(((1, 8), (2, 1), (4, 5), (8, 4), (8, 1), (55, 1), (7, 3)))
    d = rng.choice((64, 96, 128))
    if rng.random() < 0.3:
        N, B = _between(rng, 1, 512), rng.randint(1, 8)
        lo = rng.randint(0, 2000)
        while N * B * kvH * (g + 2) * d > 512 * 8 * 48 * 128:
            N = max(1, N // 2)
        return _append(None, N, B, kvH * g, kvH, d, rng.choice((d, d, d // 2, 24)), rng.random() < 0.5, lo,
                       lo + _between(rng, 1, 8000))
    draft = rng.random() < 0.3
    B = 1 if draft else rng.randint(1, min(16, 64 // g))
    hi = _between(rng, 20, 32768)
    lo = rng.randint(0, hi)
    N = _between(rng, 1, 32)
    while N * (hi + B) * kvH * d > 8 * 32768 * 8 * 128 or N * kvH * (hi + B) * g * B > 8 * 8 * 32768 * 32:
        if N > 1:
            N //= 2
        else:
            hi //= 2
            lo = min(lo, hi)
    W = rng.choice((0, 8, 16, 64, 64, 200))
    bits = rng.choice((8, 8, 16))
    kind = rng.randint(0, 3) if bits == 8 else rng.randint(1, 3)
    cap = float(rng.choice((20, 30, 50))) if kind & 1 else 0.0
    return _attention(None, N, B, kvH * g, kvH, d, W, lo, hi, bits, cap, kind >= 2, rng.choice((1.0, 3.0, 8.0)), draft)


def _lengths(c):
    return [c["T_lo"] + (c["T_hi"] - c["T_lo"]) * n // max(1, c["N"] - 1) for n in range(c["N"])]


def work(case):
    c, T = case, _lengths(case)
    if c["op"] == "append":
        rows = c["N"] * c["B"]
        positions = len({t + j for t in T for j in range(c["B"])})
        read = 2 * rows * (c["Hq"] + 2 * c["kvH"]) * c["d"] + 4 * positions * c["rot"]
        return {"bytes": 2 * read - 4 * positions * c["rot"], "flops": 3 * rows * (c["Hq"] + c["kvH"]) * c["rot"]}
    g, size = c["Hq"] // c["kvH"], 0
    deep = flops = 0
    for t in T:
        D = max(0, t - c["W"])
        D8 = D // BLOCK * BLOCK if c["bits"] == 8 else 0
        # keys that some query takes at the deepest plane, and the window and the block at plane LOOP
        rest = min(t, max(0, t + c["B"] - 1 - c["W"])) - D8 + t + c["B"] - D
        deep += D8
        size += 2 * c["kvH"] * c["d"] * (D8 + 2 * rest) + (8 * c["kvH"] * D8 // BLOCK)
        flops += sum(4 * c["Hq"] * c["d"] * (t + j + 1) for j in range(c["B"]))
    rows = c["N"] * c["B"] * c["Hq"]
    size += rows * (4 * c["d"] + 4)
    if c["draft"]:
        size += 4 * c["N"] * c["kvH"] * c["d"]
    return {"bytes": size, "flops": flops}


# ------------------------------------------------------------------ inputs
def _normal(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)


def _append_inputs(c, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    N, B, d = c["N"], c["B"], c["d"]
    k, v, q = (_normal(gen, N, B, h, d).bfloat16() for h in (c["kvH"], c["kvH"], c["Hq"]))
    slots = c["W"] + B
    ring_k, ring_v = (_normal(gen, 1, N, 2, c["kvH"], slots, d).bfloat16() for _ in range(2))
    half = c["rot"] // 2
    rate = 10000.0 ** (-torch.arange(half, device="cuda", dtype=torch.float64) / half)
    angle = torch.arange(c["T_hi"] + B, device="cuda", dtype=torch.float64)[:, None] * rate
    lengths = torch.tensor(_lengths(c), device="cuda", dtype=torch.int32)
    return k, v, q, ring_k, ring_v, angle.cos().float(), angle.sin().float(), lengths


def _attention_inputs(c, seed):
    """The planes R - 1 and LOOP of every position up to the end of the block, and the queries."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    shape = (c["N"], c["kvH"], c["T_hi"] + c["B"], c["d"])
    planes = []
    for _ in range(2):
        top = _normal(gen, *shape)
        planes += [top.bfloat16(), top.add_(_normal(gen, *shape), alpha=0.88 ** LOOP).bfloat16()]
    q = (_normal(gen, c["N"], c["B"], c["Hq"], c["d"]) * (c["q_std"] / math.sqrt(c["d"]))).bfloat16()
    return planes[0], planes[1], planes[2], planes[3], q


def _slopes(c):
    return [2.0 ** (-8.0 * (h + 1) / c["Hq"]) for h in range(c["Hq"])]


def _rows(plane, start, count):
    """Rows [start_n, start_n + count) of a plane [N][kvH][len][d]; past the end, the last row."""
    at = (start[:, None] + torch.arange(count, device="cuda")).clamp(max=plane.shape[2] - 1)
    return plane.gather(2, at[:, None, :, None].expand(-1, plane.shape[1], -1, plane.shape[3]))


def _quantised(x):
    """Signed 8-bit values and one scale for each 64 tokens of a head, of x [N][kvH][blocks * 64][d]."""
    y = x.float().reshape(*x.shape[:2], -1, BLOCK, x.shape[3])
    scale = (y.abs().amax((3, 4)) / 127).clamp(min=2.0 ** -80)
    return (y / scale[..., None, None]).round().to(torch.int8).reshape(x.shape), scale


def prepare(case, seed):
    c = case
    if c["op"] == "append":
        k, v, q, ring_k, ring_v, cos, sin, lengths = _append_inputs(c, seed)
        s = dict(c=c, k=k, v=v, q=q, ring_k=ring_k, ring_v=ring_v, cos=cos, sin=sin, lengths=lengths, q_out=torch.empty_like(q))
        if own:
            from self_speculative_decode_b200 import ripe

            s["table"] = ripe.RotaryTable(cos, sin, interleaved=c["interleaved"])
            s["view"] = ripe.CacheView(batch=c["N"], layers=1, q_heads=c["Hq"], kv_heads=c["kvH"], head_dim=c["d"], loops=2,
                                       window=c["W"], max_T=c["T_hi"] + 1000, max_B=c["B"], window_mode=0, block_len=c["B"],
                                       k_ring=ring_k.data_ptr(), v_ring=ring_v.data_ptr(), lengths=lengths.data_ptr())
            s["error"] = torch.zeros(1, dtype=torch.int32, device="cuda")
        return s
    kt, kr, vt, vr, q = _attention_inputs(c, seed)
    T, B, W = _lengths(c), c["B"], c["W"]
    s = dict(c=c, q=q)
    Td = torch.tensor(T, device="cuda")
    kb, vb = (_rows(x, Td, B).transpose(1, 2).contiguous() for x in (kr, vr))
    if own:
        from self_speculative_decode_b200.ripe import RipeCache

        cache = RipeCache(c["N"], 1, c["Hq"], c["kvH"], c["d"], LOOPS, W, c["T_hi"] + B, B, kv_bits=c["bits"])
        cache.load_prefix(0, LOOPS - 1, T, kt, vt)
        cache.load_prefix(0, LOOP, T, kr, vr)
        if c["cap"] or c["bias"]:
            cache.set_scores(softcap=c["cap"], slopes=_slopes(c) if c["bias"] else None)
        if not c["draft"]:
            cache.append_block(0, LOOP, kb, vb)
        s.update(cache=cache, k=kb, v=vb, lse=torch.empty(q.shape[:3], device="cuda"))
        return s
    # as stored: the deepest plane of [0, D) (in 8 bits: whole blocks of 64), the deepest plane of [D, T) beside it,
    # and plane LOOP of the window and the block
    unit = BLOCK if c["bits"] == 8 else 1
    D = (Td - W).clamp(min=0) // unit * unit
    most = int(max(0, c["T_hi"] - W) // unit * unit)
    lo = (Td - W).clamp(min=0)
    s["deep"] = [_quantised(x[:, :, :most]) if unit > 1 else (x[:, :, :most].contiguous(), None) for x in (kt, vt)]
    s["top"] = [_rows(x, D, W + unit - 1) for x in (kt, vt)]
    s["ring"] = [_rows(x, lo, W + B) for x in (kr, vr)]
    s.update(T=Td, D=D, lo=lo, most=most, slopes=torch.tensor(_slopes(c), device="cuda"), block=(kb, vb))
    return s


# ------------------------------------------------------------------ one pass
def _turned(x, cos, sin, interleaved):
    """x [N][B][heads][d] with its first 2 * cos.shape[-1] elements of each head rotated; cos, sin [N][B][1][half]."""
    half = cos.shape[-1]
    x = x.float()
    head, rest = x[..., : 2 * half], x[..., 2 * half:]
    if interleaved:
        a, b = head[..., 0::2], head[..., 1::2]
        head = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = head[..., :half], head[..., half:]
        head = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((head, rest), -1).bfloat16()


def _plain_append(s):
    c, T = s["c"], s["lengths"].long()
    at = T[:, None] + torch.arange(c["B"], device="cuda")
    cos, sin = s["cos"][at][:, :, None], s["sin"][at][:, :, None]
    slot, n = at % s["ring_k"].shape[4], torch.arange(c["N"], device="cuda")[:, None]
    s["ring_k"][0, n, LOOP, :, slot] = _turned(s["k"], cos, sin, c["interleaved"])
    s["ring_v"][0, n, LOOP, :, slot] = s["v"]
    s["q_out"].copy_(_turned(s["q"], cos, sin, c["interleaved"]))


def _stored(part):
    values, scale = part
    return values.float() if scale is None else values.float() * scale.repeat_interleave(BLOCK, 2)[..., None]


def _plain_attention(s):
    c = s["c"]
    N, B, Hq, kvH, d, W = (c[x] for x in ("N", "B", "Hq", "kvH", "d", "W"))
    step = torch.arange(B, device="cuda")
    if c["draft"]:  # the drafted token's own row goes into the ring first
        at = (s["T"] - s["lo"])[:, None, None, None].expand(-1, kvH, 1, d)
        s["ring"] = [x.scatter(2, at, b.transpose(1, 2)) for x, b in zip(s["ring"], s["block"])]
    k, v = (torch.cat((_stored(s["deep"][i]), s["top"][i].float(), s["ring"][i].float()), 2) for i in range(2))
    p = s["T"][:, None] + step
    t0 = torch.arange(s["most"], device="cuda").expand(N, -1)
    t1 = s["D"][:, None] + torch.arange(s["top"][0].shape[2], device="cuda")
    t2 = s["lo"][:, None] + torch.arange(W + B, device="cuda")
    t = torch.cat((t0, t1, t2), 1)[:, None]
    old = (t < p[..., None] - W) & (t < s["T"][:, None, None])
    near = (t >= p[..., None] - W) & (t <= p[..., None])
    seen = torch.cat((old[..., : s["most"]] & (t0[:, None] < s["D"][:, None, None]),
                      old[..., s["most"]: s["most"] + t1.shape[1]], (near | (t >= s["T"][:, None, None]) & (t <= p[..., None]))[..., -t2.shape[1]:]), -1)
    q = s["q"].float().reshape(N, B, kvH, Hq // kvH, d).permute(0, 2, 1, 3, 4).reshape(N, kvH, -1, d)
    x = (q @ k.transpose(2, 3)).reshape(N, kvH, B, Hq // kvH, -1)
    if c["cap"]:
        x = c["cap"] * torch.tanh(x / c["cap"])
    if c["bias"]:
        x = x + s["slopes"].reshape(kvH, 1, -1, 1) * (t - p[..., None]).float()[:, None, :, None]
    x = x.masked_fill(~seen[:, None, :, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    w = (x - top).exp()
    total = w.sum(-1, keepdim=True)
    out = (w / total).reshape(N, kvH, -1, x.shape[-1]) @ v
    lse = (top + total.log()).squeeze(-1).permute(0, 2, 1, 3).reshape(N, B, Hq)
    return out.reshape(N, kvH, B, Hq // kvH, d).permute(0, 2, 1, 3, 4).reshape(N, B, Hq, d).bfloat16(), lse


def run(state):
    s = state
    if s["c"]["op"] == "append":
        if own:
            from self_speculative_decode_b200 import ripe

            ripe.append_rope_static(s["view"], 0, LOOP, s["k"], s["v"], s["q"], s["table"], q_out=s["q_out"], device_error=s["error"])
        else:
            _plain_append(s)
        return {"q": s["q_out"], "k_ring": s["ring_k"], "v_ring": s["ring_v"]}
    if own:
        if s["c"]["draft"]:
            out = s["cache"].draft_attn(0, LOOP, 0, s["k"], s["v"], s["q"], lse=s["lse"])
        else:
            out = s["cache"].verify_attn(0, LOOP, s["q"], lse=s["lse"])
        return {"out": out, "lse": s["lse"]}
    out, lse = _plain_attention(s)
    return {"out": out, "lse": lse}


# ------------------------------------------------------------------ the definitions, in 64 bits
def _exact_append(c, seed):
    k, v, q, ring_k, ring_v, cos, sin, lengths = _append_inputs(c, seed)
    half = c["rot"] // 2
    first = torch.arange(half, device="cuda") * (2 if c["interleaved"] else 1)
    second = first + (1 if c["interleaved"] else half)
    at = lengths.long()[:, None] + torch.arange(c["B"], device="cuda")
    z = torch.complex(cos[at].double(), sin[at].double())[:, :, None]
    turned = []
    for x in (k.double(), q.double()):
        y = torch.complex(x[..., first], x[..., second]) * z
        x[..., first], x[..., second] = y.real, y.imag
        turned.append(x)
    out = {"q": turned[1], "k_ring": ring_k.double(), "v_ring": ring_v.double()}
    for n, T in enumerate(_lengths(c)):
        for j in range(c["B"]):
            out["k_ring"][0, n, LOOP, :, (T + j) % ring_k.shape[4]] = turned[0][n, j]
            out["v_ring"][0, n, LOOP, :, (T + j) % ring_k.shape[4]] = v[n, j].double()
    return out


def _exact_deep(x, D, bits):
    """The deepest plane x [kvH][T][d] as the cache holds it, in 64 bits: positions before D in whole blocks of 8-bit values."""
    y = x.double()
    if bits == 8 and D:
        b = y[:, :D].reshape(y.shape[0], D // BLOCK, -1)
        unit = (b.abs().max(2, keepdim=True).values.float() / 127).clamp(min=2.0 ** -80).double()
        y[:, :D] = ((b / unit).float().round().double() * unit).reshape(y.shape[0], D, -1)
    return y


def exact(case, seed):
    c = case
    if c["op"] == "append":
        return _exact_append(c, seed)
    kt, kr, vt, vr, q = _attention_inputs(c, seed)
    kvH, g, W = c["kvH"], c["Hq"] // c["kvH"], c["W"]
    if c["N"] * c["B"] * kvH * c["d"] * c["T_hi"] > 1 << 34:
        return None
    slope = torch.tensor(_slopes(c), device="cuda", dtype=torch.float64).reshape(kvH, g, 1)
    out = torch.empty(q.shape, device="cuda", dtype=torch.float64)
    lse = torch.empty(q.shape[:3], device="cuda", dtype=torch.float64)
    for n, T in enumerate(_lengths(c)):
        D = max(0, T - W) // BLOCK * BLOCK
        deep = [_exact_deep(x[n, :, :T], D, c["bits"]) for x in (kt, vt)]
        for j in range(c["B"]):
            p = T + j
            cut = min(T, max(0, p - W))  # keys before the cut at the deepest plane, from it on at the verified loop
            K, V = (torch.cat((a[:, :cut], b[n, :, cut: p + 1].double()), 1) for a, b in zip(deep, (kr, vr)))
            x = torch.einsum("hgd,htd->hgt", q[n, j].double().reshape(kvH, g, -1), K)
            if c["cap"]:
                x = torch.tanh(x / c["cap"]) * c["cap"]
            if c["bias"]:
                x = x - slope * (p - torch.arange(p + 1, device="cuda", dtype=torch.float64))
            lse[n, j] = torch.logsumexp(x, 2).reshape(-1)
            out[n, j] = torch.einsum("hgt,htd->hgd", torch.softmax(x, 2), V).reshape(c["Hq"], -1)
    return {"out": out, "lse": lse}
