"""A plain 64-bit implementation of what the newer calls compute, and a GPU cache beside it.

``Pair`` draws every plane of every position once (each plane its own N(0, 1), so that a wrong plane moves a result by
O(1)) and drives a ``RipeCache`` with it.  ``Pair.expect`` computes a query row from the definition: the keys t <= p at
the plane of the oracle's rule, 8-bit blocks as the stated rule quantises them, scores capped and biased, softmax, sum.

Tolerances follow from the roundings of the kernels (half a step relative to the value: bf16 2^-8, f16 2^-11, fp32 2^-24).
With w the weights, A = sum w |V - out| and B = sum w |V|:
  * the output is rounded to bf16: 2^-8 |out|;
  * bf16 probabilities, normalised by the sum of the rounded ones: 2^-8 A; f16 ones, normalised by the exact sum: 2^-11 B;
  * a score is off by at most eps = d 2^-23 sum |scale q k| (fp32 sums of d products, one rounding an addition) +
    2^-21 cap (two approximate steps of 2^-22 and a rounding, times the cap) + 2^-21 max|x| (its own roundings and those
    of the exponent), which moves a weight by 2 eps relative: 2 eps B; 2^-18 B for the approximate exponential and the sums
    over a few thousand keys;
  * the log-sum-exp moves by eps + 2^-18 + 2^-22 |lse|.
"""
import numpy as np
import torch

from oracle import ripe_oracle as orc
from self_speculative_decode_b200 import synth
from self_speculative_decode_b200.ripe import RipeCache

F32 = np.float32


def quantised(x):
    """Blocks of 64 tokens of x [heads][64 * n][d] (float64 holding bf16 values): int8 u and fp32 scales [heads][n]."""
    b = x.astype(F32).reshape(x.shape[0], -1, 64, x.shape[2])
    s = np.maximum((np.abs(b).max((2, 3)) * (F32(1) / F32(127))).astype(F32), F32(2.0 ** -80))
    return np.rint(b / s[:, :, None, None]).astype(np.int8).reshape(x.shape), s


def bits_dev(bits):
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).cuda().view(torch.bfloat16)


class Pair:
    def __init__(self, N, Hq, kvH, d, R, W, T, max_B, bits=8, mode=0, cap=0.0, slopes=None, room=0, seed=0, scale=1.0,
                 q_std=1.0, L=1):
        self.N, self.Hq, self.kvH, self.d, self.R, self.g = N, Hq, kvH, d, R, Hq // kvH
        self.T = [int(t) for t in (T if hasattr(T, "__len__") else [T] * N)]
        self.max_T = max(self.T) + max_B + room
        self.W, self.max_B, self.bits, self.mode = min(W, self.max_T), max_B, bits, mode
        self.cap, self.slopes, self.scale, self.q_std, self.seed, self.L = cap, slopes, scale, q_std, seed, L
        self.planes = []  # [layer][plane] = (K, V) as bf16 bits [N][kvH][max_T][d]
        for layer in range(L):
            src = synth.PlaneSource(N, kvH, d, R, self.max_T, 0.88, seed, layer=layer, independent=True)
            self.planes.append([(src.plane(r, "K"), src.plane(r, "V")) for r in range(R)])
        self.gpu = RipeCache(N, L, Hq, kvH, d, R, W, self.max_T, max_B, mode, kv_bits=bits)
        if cap or slopes is not None:
            self.gpu.set_scores(cap, slopes)
        self.step = 0

    def load(self):
        for layer in range(self.L):
            for r, (k, v) in enumerate(self.planes[layer]):
                self.gpu.load_prefix(layer, r, self.T, bits_dev(k), bits_dev(v))
        return self

    def rows(self, layer, r, j, B):
        """k, v [N][B][kvH][d] of positions T_n + j onward, as bf16 bits."""
        return tuple(np.stack([x[n, :, self.T[n] + j: self.T[n] + j + B].transpose(1, 0, 2) for n in range(self.N)])
                     for x in self.planes[layer][r])

    def append(self, B, loops=None):
        for layer in range(self.L):
            for r in range(self.R) if loops is None else loops:
                self.gpu.append_block(layer, r, *map(bits_dev, self.rows(layer, r, 0, B)))
        return self

    def commit(self, accepted):
        self.gpu.commit(accepted)
        self.T = [t + a for t, a in zip(self.T, accepted)]

    def queries(self, B):
        self.step += 1
        rng = np.random.default_rng([self.seed, 77, self.step])
        x = rng.standard_normal((self.N, B, self.Hq, self.d)) * (self.q_std / np.sqrt(self.d))
        return synth.f32_to_bf16_bits(x.astype(F32))

    def D(self, n):
        A = max(0, self.T[n] - self.W)
        return A // 64 * 64 if self.bits == 8 else A

    def expect(self, q, n, j, r, layer=0, sink=0, window=None):
        """Query row q [Hq][d] (bf16 bits) of position T_n + j at loop r: out [Hq][d], its tolerance, lse [Hq], its own."""
        T = self.T[n]
        p = T + j
        ts = np.array([t for t in range(p + 1) if window is None or t < sink or t >= p - window])
        plane = np.array([orc.plane_of(p, int(t), r, self.R, T, self.W, self.mode) for t in ts])
        kv = []
        for w in range(2):
            x = np.zeros((self.kvH, p + 1, self.d))
            for pl in set(plane):
                at = ts[plane == pl]
                x[:, at] = synth.bf16_bits_to_f32(self.planes[layer][pl][w][n][:, at])
            D = self.D(n)
            if self.bits == 8 and D:
                # the deepest plane of whole blocks, where the rule reads the deepest plane
                u, s = quantised(synth.bf16_bits_to_f32(self.planes[layer][self.R - 1][w][n][:, :D]).astype(np.float64))
                deq = u.astype(np.float64) * np.repeat(s.astype(np.float64), 64, 1)[:, :, None]
                at = ts[(plane == self.R - 1) & (ts < D)]
                x[:, at] = deq[:, at]
            kv.append(np.repeat(x[:, ts], self.g, 0))
        qf = synth.bf16_bits_to_f32(q).astype(np.float64)
        x = self.scale * np.einsum("hd,htd->ht", qf, kv[0])
        eps = self.d * 2.0 ** -23 * abs(self.scale) * np.einsum("hd,htd->ht", abs(qf), abs(kv[0])).max(1)
        if self.cap:
            x = self.cap * np.tanh(x / self.cap)
            eps += 2.0 ** -21 * self.cap
        if self.slopes is not None:
            x = x - np.asarray(self.slopes, np.float64)[:, None] * (p - ts)
        eps += 2.0 ** -21 * abs(x).max(1)
        m = x.max(1, keepdims=True)
        w = np.exp(x - m)
        lse = m[:, 0] + np.log(w.sum(1))
        w /= w.sum(1, keepdims=True)
        out = np.einsum("ht,htd->hd", w, kv[1])
        A = np.einsum("ht,htd->hd", w, abs(kv[1] - out[:, None]))
        Bs = np.einsum("ht,htd->hd", w, abs(kv[1]))
        tol = 2.0 ** -8 * (abs(out) + A) + (2.0 ** -11 + 2 * eps[:, None] + 2.0 ** -18) * Bs
        return out, tol, lse, eps + 2.0 ** -18 + 2.0 ** -22 * abs(lse)

    def check(self, out, lse, q, loops, j0=0, layer=0, sink=0, window=None, rows=None):
        """out [N][B][Hq][d] and lse of queries q against expect, for rows (n, i) or all."""
        got, gl = out.double().cpu().numpy(), lse.double().cpu().numpy()
        for n in range(self.N):
            for i in range(q.shape[1]):
                if rows is not None and (n, i) not in rows:
                    continue
                r = loops[i] if hasattr(loops, "__len__") else loops
                eo, to, el, tl = self.expect(q[n, i], n, j0 + i, r, layer, sink, window)
                bad = ~(abs(got[n, i] - eo) <= to)
                assert not bad.any(), (n, i, float(abs(got[n, i] - eo).max()), float((abs(got[n, i] - eo) / to).max()))
                assert (abs(gl[n, i] - el) <= tl).all(), (n, i, float(abs(gl[n, i] - el).max()), float(tl.min()))

    def lse(self, B):
        return torch.full((self.N, B, self.Hq), float("nan"), device="cuda")

    def verify(self, r, B, layer=0, rows=None):
        q, lse = self.queries(B), self.lse(B)
        out = self.gpu.verify_attn(layer, r, bits_dev(q), lse=lse, scale=self.scale)
        self.check(out, lse, q, r, layer=layer, rows=rows)
        return out, lse

    def wave(self, loops, rows=None):
        q, lse = self.queries(len(loops)), self.lse(len(loops))
        out = self.gpu.verify_attn_wave(0, loops, bits_dev(q), lse=lse, scale=self.scale)
        self.check(out, lse, q, loops, rows=rows)

    def draft(self, r, j, sink=None, window=None):
        q, lse = self.queries(1), self.lse(1)
        k, v = map(bits_dev, self.rows(0, r, j, 1))
        out = self.gpu.draft_attn(0, r, j, k, v, bits_dev(q), lse=lse, scale=self.scale, sink=sink, window=window)
        if sink is None and window is None:
            self.check(out, lse, q, r, j0=j)
        else:
            self.check(out, lse, q, r, j0=j, sink=sink or 0, window=window)

    def close(self):
        assert self.gpu.device_error() == 0
        self.gpu.close()
