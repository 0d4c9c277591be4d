"""The tile plan of the attention over 8-bit caches and with capped or biased scores (csrc/ripe_score.cuh), and the
byte order of an 8-bit block, on the host.

For every query of a call, the keys that it sees over all tiles are compared with the keys t <= p that it attends to
(all of them, or a draft's sink and window), each exactly once and at the plane of the oracle's rule; every tile is one
box of consecutive rows inside its region, and an 8-bit tile whole blocks of it."""
import os
import random
import shutil
import subprocess

import pytest

from oracle import ripe_oracle as orc

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
KDEEP, KRING, KDUAL = 0, 1, 2


@pytest.fixture(scope="module")
def dump_exe(tmp_path_factory):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("nvcc not found")
    exe = str(tmp_path_factory.mktemp("plan") / "score_plan_dump")
    subprocess.run([nvcc, "-std=c++17", "-gencode", "arch=compute_100a,code=sm_100a",
                    "-I", os.path.join(ROOT, "include"),
                    "-I", os.path.join(ROOT, "self_speculative_decode_b200", "csrc"),
                    "-o", exe, os.path.join(ROOT, "tests", "score_plan_dump.cu")],
                   check=True, capture_output=True, timeout=600)
    return exe


def _cases():
    rng = random.Random(5)
    out = []
    for unit in (1, 64):
        for _ in range(150):
            R = rng.choice((1, 2, 4))
            W = rng.choice((0, 1, 7, 16, 64, 100, 5000))
            max_B = rng.choice((1, 4, 16))
            T = rng.choice((0, 1, 5, 63, 64, 65, 127, 200, 333, 517))
            max_T = T + max_B + rng.choice((0, 1, 40, 300))
            mode = rng.randint(0, 1)
            kind = rng.randint(0, 3)
            wide = rng.randint(0, 1) if unit > 1 else 0  # smaller tiles, for more than 16 query rows
            if kind < 2:  # one loop
                B = rng.randint(1, max_B)
                out.append((T, W, R, max_T, max_B, mode, unit, wide, B, 0, B, 0, -1, [rng.randrange(R)]))
            elif kind == 2:  # a loop per position
                B = rng.randint(1, max_B)
                out.append((T, W, R, max_T, max_B, mode, unit, wide, B, 0, B, 0, -1, [rng.randrange(R) for _ in range(B)]))
            else:  # a draft step
                j = rng.randrange(max_B)
                sink, window = rng.choice(((0, -1), (0, 0), (4, 30), (100, 10), (64, 64), (1 << 30, 5), (3, 1 << 30)))
                out.append((T, W, R, max_T, max_B, mode, unit, wide, j + 1, j, 1, sink, window, [rng.randrange(R)]))
    return out


def test_every_query_sees_its_keys_once_at_their_plane(dump_exe):
    cases = _cases()
    text = "\n".join(" ".join(map(str, (*c[:13], len(c[13]), *c[13]))) for c in cases) + "\n"
    lines = iter(subprocess.run([dump_exe], input=text, capture_output=True, text=True, check=True,
                                timeout=120).stdout.splitlines())
    for c in cases:
        T, W, R, max_T, max_B, mode, unit, wide, B, j0, qB, sink, window, loops = c
        Wc = min(W, max_T)
        D = max(0, T - Wc) // unit * unit
        S, deep_rows = map(int, next(lines).split())
        assert S >= min(T - D + B, max_T) and deep_rows >= D
        seen = [{} for _ in range(qB)]
        total = 0
        while True:
            f = next(lines).split()
            if f[0] == "E":
                assert int(f[1]) == total
                break
            total += 1
            kind, t0, cnt, y, plane = map(int, f[:5])
            assert cnt >= 1 and t0 >= 0
            if kind == KDEEP:
                assert y == t0 and t0 + cnt <= D and plane == R - 1
                assert cnt <= (128 if unit > 1 and not wide else 64)
                assert unit == 1 or (t0 % 64 == 0 and cnt % 64 == 0)
            else:
                assert cnt <= (32 if wide else 64) and t0 >= D and t0 + cnt <= (T if kind == KDUAL else T + B), c
                assert 0 <= y and y + cnt <= S and y == t0 % S
            for q in range(qB):
                for i, bit in enumerate(f[5 + q]):
                    if bit == "1":
                        assert t0 + i not in seen[q], (c, kind, t0 + i)
                        seen[q][t0 + i] = plane
        for q in range(qB):
            p, r = T + j0 + q, loops[(j0 + q) % len(loops)]
            want = {t: orc.plane_of(p, t, r, R, T, Wc, mode) for t in range(p + 1)
                    if window < 0 or t < sink or t >= p - window}
            assert seen[q] == want, c


def test_every_element_of_a_block_has_a_byte_of_its_own(dump_exe):
    out = subprocess.run([dump_exe, "offsets"], capture_output=True, text=True, check=True, timeout=120).stdout
    k, v = {}, {}
    for line in out.splitlines():
        d, _, _, ko, vo = map(int, line.split())
        k.setdefault(d, set()).add(ko)
        v.setdefault(d, set()).add(vo)
    for d in (64, 96, 128):
        assert k[d] == v[d] == set(range(64 * d))
