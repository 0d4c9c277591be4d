"""How the attention over 8-bit caches and with capped or biased scores cuts the heads' tile lists into CTAs, on the host.

Every tile of every head belongs to one CTA, in order; the CTAs that a head's merge counts are those that hold its
tiles; only a CTA's first and last head are shared; and the slots of the partial results (CTA + head) are unique and lie
in the scratch of SMs + heads slots."""
import os
import random
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SMS = 148


def _cases():
    rng = random.Random(11)
    out = []
    for i in range(700):
        q8 = rng.randint(0, 1)
        rows = rng.choice((1, 8, 9, 16, 17, 32))
        wide = int(q8 and rows > 16)
        groups = rng.choice((1, 2)) if rows > 16 else 1
        kvH = rng.choice((1, 1, 2, 3, 8, 55))
        N = rng.choice((1, 1, 2, 3, 16, 40, 300))
        grid = rng.choice((1, 2, 17, 100, SMS, SMS, SMS, SMS))
        W, B, R = rng.choice((0, 5, 16, 64, 200)), rng.randint(1, 16), rng.choice((1, 2, 4))
        most = rng.choice((0, 3, 70, 500, 3000, 40000 if N * kvH < 200 else 3000))
        T = [rng.randint(0, most) for _ in range(N)]
        if rng.random() < 0.5:
            T = [most] * N
        draft = rng.random() < 0.2
        loop = rng.randrange(R) if draft or rng.random() < 0.7 else -1
        sink, window = (rng.choice((0, 4, 100)), rng.choice((0, 30, 1000))) if draft else (0, -1)
        out.append((q8, wide, rows, kvH, groups, grid, W, B, R, max(T) + 16 + rng.choice((0, 50)), 16, loop, sink, window, N, *T))
    return out


def test_every_tile_has_one_cta_and_every_merge_its_partials(tmp_path):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("nvcc not found")
    exe = str(tmp_path / "score_chunk_dump")
    subprocess.run([nvcc, "-std=c++17", "-gencode", "arch=compute_100a,code=sm_100a", "-I", os.path.join(ROOT, "include"),
                    "-I", os.path.join(ROOT, "self_speculative_decode_b200", "csrc"), "--expt-relaxed-constexpr",
                    "-o", exe, os.path.join(ROOT, "tests", "score_chunk_dump.cu")], check=True, capture_output=True, timeout=600)
    cases = _cases()
    text = "".join(" ".join(map(str, c)) + "\n" for c in cases)
    lines = iter(subprocess.run([exe], input=text, capture_output=True, text=True, check=True, timeout=300).stdout.splitlines())
    split = 0
    for c in cases:
        heads = c[3] * c[4]
        totals = [int(x) for x in next(lines).split()[1:]]
        holders, ctas, parts = {}, [], []
        for line in lines:
            if line == "E":
                break
            (ctas if line[0] == "C" else parts).append([int(x) for x in line.split()[1:]])
        p, lt = 0, 0  # the next tile in order
        for cta, (p_first, at, p_last, ntiles) in enumerate(ctas):
            if ntiles <= 0:
                continue
            assert (p_first, at) == (p, lt), c
            for _ in range(ntiles):
                holders.setdefault(p, []).append(cta)
                last = p
                lt += 1
                if lt == totals[p // heads]:
                    p, lt = p + 1, 0
            assert p_last == last, c
        assert p == len(parts) == len(totals) * heads and lt == 0, c
        slots = set()
        for h, (first, count) in enumerate(parts):
            have = sorted(set(holders[h]))
            assert have == list(range(first, first + count)), (c, h)
            if count > 1:
                split += 1
                for cta in have:
                    assert cta + h not in slots and cta + h < SMS + len(parts), (c, h)
                    slots.add(cta + h)
                    assert h in (ctas[cta][0], ctas[cta][2]), (c, h)  # shared: the CTA's first or last head
    assert split > 100
