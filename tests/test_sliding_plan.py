"""The plan of the sliding decodes, made on the host with the kernel's own functions:
whatever the batch, and with every quotient of the plan off by two units in its last
place, the pieces' partial results have places of their own in the workspace."""
import os
import random
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
PKG = os.path.join(os.path.dirname(HERE), "paged_kv_decode_25_gb300")


@pytest.fixture(scope="module")
def walk(tmp_path_factory):
    from paged_kv_decode_25_gb300 import build
    exe = str(tmp_path_factory.mktemp("plan") / "sliding_plan")
    subprocess.run([build._nvcc(), "-std=c++17", "-O1", "-I" + build.INCLUDE, "-I" + build.CSRC, *build.ARCH,
                    os.path.join(HERE, "sliding_plan_host.cu"), "-o", exe], check=True, capture_output=True)

    def run(cases):
        """cases: (sms, bytes, Hkv, G, head_dim, blocks in sight of each request)"""
        out = []
        for ulp in (0, 2):
            text = "".join(" ".join(map(str, (*c[:5], ulp, len(c[5]), *c[5]))) + "\n" for c in cases)
            p = subprocess.run([exe], input=text, capture_output=True, text=True)
            assert p.returncode == 0, p.returncode
            rows = [tuple(map(int, line.split())) for line in p.stdout.splitlines()]
            assert len(rows) == len(cases)
            for (places, split, top, twice, lost, even, step, tail), c in zip(rows, cases):
                assert lost == 0 and twice == 0 and split <= places and top == split - 1, (rows, c[:5], len(c[5]))
            out += rows
        return out
    return run


def test_usual_batches(walk):
    """Equal windows (places by division), cut in one way and in two, and unequal ones."""
    cases = []
    for sms in (148, 152):
        for bytes_ in (1, 2):
            for Hkv, G, hd in ((8, 4, 128), (4, 7, 128), (8, 2, 128), (1, 8, 64), (1, 1, 64)):
                for B in (1, 2, 3, 7, 16, 64, 100, 128, 228, 229, 256, 400, 512, 513, 700, 2000):
                    for nb in (1, 2, 9, 65, 257, 1251, 8193):
                        cases.append((sms, bytes_, Hkv, G, hd, [nb] * B))
                    cases.append((sms, bytes_, Hkv, G, hd, [65] * (B - 1) + [64]))
                    cases.append((sms, bytes_, Hkv, G, hd, [0] * (B - 1) + [1000]))
    rows = walk(cases)
    assert any(r[5] and r[6] != r[7] for r in rows) and any(not r[5] for r in rows)


def test_arbitrary_batches(walk):
    r = random.Random(93)
    cases = []
    for _ in range(600):
        B = int(2 ** r.uniform(0, 12))
        top = int(2 ** r.uniform(0, 17 if B < 200 else 11))
        least = r.choice([0, 0, 1, top // 2, max(1, top - 1), top])
        nb = [r.randrange(least, top + 1) for _ in range(B)]
        if r.random() < 0.3:  # some long ones among short ones
            nb = [x if r.random() < 0.05 else min(x, r.choice([0, 1, 3])) for x in nb]
        nb[r.randrange(B)] = max(1, top)
        cases.append((r.choice([1, 2, 100, 148, 152]), r.choice([1, 2]), r.choice([1, 2, 4, 8, 16]), r.randrange(1, 9),
                      r.choice([64, 128]), nb))
    walk(cases)


def test_the_longest_tables(walk):
    """One request, and many, over tables of 2^27 blocks: counts that fp32 rounds, and steps
    that no int holds."""
    most = (1 << 27) - 128
    walk([(sms, bytes_, Hkv, 8, 128, nb) for sms in (1, 148, 152) for bytes_ in (1, 2) for Hkv in (1, 8)
          for nb in ([most], [most - 1] * 3, [most] + [1] * 100, [most // 2, most // 3, 5], [most] * 200, [most] * 4000)])
