"""The plan of mi_paged_prefill_scores, walked on the host with the kernels' own
functions: every slot of partial log-sum-exps that a launch reads is in the
workspace and was written by the launch before. (The kernels drop what they read
for rows that do not exist, so no output shows a stray read.)"""
import os
import random
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
PKG = os.path.join(os.path.dirname(HERE), "paged_kv_decode_25_gb300")


@pytest.fixture(scope="module")
def walk(tmp_path_factory):
    from paged_kv_decode_25_gb300 import build
    exe = str(tmp_path_factory.mktemp("plan") / "window_plan")
    subprocess.run([build._nvcc(), "-std=c++17", "-O1", "-I" + build.INCLUDE, "-I" + build.CSRC, *build.ARCH,
                    os.path.join(HERE, "window_plan_host.cu"), "-o", exe], check=True, capture_output=True)

    def run(cases):
        """cases: (Hkv, G, max_q, grid, [(n, m), ..]); resident rows where max_q fits a row block."""
        text = "".join(f"{Hkv} {G} {len(req)} {most} {grid} {int(most <= 256 // G)} "
                       + " ".join(f"{n} {m}" for n, m in req) + "\n" for Hkv, G, most, grid, req in cases)
        p = subprocess.run([exe], input=text, capture_output=True, text=True)
        assert p.returncode == 0, p.returncode
        out = [tuple(map(int, line.split())) for line in p.stdout.splitlines()]
        assert len(out) == len(cases)
        for (have, wrote, twice, top, stray), case in zip(out, cases):
            assert stray == 0 and twice == 0 and top < have, (have, wrote, twice, top, stray, case)
        return out
    return run


def test_requests_without_queries(walk):
    """Keys and no query tokens, beside windows and alone: nothing is read for them."""
    for grid in (148, 152, 256):
        out = walk([(8, 4, 0, grid, [(60000, 0)]),
                    (8, 4, 8, grid, [(4000, 8), (100000, 0)]),
                    (8, 4, 32, grid, [(1000, 32)] * 15 + [(60000, 0)]),
                    (1, 8, 1, grid, [(1 << 30, 0), (16, 1)]),
                    (8, 4, 300, grid, [(4000, 8), (100000, 0), (300, 300)])])
        assert out[0][1] == 0 and out[0][3] == -1


def test_batches(walk):
    r = random.Random(12)
    cases = []
    for _ in range(400):
        Hkv, G = r.choice([(1, 1), (1, 8), (2, 3), (4, 7), (8, 4), (8, 8), (8, 1)])
        whole, req = r.random() < 0.3, []
        for _ in range(r.choice([1, 1, 2, 5, 16, 60])):
            n = int(2 ** r.uniform(0, 14 if whole else 18)) - 1
            m = n if whole else min(n, r.choice([0, 0, 1, 2, 30, 32, 33, 63, 64]))
            if r.random() < 0.1:
                m += 5  # rows before position 0
            req.append((n, m))
        most = max(m for _, m in req) + r.choice([0, 0, 7])
        if r.random() < 0.1:
            most = max(most // 2, 0)  # the longest are left alone
        cases.append((Hkv, G, most, r.choice([1, 100, 148, 152, 256]), req))
    walk(cases)
