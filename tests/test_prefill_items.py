"""The work items of the prefill kernels, made on the host with the kernels' own
functions from words that nobody has checked: every item stays within q's rows and
its table row, and those of good requests cover their rows."""
import os
import random
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
LEAST, MOST = -2 ** 31, 2 ** 31 - 1


@pytest.fixture(scope="module")
def walk(tmp_path_factory):
    from paged_kv_decode_25_gb300 import build
    exe = str(tmp_path_factory.mktemp("items") / "prefill_items")
    subprocess.run([build._nvcc(), "-std=c++17", "-O1", "-I" + build.INCLUDE, "-I" + build.CSRC, *build.ARCH,
                    os.path.join(HERE, "prefill_items_host.cu"), "-o", exe], check=True, capture_output=True)

    def run(cases):
        """cases: (G, mbps, T, max_q, window, sinks, lens, starts)"""
        text = "".join(" ".join(map(str, (*c[:6], len(c[6]), *c[6], *c[7]))) + "\n" for c in cases)
        p = subprocess.run([exe], input=text, capture_output=True, text=True)
        assert p.returncode == 0, p.returncode
        out = [tuple(map(int, line.split())) for line in p.stdout.splitlines()]
        assert len(out) == len(cases)
        for (items, bad, rows, slide_rows), c in zip(out, cases):
            G, _, T, max_q, _, _, lens, starts = c
            assert bad == 0, c
            want = sum(b - a for a, b in zip(starts, starts[1:]) if 0 <= a <= b <= T and b - a <= max_q) * G
            assert rows == want and slide_rows == want, (rows, slide_rows, want, c)
        return out
    return run


def test_lengths_that_would_wrap(walk):
    """A length near the least word, less the new tokens, is not a far position."""
    for n in (LEAST, LEAST + 1, LEAST + 299, LEAST + 300, -1, 0, 1, 299, 300, 301, MOST):
        for window, sinks in ((1, 0), (100, 4), (MOST, MOST)):
            out = walk([(G, 64, 300, 300, window, sinks, [n], [0, 300]) for G in (1, 3, 8)])
            assert all(items > 0 for items, *_ in out)


def test_starts_that_would_wrap(walk):
    """Starts past the end and before the beginning whose difference is a small number."""
    for a, b in ((MOST, LEAST), (MOST - 9, LEAST + 90), (600, LEAST + 500), (501, LEAST + 501), (-1, 99), (LEAST, LEAST + 5),
                 (LEAST, MOST), (MOST, MOST), (500, 499), (401, 501), (0, MOST)):
        out = walk([(4, 64, 500, q, 50, 4, [200], [a, b]) for q in (200, 500)])
        assert all(items == 0 for items, *_ in out), (a, b)


def test_arbitrary_words(walk):
    r = random.Random(90)
    words = [LEAST, LEAST + 1, LEAST + 40, -1000, -17, -1, 0, 1, 15, 16, 17, 500, 1000, 1024, 5000, MOST - 1, MOST]

    def word():
        return r.choice([r.choice(words), r.randrange(-50, 1200), r.randrange(LEAST, MOST + 1)])

    cases = []
    for _ in range(1500):
        G, mbps, R = r.randrange(1, 9), r.choice([1, 5, 64, (1 << 27) - 128]), r.randrange(1, 9)
        starts = [word() for _ in range(R + 1)]
        if r.random() < 0.5:
            starts = sorted(r.randrange(0, 1001) for _ in range(R + 1))
        cases.append((G, mbps, 1000, r.choice([1, 100, 1000]), max(1, abs(word()) & MOST), abs(word()) & MOST,
                      [word() for _ in range(R)], starts))
    walk(cases)
