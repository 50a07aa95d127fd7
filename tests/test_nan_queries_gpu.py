"""Queries that are not finite: their rows are NaN, however the request is cut, and all
other rows are as they were, bit for bit. (A row whose scores are all -inf counts as
one that sees no key: an infinite query, and few keys, all on its other side.)"""
import pytest
import torch

from test_sliding_gpu import Case
from test_sliding_prefill_gpu import make, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("kind", ["bf16", "fp8", "int8"])
@pytest.mark.parametrize("lens,window", [([900, 40, 700], 600), ([3000] * 300, 100)])
def test_decode(cuda_device, kind, lens, window, bad):
    """Few requests, in pieces that are added up, and more units than warps, in one piece each."""
    c = Case(lens, 8, 2, 64, window, 4, 94, kind)
    want, _ = c.call(cuda_device)
    rows = [(0, 1), (2, 7), (1, 4)]
    for s, j in rows:
        c.dev["q"][s, j, 5] = bad
    out, err = c.call(cuda_device)
    assert err.item() == 0
    same = torch.ones(out.shape[:2], dtype=torch.bool, device=out.device)
    for s, j in rows:
        assert torch.isnan(out[s, j].float()).all(), (s, j)
        same[s, j] = False
    assert torch.equal(out[same].view(torch.int16), want[same].view(torch.int16))


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_prefill(cuda_device, bad):
    lens, news = [900, 200, 700], [300, 200, 1]
    b, q, kv = make(lens, news, 8, 2, 64, 150, 4, 95)
    want, _ = run(cuda_device, b, news, 8, 150, 4, q)
    rows = [(0, 0), (17, 3), (255, 7), (300, 2), (499, 5), (500, 1)]
    for i, j in rows:
        q[i, j, 5] = bad
    out, err = run(cuda_device, b, news, 8, 150, 4, q)
    assert err == 0
    same = torch.ones(out.shape[:2], dtype=torch.bool)
    for i, j in rows:
        same[i, j] = False
        if (i, j) == (300, 2) and bad > 0 and kv[1][0][0][0, 5] < 0:  # a first token: it sees itself alone
            assert torch.count_nonzero(out[i, j].float()) == 0
        else:
            assert torch.isnan(out[i, j].float()).all(), (i, j)
    assert torch.equal(out[same].view(torch.int16), want[same].view(torch.int16))
