"""Queries that are not finite: their rows are NaN, however the request is cut, and all
other rows are as they were, bit for bit."""
import pytest
import torch

from test_sliding_gpu import Case

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
