"""Waits that give up at once while copies are under way: the launch lets its own
copies land before it ends and reports MI_DEVERR_TIMEOUT, or its outputs are
right; and the calls after it are."""
import pytest
import torch

import test_prefix_gpu as prefix
from paged_ref import Batch, attention_ref

pytestmark = pytest.mark.gpu


def _mi():
    import paged_kv_decode_25_gb300 as mi
    return mi


def hurried(call, want):
    """call() -> (out, dev_err), with waits of one poll."""
    mi = _mi()
    assert mi.mi_test_set_wait_limit(1) == mi.MI_OK
    try:
        for _ in range(20):
            out, err = call()
            assert err & ~mi.MI_DEVERR_TIMEOUT == 0
            assert err or torch.equal(out.view(torch.int16), want.view(torch.int16))
    finally:
        mi.mi_test_set_wait_limit(0)


@pytest.mark.parametrize("d", [64, 128])
def test_prefix(cuda_device, d):
    own = [40, 0, 700, 3, 90]
    both, ptab, tables = prefix.make([2000, 90], own, 2, d, 74)
    q = both.queries(5, 8)

    def run():
        return prefix.call(_mi(), cuda_device, both, ptab, [2000, 90], [0, 3, 5], tables, own, q, 0.1)

    hurried(run, run()[0])
    out, err = run()
    assert err == 0
    prefix.check(both, 2, [0, 3, 5], own, q, out, 0.1)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("variant", [2, 3])  # one Q tile, two
def test_prefill(cuda_device, variant, d):
    mi, dev = _mi(), cuda_device
    lens, m, Hq, Hkv = [700, 130], [300, 130], 8, 2
    batch = Batch(lens, Hkv, d, 75)
    q = batch.queries(sum(m), Hq)
    d_ = mi.dims(2, Hq, Hkv, d, batch.num_blocks, batch.width)
    args = [x.to(dev) for x in (q, batch.k, batch.v, batch.tables, torch.tensor(lens, dtype=torch.int32),
                                torch.tensor([0, m[0], sum(m)], dtype=torch.int32))]
    out = torch.zeros(sum(m), Hq, d, dtype=torch.bfloat16, device=dev)
    err = torch.zeros(1, dtype=torch.int32, device=dev)

    def run():
        err.zero_()
        out.zero_()
        mi.check(mi.mi_paged_prefill_attention_variant(d_, sum(m), max(m), *args, d ** -0.5, out, dev_err=err,
                                                       variant=variant))
        torch.cuda.synchronize()
        return out.cpu(), err.item()

    hurried(run, run()[0])
    got, late = run()
    assert late == 0
    got, at = got.double(), 0
    for r, (n, k) in enumerate(zip(lens, m)):
        for i in range(0, k, 37):
            for h in range(Hkv):
                keys, vals = (batch.tokens(x, r, h)[:n - k + i + 1] for x in (batch.k, batch.v))
                rows = slice(h * Hq // Hkv, (h + 1) * Hq // Hkv)
                want, tol = attention_ref(q[at + i, rows].double(), keys, vals, d ** -0.5)
                assert torch.all((got[at + i, rows] - want).abs() <= tol)
        at += k
