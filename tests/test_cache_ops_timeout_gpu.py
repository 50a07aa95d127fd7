"""A copy that never lands in the cache operators' kernels: the call reports
MI_DEVERR_TIMEOUT and returns, and the next one is right.

The hooks make one producer of every block neither copy nor announce a stage,
and shorten every wait to 1 ms; nothing is left in flight."""
import time

import pytest
import torch

import test_prefix_gpu as prefix
import test_scored_gpu as scored
import test_window_gpu as window
from paged_ref import BLOCK, Batch

pytestmark = pytest.mark.gpu


def _mi():
    import paged_kv_decode_25_gb300 as mi
    return mi


def expect_timeout(call):
    """call() -> dev_err, with a copy withheld."""
    mi = _mi()
    assert mi.mi_test_set_wait_limit(1_000_000) == mi.MI_OK
    assert mi.mi_test_withhold_copy(1) == mi.MI_OK
    try:
        t = time.perf_counter()
        err = call()
        t = time.perf_counter() - t
    finally:
        mi.mi_test_withhold_copy(0)
        mi.mi_test_set_wait_limit(0)
    assert err & mi.MI_DEVERR_TIMEOUT
    assert t < 1.0, t


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("own", [[0, 0, 0], [40, 0, 700]])
def test_prefix(cuda_device, d, own):
    both, ptab, tables = prefix.make([2000], own, 2, d, 71)
    q = both.queries(3, 8)

    def run():
        return prefix.call(_mi(), cuda_device, both, ptab, [2000], [0, 3], tables, own, q, 0.1)

    run()
    expect_timeout(lambda: run()[1])
    out, err = run()
    assert err == 0
    prefix.check(both, 1, [0, 3], own, q, out, 0.1)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("m", [[64, 3], [700, 3]])
def test_prompt_scores(cuda_device, d, m):
    batch = Batch([900, 40], 2, d, 72)
    q = batch.queries(sum(m), 8)
    before = torch.rand(batch.num_blocks, 2, BLOCK, generator=batch.gen)

    def run(got):
        return window.call(_mi(), cuda_device, batch, q, 8, window.starts_of(m), max(m), got, False)

    run(before.to(cuda_device))
    expect_timeout(lambda: run(before.to(cuda_device)))
    got = before.to(cuda_device)
    assert run(got) == 0
    window.check(batch, q, 8, window.starts_of(m), before, got.cpu(), False)


@pytest.mark.parametrize("d", [64, 128])
def test_scored(cuda_device, d):
    batch = Batch([900, 40, 0], 2, d, 73)
    q = batch.queries(3, 8)
    before = torch.rand(batch.num_blocks, 2, BLOCK, generator=batch.gen)

    def run(got):
        return scored.step(_mi(), cuda_device, batch, q, 8, got, False)

    run(before.to(cuda_device))
    expect_timeout(lambda: run(before.to(cuda_device))[1])
    got = before.to(cuda_device)
    out, err = run(got)
    assert err == 0
    scored.check(batch, q, 8, before, got.cpu(), out, False)
