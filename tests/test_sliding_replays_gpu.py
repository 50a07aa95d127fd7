"""Captured sliding calls replayed over other lengths, tables and starts than they were
captured with (a serving loop's padded batch): the plan is made on the device, so each
replay gives what a call of its own gives."""
import pytest
import torch

from test_sliding_gpu import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["bf16", "fp8", "int8"])
def test_decode_over_other_lengths(cuda_device, kind):
    """Long units that are split, short ones, none at all, and back, on one workspace."""
    full = [2500, 900, 16, 40, 333, 1, 2000, 77]
    c = Case(full, 8, 2, 64, 700, 20, 98, kind, hide=False)
    lens = torch.tensor(full, dtype=torch.int32, device=cuda_device)
    out, err = c.call(cuda_device, lens=lens)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.call(cuda_device, lens=lens, out=out, ws=c.ws, err=err)
    for now in (full, [0] * 8, [1] * 8, [0, 0, 0, 0, 0, 0, 2000, 0], [n // 2 for n in full], [30, 900, 0, 0, 0, 0, 0, 0], full):
        lens.copy_(torch.tensor(now, dtype=torch.int32))
        want, _ = c.call(cuda_device, lens=lens, ws=torch.full_like(c.ws, 0x55))
        out.fill_(float("nan"))
        for _ in range(2):
            graph.replay()
        torch.cuda.synchronize()
        assert err.item() == 0 and torch.equal(out.view(torch.int16), want.view(torch.int16)), now
    c.check(out, lens=full)


def test_prefill_over_other_batches(cuda_device):
    """max_query_len and total_q as captured bound the batches that come."""
    import paged_kv_decode_25_gb300 as mi
    from test_sliding_prefill_gpu import check, make
    lens, news = [900, 400, 300], [500, 400, 124]
    b, q, kv = make(lens, news, 8, 2, 64, 1 << 20, 0, 99, hide=False)  # (no token out of sight: no poison)
    dev = cuda_device
    qd, k, v, tab = q.to(dev), b.k.to(dev), b.v.to(dev), b.tables.to(dev)
    n, s = torch.zeros(3, dtype=torch.int32, device=dev), torch.zeros(4, dtype=torch.int32, device=dev)
    out, err = torch.empty_like(qd), torch.zeros(1, dtype=torch.int32, device=dev)

    def call(o):
        mi.check(mi.mi_paged_prefill_attention_sliding(mi.dims(3, 8, 2, 64, b.num_blocks, b.width), 1024, 500, qd, k, v, tab,
                                                       n, s, 150, 4, 0.125, o, err))

    call(out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(out)
    for ln, nw in ((lens, news), ([0, 0, 0], [0, 0, 0]), ([700, 0, 1], [1, 0, 1]), ([900, 400, 300], [0, 64, 300]), (lens, news)):
        start = torch.tensor([0] + list(torch.tensor(nw).cumsum(0)), dtype=torch.int32)
        n.copy_(torch.tensor(ln, dtype=torch.int32))
        s.copy_(start)
        want = torch.full_like(out, 3.0)
        call(want)
        out.fill_(3.0)
        for _ in range(2):
            graph.replay()
        torch.cuda.synchronize()
        assert err.item() == 0 and torch.equal(out.view(torch.int16), want.view(torch.int16)), nw
        assert torch.all(out[sum(nw):] == 3.0)  # rows behind the last request
        b.lens = ln
        check(b, kv, nw, 8, 150, 4, q, out.cpu(), rows=[0, 1, 63, 64, 123, 299])
