"""The cache operators on two streams at once, and from two captured graphs over
one workspace: the same bits as one call after another."""
import pytest
import torch

from paged_ref import BLOCK, Batch

pytestmark = pytest.mark.gpu


def _mi():
    import paged_kv_decode_25_gb300 as mi
    return mi


def operator(name, dev, seed, space=None):
    """(call, outputs, workspace): call() queues one call on the current stream."""
    mi = _mi()
    lens, Hkv, Hq, d = [900, 40 + seed, 0, 2300, 17], 2, 8, 128
    batch = Batch(lens, Hkv, d, 90 + seed)
    B, tables, n = len(lens), batch.tables.to(dev), torch.tensor(lens, dtype=torch.int32, device=dev)
    d_ = mi.dims(B, Hq, Hkv, d, batch.num_blocks, batch.width)
    k, v = (torch.nan_to_num(x).to(dev) for x in (batch.k, batch.v))
    out = torch.zeros(B, Hq, d, dtype=torch.bfloat16, device=dev)
    scores = torch.zeros(batch.num_blocks, Hkv, BLOCK, device=dev)

    def room(size):
        return torch.empty(size, dtype=torch.uint8, device=dev) if space is None else space[:size]

    if name == "prefix":  # request 3's tokens are the prefix of the others
        q, ws = batch.queries(B, Hq).to(dev), room(mi.mi_paged_prefix_workspace_bytes(d_, 1, batch.width))
        starts = torch.tensor([0, B], dtype=torch.int32, device=dev)
        ptab, plen = tables[3:4].contiguous(), n[3:4].contiguous()

        def call():
            mi.check(mi.mi_paged_decode_attention_prefix(d_, 1, batch.width, q, k, v, ptab, plen, starts, tables, n, 0.1,
                                                         out, ws))
        return call, [out], ws
    if name == "scored":
        q, ws = batch.queries(B, Hq).to(dev), room(mi.mi_paged_scored_workspace_bytes(d_))

        def call():
            mi.check(mi.mi_paged_decode_attention_scored(d_, q, k, v, tables, n, 0.1, True, out, scores, ws))
        return call, [out, scores], ws
    if name in ("window", "prompt"):
        m = [min(x, 30 if name == "window" else 700) for x in lens]
        starts = torch.tensor([0] + torch.tensor(m).cumsum(0).tolist(), dtype=torch.int32, device=dev)
        q = batch.queries(sum(m), Hq).to(dev)
        ws = room(mi.mi_paged_prefill_scores_workspace_bytes(d_, sum(m), max(m)))

        def call():
            mi.check(mi.mi_paged_prefill_scores(d_, sum(m), max(m), q, k, tables, n, starts, 0.1, True, scores, ws))
        return call, [scores], ws
    weights = torch.rand(scores.shape, generator=batch.gen).to(dev)
    budgets = torch.full((B,), 100, dtype=torch.int32, device=dev)
    new, ws, kk, vv = torch.zeros_like(n), room(mi.mi_paged_kv_evict_workspace_bytes(d_)), k.clone(), v.clone()

    def call():
        kk.copy_(k)
        vv.copy_(v)
        scores.copy_(weights)
        mi.check(mi.mi_paged_kv_evict(d_, kk, vv, scores, tables, n, budgets, 10, tables, new, ws))
    return call, [kk, vv, scores, new], ws


def bits(tensors):
    return [t.clone().view(torch.uint8) for t in tensors]


NAMES = ["prefix", "scored", "window", "prompt", "evict"]


@pytest.mark.parametrize("other", NAMES)
@pytest.mark.parametrize("name", NAMES)
def test_two_streams(cuda_device, name, other):
    ops = [operator(name, cuda_device, 1), operator(other, cuda_device, 2)]
    want = []
    for call, outs, _ in ops:
        call()
        torch.cuda.synchronize()
        want.append(bits(outs))
        for t in outs:
            t.zero_()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(12):
        for (call, _, _), stream in zip(ops, streams):
            with torch.cuda.stream(stream):
                call()
    torch.cuda.synchronize()
    for (_, outs, _), ref in zip(ops, want):
        assert all(torch.equal(a, b) for a, b in zip(bits(outs), ref))


@pytest.mark.parametrize("name", NAMES)
def test_two_graphs_over_one_workspace(cuda_device, name):
    _, _, a = operator(name, cuda_device, 1)
    _, _, b = operator(name, cuda_device, 2)
    space = torch.empty(max(a.numel(), b.numel()), dtype=torch.uint8, device=cuda_device)
    ops = [operator(name, cuda_device, seed, space) for seed in (1, 2)]
    want, graphs, stream = [], [], torch.cuda.Stream()
    for call, outs, _ in ops:
        call()
        torch.cuda.synchronize()
        want.append(bits(outs))
    with torch.cuda.stream(stream):
        for call, _, _ in ops:
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=stream):
                call()
                call()
            graphs.append(g)
        for i in range(10):
            graphs[i % 2].replay()
            graphs[i // 2 % 2].replay()
    torch.cuda.synchronize()
    for (_, outs, _), ref in zip(ops, want):
        assert all(torch.equal(x, y) for x, y in zip(bits(outs), ref))


@pytest.mark.parametrize("name", NAMES)
def test_replays_write_everything(cuda_device, name):
    """Two graphs over one workspace, every output poisoned before each replay:
    a replay leaves the bits that an eager call leaves over the same poison."""
    _, _, a = operator(name, cuda_device, 1)
    _, _, b = operator(name, cuda_device, 2)
    space = torch.empty(max(a.numel(), b.numel()), dtype=torch.uint8, device=cuda_device)
    ops = [operator(name, cuda_device, seed, space) for seed in (1, 2)]

    def poison(outs):
        for t in outs:
            t.view(torch.uint8).fill_(0x3C)

    want, graphs, stream = [], [], torch.cuda.Stream()
    for call, outs, _ in ops:
        poison(outs)
        call()
        torch.cuda.synchronize()
        want.append(bits(outs))
        poison(outs)
        assert not all(torch.equal(x, y) for x, y in zip(bits(outs), want[-1]))
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        for call, _, _ in ops:
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=stream):
                call()
            graphs.append(g)
        for i in (0, 1, 1, 0, 0, 1, 0, 1):
            poison(ops[i][1])
            graphs[i].replay()
            got = bits(ops[i][1])
            assert all(torch.equal(x, y) for x, y in zip(got, want[i]))
    torch.cuda.synchronize()
