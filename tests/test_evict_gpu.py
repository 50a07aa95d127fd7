"""mi_paged_kv_evict: which tokens stay, bit for bit, and that nothing else moves."""
import numpy as np
import pytest
import torch

from paged_ref import BLOCK, Batch, blocks_of, evict_ref

pytestmark = pytest.mark.gpu


def _mi():
    import paged_kv_decode_25_gb300 as mi
    return mi


def scores_for(batch, kind, seed):
    g = torch.Generator().manual_seed(seed)
    shape = (batch.num_blocks, batch.Hkv, BLOCK)
    if kind == "spread":
        return torch.exp(2 * torch.randn(shape, generator=g)) * 1e-3
    if kind == "ties":
        return torch.randint(0, 3, shape, generator=g).float() * 0.25
    if kind == "equal":
        return torch.full(shape, 0.5)
    if kind == "odd":  # infinities, NaN, both zeros, negatives, denormals
        pick = torch.tensor([float("inf"), float("-inf"), float("nan"), 0.0, -0.0, -1.0, 1e-42, -1e-42, 1.0, -float("nan")])
        return pick[torch.randint(0, len(pick), shape, generator=g)]
    raise ValueError(kind)


def fill(cache, batch, seed):
    """Random bits in every row, so that any stray copy shows (bf16 or bytes)."""
    g = torch.Generator().manual_seed(seed)
    return torch.randint(0, 256, tuple(cache.shape) + (cache.element_size(),), generator=g, dtype=torch.uint8)


def run(lens, budgets, recent, Hkv, d, fp8, kind, in_place, seed=1, cuda=None, width=None, err_expected=0, mangle=None):
    mi = _mi()
    batch = Batch(lens, Hkv, d, seed, spare=sum(blocks_of(n) for n in lens) + 3, width=width, fp8=fp8)
    scores = scores_for(batch, kind, seed + 1)
    kraw, vraw = fill(batch.k, batch, seed + 2), fill(batch.v, batch, seed + 3)
    B, kept = len(lens), [min(n, max(x, 0)) for n, x in zip(lens, budgets)]
    if in_place:
        dst = batch.tables
    else:
        dst, at = torch.full_like(batch.tables, -1), 0
        for b, k in enumerate(kept):
            dst[b, :blocks_of(k)] = batch.free[at:at + blocks_of(k)]
            at += blocks_of(k)
    want_k, want_v, want_s = kraw.clone(), vraw.clone(), scores.clone()
    for b, n in enumerate(lens):
        blk, off = batch.rows(b)
        to, to_off = batch.rows(b, kept[b], dst)
        for h in range(Hkv):
            src = torch.from_numpy(evict_ref(scores[blk, h, off].numpy(), n, budgets[b], recent))
            for want, have in ((want_k, kraw), (want_v, vraw), (want_s, scores)):
                want[to, h, to_off] = have[blk[src], h, off[src]]
    dev = cuda
    tables = batch.tables.to(dev)
    dst_d = tables if in_place else dst.to(dev)
    kd, vd, sd = kraw.to(dev), vraw.to(dev), scores.to(dev)
    d_ = mi.dims(B, Hkv, Hkv, d, batch.num_blocks, batch.width)
    ws = torch.empty(mi.mi_paged_kv_evict_workspace_bytes(d_), dtype=torch.uint8, device=dev)
    new, err = torch.full((B,), -7, dtype=torch.int32, device=dev), torch.zeros(1, dtype=torch.int32, device=dev)
    fn = mi.mi_paged_kv_evict_fp8 if fp8 else mi.mi_paged_kv_evict
    mi.check(fn(d_, kd, vd, sd, tables, torch.tensor(lens, dtype=torch.int32, device=dev),
                torch.tensor(budgets, dtype=torch.int32, device=dev), recent, dst_d, new, ws, dev_err=err))
    torch.cuda.synchronize()
    assert err.item() == 0
    assert new.tolist() == kept
    assert torch.equal(kd.cpu(), want_k) and torch.equal(vd.cpu(), want_v)
    assert torch.equal(sd.cpu().view(torch.int32), want_s.view(torch.int32))


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("d,fp8", [(64, False), (128, False), (64, True), (128, True)])
def test_types_and_heads(cuda_device, in_place, d, fp8):
    run([100, 17, 0, 1, 333], [40, 40, 40, 40, 100], 10, 3, d, fp8, "spread", in_place, cuda=cuda_device)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("kind", ["spread", "ties", "equal", "odd"])
@pytest.mark.parametrize("n,budget,recent", [(1, 0, 0), (1, 1, 5), (2, 1, 0), (16, 15, 0), (17, 16, 16), (65, 64, 63),
                                             (300, 1, 0), (300, 299, 0), (300, 128, 200), (1000, 333, 7),
                                             (5000, 4097, 64), (9000, 37, 5)])
def test_lengths_and_ties(cuda_device, in_place, kind, n, budget, recent):
    run([n], [budget], recent, 2, 64, False, kind, in_place, cuda=cuda_device)


def test_many_requests(cuda_device):
    g = np.random.default_rng(5)
    lens = [int(x) for x in g.integers(0, 400, 300)]
    run(lens, [int(x) for x in g.integers(-3, 300, 300)], 33, 1, 64, False, "ties", False, cuda=cuda_device)
    run(lens, [int(x) for x in g.integers(-3, 300, 300)], 0, 1, 64, True, "spread", True, cuda=cuda_device)


@pytest.mark.parametrize("in_place", [False, True])
def test_long(cuda_device, in_place):
    run([70001, 40], [20011, 40], 500, 2, 64, True, "spread", in_place, cuda=cuda_device)


@pytest.mark.parametrize("kind", ["spread", "ties", "odd"])
@pytest.mark.parametrize("lens,Hkv", [([4500, 100], 2), ([9000, 0, 8999, 3], 1), ([16500, 16493, 5, 700], 2), ([16401, 2049, 2048, 2047, 900], 8)])
def test_several_blocks_a_request(cuda_device, lens, Hkv, kind):
    """Tables of 4,096, 8,192 and 16,384 tokens and more are shared by 2, 4 and
    8 blocks where few (request, head) pairs stand for them."""
    run(lens, [max(1, n // 3) for n in lens], 20, Hkv, 64, True, kind, False, cuda=cuda_device)
    run(lens, [n - 1 for n in lens], 0, Hkv, 64, True, kind, True, cuda=cuda_device)


@pytest.mark.parametrize("kind", ["spread", "ties"])
def test_more_keys_than_shared_memory(cuda_device, kind):
    """Eight blocks hold 24,576 keys each; the rest is read again."""
    run([200500], [90001], 500, 1, 64, True, kind, False, cuda=cuda_device)


def test_bad_blocks_and_lengths(cuda_device):
    """A bad source block drops out of the choice, a bad destination block
    drops its rows, a length past the table is cut: reported, nothing else moves."""
    mi, dev = _mi(), cuda_device
    batch = Batch([80], 1, 64, 3, spare=12)
    tables = batch.tables.clone()
    tables[0, 1] = batch.num_blocks + 5
    dst = torch.full_like(tables, -1)
    dst[0, :3] = batch.free[:3]
    dst[0, 1] = -4
    scores = scores_for(batch, "spread", 9)
    k0 = torch.randn(batch.k.shape).to(torch.bfloat16)
    kd, vd, sd = k0.to(dev), k0.to(dev), scores.to(dev)
    d_ = mi.dims(1, 1, 1, 64, batch.num_blocks, batch.width)
    ws = torch.empty(mi.mi_paged_kv_evict_workspace_bytes(d_), dtype=torch.uint8, device=dev)
    new, err = torch.zeros(1, dtype=torch.int32, device=dev), torch.zeros(1, dtype=torch.int32, device=dev)
    mi.check(mi.mi_paged_kv_evict(d_, kd, vd, sd, tables.to(dev), torch.tensor([900], dtype=torch.int32, device=dev),
                                  torch.tensor([40], dtype=torch.int32, device=dev), 8, dst.to(dev), new, ws, dev_err=err))
    torch.cuda.synchronize()
    assert err.item() == mi.MI_DEVERR_BAD_BLOCK | mi.MI_DEVERR_BAD_CONTEXT
    assert new.item() == 40
    s = np.full(80, -np.inf)
    for t in range(80):
        if not 16 <= t < 32:
            s[t] = scores[tables[0, t // 16].item(), 0, t % 16]
    s[16:32] = np.nan  # lowest of all
    src = evict_ref(s, 80, 40, 8)
    want = k0.clone()
    for i, t in enumerate(src):
        if not 16 <= t < 32 and not 16 <= i < 32:
            want[dst[0, i // 16].item(), 0, i % 16] = k0[tables[0, t // 16].item(), 0, t % 16]
    assert torch.equal(kd.cpu(), want) and torch.equal(vd.cpu(), want)


def test_graph_replay_and_stream(cuda_device):
    """Captured once on a stream of its own, replayed with other scores."""
    mi, dev = _mi(), cuda_device
    batch = Batch([200, 90], 2, 128, 4, spare=20)
    dst = torch.full_like(batch.tables, -1)
    dst[0, :4], dst[1, :4] = batch.free[:4], batch.free[4:8]
    d_ = mi.dims(2, 2, 2, 128, batch.num_blocks, batch.width)
    k0 = torch.randn(batch.k.shape).to(torch.bfloat16)
    tables, dst_d = batch.tables.to(dev), dst.to(dev)
    lens = torch.tensor([200, 90], dtype=torch.int32, device=dev)
    bud = torch.tensor([64, 50], dtype=torch.int32, device=dev)
    kd, vd, sd = k0.to(dev), k0.to(dev), scores_for(batch, "spread", 1).to(dev)
    ws = torch.empty(mi.mi_paged_kv_evict_workspace_bytes(d_), dtype=torch.uint8, device=dev)
    new = torch.zeros(2, dtype=torch.int32, device=dev)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())

    def call():
        mi.check(mi.mi_paged_kv_evict(d_, kd, vd, sd, tables, lens, bud, 5, dst_d, new, ws))

    with torch.cuda.stream(side):
        call()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        call()
    for seed in (7, 8):
        scores = scores_for(batch, "ties", seed)
        sd.copy_(scores)
        graph.replay()
        torch.cuda.synchronize()
        got = kd.cpu()
        for b, (n, k) in enumerate(((200, 64), (90, 50))):
            blk, off = batch.rows(b)
            to, to_off = batch.rows(b, k, dst)
            for h in range(2):
                src = torch.from_numpy(evict_ref(scores[blk, h, off].numpy(), n, k, 5))
                assert torch.equal(got[to, h, to_off], k0[blk[src], h, off[src]])
