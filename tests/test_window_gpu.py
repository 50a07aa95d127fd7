"""mi_paged_prefill_scores against the weights in 64 bits."""
import pytest
import torch

from paged_ref import BLOCK, Batch, logit_slack, softmax_parts, weight_tolerance

pytestmark = pytest.mark.gpu


def _mi():
    import paged_kv_decode_25_gb300 as mi
    return mi


def call(mi, dev, batch, q, Hq, starts, most, scores, fresh, total=None, tables=None, lens=None, scale=None):
    tables = batch.tables if tables is None else tables
    R = tables.shape[0]
    total = q.shape[0] if total is None else total
    d_ = mi.dims(R, Hq, batch.Hkv, batch.d, batch.num_blocks, tables.shape[1])
    n = mi.mi_paged_prefill_scores_workspace_bytes(d_, total, most)
    assert n > 0
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device=dev)
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    mi.check(mi.mi_paged_prefill_scores(d_, total, most, q.to(dev), batch.k.to(dev), tables.to(dev),
                                        torch.tensor(batch.lens if lens is None else lens, dtype=torch.int32, device=dev),
                                        torch.tensor(starts, dtype=torch.int32, device=dev),
                                        batch.d ** -0.5 if scale is None else scale, fresh, scores, ws, dev_err=err))
    torch.cuda.synchronize()
    return err.item()


def check(batch, q, Hq, starts, before, got, fresh, skipped=(), scale=None):
    G, scale = Hq // batch.Hkv, batch.d ** -0.5 if scale is None else scale
    seen = torch.zeros(before.shape, dtype=torch.bool)
    for r, n in enumerate(batch.lens):
        if n == 0 or r in skipped:
            continue
        m = starts[r + 1] - starts[r]
        blk, off = batch.rows(r)
        keep = torch.arange(n) <= (n - m + torch.arange(m))[:, None]  # [m][n]
        for h in range(batch.Hkv):
            k = batch.tokens(batch.k, r, h)
            w, slack = torch.zeros(n, dtype=torch.float64), 0.0
            for j in range(h * G, (h + 1) * G):
                qs = q[starts[r]:starts[r + 1], j].double()
                if m:
                    w += softmax_parts(qs, k, scale, keep).sum(0)
                slack = max(slack, logit_slack(qs, k, scale))
            old = before[blk, h, off].double()
            if fresh:
                old = torch.zeros_like(old)
            elif m:
                old[max(n - m, 0):] = 0
            tol = weight_tolerance(w, n + m * G, slack, old)
            err = (got[blk, h, off].double() - (old + w)).abs()
            assert torch.all(err <= tol), (r, h, float((err / tol).max()))
            seen[blk, h, off] = True
    assert torch.equal(got.view(torch.int32)[~seen], before.view(torch.int32)[~seen])


def starts_of(m):
    return [0] + torch.tensor(m).cumsum(0).tolist()


@pytest.mark.parametrize("fresh", [False, True])
@pytest.mark.parametrize("Hq,Hkv,d", [(4, 2, 64), (8, 8, 64), (3, 1, 128), (16, 8, 128), (28, 4, 128), (8, 1, 128), (5, 1, 64)])
def test_windows(cuda_device, Hq, Hkv, d, fresh):
    lens, m = [1, 17, 0, 64, 333, 129, 700], [1, 5, 0, 64, 33, 0, 1]
    batch = Batch(lens, Hkv, d, 20)
    q = batch.queries(sum(m), Hq)
    before = torch.rand(batch.num_blocks, Hkv, BLOCK, generator=batch.gen)
    got = before.to(cuda_device)
    assert call(_mi(), cuda_device, batch, q, Hq, starts_of(m), 64, got, fresh) == 0
    check(batch, q, Hq, starts_of(m), before, got.cpu(), fresh)


@pytest.mark.parametrize("n", [2, 15, 16, 63, 64, 65, 127, 128, 129, 257, 1000])
def test_whole_prompts(cuda_device, n):
    batch = Batch([n, max(n - 3, 1)], 2, 64, 21)
    m = batch.lens
    q = batch.queries(sum(m), 6)
    before = torch.rand(batch.num_blocks, 2, BLOCK, generator=batch.gen)
    got = before.to(cuda_device)
    assert call(_mi(), cuda_device, batch, q, 6, starts_of(m), n, got, False) == 0
    check(batch, q, 6, starts_of(m), before, got.cpu(), False)


def test_long_window(cuda_device):
    batch = Batch([9000, 40], 2, 128, 22)
    m = [150, 40]
    q = batch.queries(190, 8)
    before = torch.rand(batch.num_blocks, 2, BLOCK, generator=batch.gen)
    got = before.to(cuda_device)
    assert call(_mi(), cuda_device, batch, q, 8, starts_of(m), 150, got, True) == 0
    check(batch, q, 8, starts_of(m), before, got.cpu(), True)


def test_shares_end_anywhere(cuda_device):
    """One head and unequal requests: shares of the work end within a request's
    rows and keys, windows and prompts alike."""
    for lens, m in (([9000, 40, 5100, 1], [64, 3, 64, 1]), ([2500, 40, 1100], [2500, 40, 700])):
        batch = Batch(lens, 1, 64, 25)
        q = batch.queries(sum(m), 3)
        before = torch.rand(batch.num_blocks, 1, BLOCK, generator=batch.gen)
        got = before.to(cuda_device)
        assert call(_mi(), cuda_device, batch, q, 3, starts_of(m), max(m), got, False) == 0
        check(batch, q, 3, starts_of(m), before, got.cpu(), False)


def test_many_short_requests(cuda_device):
    """More requests than one warp plans for."""
    g = torch.Generator().manual_seed(6)
    lens = torch.randint(0, 50, (600,), generator=g).tolist()
    m = [min(n, 1 + i % 5) for i, n in enumerate(lens)]
    batch = Batch(lens, 1, 64, 26)
    q = batch.queries(sum(m), 2)
    before = torch.rand(batch.num_blocks, 1, BLOCK, generator=batch.gen)
    for most in (5, 300):  # resident rows, resident keys
        got = before.to(cuda_device)
        assert call(_mi(), cuda_device, batch, q, 2, starts_of(m), most, got, False) == 0
        check(batch, q, 2, starts_of(m), before, got.cpu(), False)


@pytest.mark.parametrize("step", [60.0, -60.0])
def test_logits_far_apart(cuda_device, step):
    """Logits that climb or fall by hundreds along the keys, so that the first
    ones say nothing about the size of a row's sum."""
    lens, m = [700, 300], [20, 300]
    batch = Batch(lens, 1, 64, 27)
    q = batch.queries(sum(m), 2)
    q[:, :, 0] = 2.0
    for r, n in enumerate(lens):
        blk, off = batch.rows(r)
        batch.k[blk, 0, off, 0] = (torch.arange(n) // 50 * step).to(torch.bfloat16)
    before = torch.rand(batch.num_blocks, 1, BLOCK, generator=batch.gen)
    got = before.to(cuda_device)
    assert call(_mi(), cuda_device, batch, q, 2, starts_of(m), 300, got, True, scale=0.5) == 0
    check(batch, q, 2, starts_of(m), before, got.cpu(), True, scale=0.5)


@pytest.mark.parametrize("scale", [0.0, -0.2, 1.0])
def test_scales(cuda_device, scale):
    batch = Batch([200, 90], 1, 64, 23)
    q = batch.queries(30, 4)
    before = torch.rand(batch.num_blocks, 1, BLOCK, generator=batch.gen)
    got = before.to(cuda_device)
    assert call(_mi(), cuda_device, batch, q, 4, [0, 20, 30], 20, got, True, scale=scale) == 0
    check(batch, q, 4, [0, 20, 30], before, got.cpu(), True, scale=scale)


def test_one_token_is_the_scored_step(cuda_device):
    mi, dev = _mi(), cuda_device
    batch = Batch([100, 1, 2222], 2, 128, 24)
    q = batch.queries(3, 8)
    a = torch.rand(batch.num_blocks, 2, BLOCK, generator=batch.gen).to(dev)
    b = a.clone()
    assert call(mi, dev, batch, q, 8, [0, 1, 2, 3], 1, a, False) == 0
    d_ = mi.dims(3, 8, 2, 128, batch.num_blocks, batch.width)
    ws = torch.empty(mi.mi_paged_scored_workspace_bytes(d_), dtype=torch.uint8, device=dev)
    mi.check(mi.mi_paged_decode_attention_scored(d_, q.to(dev), batch.k.to(dev), batch.v.to(dev), batch.tables.to(dev),
                                                 torch.tensor(batch.lens, dtype=torch.int32, device=dev), 128 ** -0.5,
                                                 False, torch.empty(3, 8, 128, dtype=torch.bfloat16, device=dev), b, ws))
    torch.cuda.synchronize()
    # two sums of the same fp32 weights (at most 4 each), in other orders
    assert torch.all((a - b).abs() <= 2.0 ** -14 * b.abs() + 1e-30)


def test_device_errors(cuda_device):
    """A request with more queries than max_query_len is left alone, rows before
    position 0 see nothing, a bad block drops out, a long context is cut."""
    mi, dev = _mi(), cuda_device
    batch = Batch([64, 48, 40, 33], 1, 64, 25)
    q = batch.queries(60, 2)
    before = torch.rand(batch.num_blocks, 1, BLOCK, generator=batch.gen)
    got = before.to(dev)
    starts = [0, 4, 34, 50, 60]
    assert call(mi, dev, batch, q, 2, starts, 16, got, False, lens=[64, 48, 40, 4000]) == \
        mi.MI_DEVERR_BAD_QUERY | mi.MI_DEVERR_BAD_CONTEXT | mi.MI_DEVERR_BAD_BLOCK
    # request 3 was cut to its table's 64 tokens: 15 hold NaN keys, the last 16 have no block
    got = got.cpu()
    for r in (0, 2):
        blk, off = batch.rows(r)
        assert torch.all(torch.isfinite(got[blk, 0, off]))
    sub = Batch([64, 48, 40], 1, 64, 25)
    sub.lens, sub.tables, sub.k, sub.num_blocks = [64, 48, 40], batch.tables[:3], batch.k, batch.num_blocks
    hide = batch.tables[3, :3].long()
    got[hide], before[hide] = 0.0, 0.0
    check(sub, q, 2, starts[:4], before, got, False, skipped=(1,))

    got = before.to(dev)
    assert call(mi, dev, batch, q, 2, [0, 4, 2, 50, 60], 60, got, True) == mi.MI_DEVERR_BAD_QUERY
    assert torch.equal(got.cpu(), before)
    assert call(mi, dev, batch, q, 2, [0, 4, 20, 50, 61], 60, got, True, total=60) == mi.MI_DEVERR_BAD_QUERY
    assert torch.equal(got.cpu(), before)

    short = Batch([5], 1, 64, 26)
    q = short.queries(9, 2)
    before = torch.rand(short.num_blocks, 1, BLOCK, generator=short.gen)
    got = before.to(dev)
    assert call(mi, dev, short, q, 2, [0, 9], 9, got, False) == mi.MI_DEVERR_BAD_QUERY
    # the last five rows are a whole prompt's
    check(short, q[4:], 2, [0, 5], before, got.cpu(), False)

    bad = Batch([90], 1, 64, 27)
    q = bad.queries(20, 2)
    tables = bad.tables.clone()
    tables[0, 2] = bad.num_blocks
    before = torch.rand(bad.num_blocks, 1, BLOCK, generator=bad.gen)
    got = before.to(dev)
    assert call(mi, dev, bad, q, 2, [0, 20], 20, got, True, tables=tables) == mi.MI_DEVERR_BAD_BLOCK
    keep = [t for t in range(90) if not 32 <= t < 48]
    blk, off = bad.rows(0)
    k = bad.tokens(bad.k, 0, 0)[keep]
    mask = torch.tensor(keep) <= (70 + torch.arange(20))[:, None]
    w = sum(softmax_parts(q[:, j].double(), k, 64 ** -0.5, mask).sum(0) for j in range(2))
    slack = max(logit_slack(q[:, j].double(), k, 64 ** -0.5) for j in range(2))
    got = got.cpu()
    assert torch.all((got[blk, 0, off].double()[keep] - w).abs() <= weight_tolerance(w, 130, slack))
    assert torch.equal(got[bad.tables[0, 2]], before[bad.tables[0, 2]])


def test_repeat_and_graph(cuda_device):
    mi, dev = _mi(), cuda_device
    batch = Batch([900, 33, 400], 2, 128, 28)
    q = batch.queries(100, 8).to(dev)
    k, tables = batch.k.to(dev), batch.tables.to(dev)
    lens = torch.tensor(batch.lens, dtype=torch.int32, device=dev)
    starts = torch.tensor([0, 64, 70, 100], dtype=torch.int32, device=dev)
    d_ = mi.dims(3, 8, 2, 128, batch.num_blocks, batch.width)
    ws = torch.empty(mi.mi_paged_prefill_scores_workspace_bytes(d_, 100, 64), dtype=torch.uint8, device=dev)
    scores = torch.zeros(batch.num_blocks, 2, BLOCK, device=dev)

    def once():
        mi.check(mi.mi_paged_prefill_scores(d_, 100, 64, q, k, tables, lens, starts, 0.1, True, scores, ws))

    once()
    torch.cuda.synchronize()
    first = scores.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        once()
    for _ in range(3):
        scores.zero_()
        ws.fill_(0x5A)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(scores, first)


@pytest.mark.parametrize("fresh", [False, True])
@pytest.mark.parametrize("lens,m", [([20000, 40, 30001, 900], [0, 8, 0, 32]), ([40000], [0])])
def test_long_contexts_without_queries(cuda_device, lens, m, fresh):
    """Requests with keys and no query tokens, alone (total_q 0) and beside
    windows: their weights are 0, on both paths."""
    batch = Batch(lens, 8, 64, 29)
    q = batch.queries(sum(m), 32)
    before = torch.rand(batch.num_blocks, 8, BLOCK, generator=batch.gen)
    for most in (max(m), 300):  # resident rows, resident keys
        got = before.to(cuda_device)
        assert call(_mi(), cuda_device, batch, q, 32, starts_of(m), most, got, fresh) == 0
        check(batch, q, 32, starts_of(m), before, got.cpu(), fresh)


@pytest.mark.parametrize("most", [1, 300])  # resident rows, resident keys
def test_context_of_268_million(cuda_device, most):
    """More than 2^31 / G tokens (most of them in one block, again and again):
    the first and the last block's scores."""
    mi, dev = _mi(), cuda_device
    n, G, d = (1 << 28) + 4096, 8, 64
    batch = Batch([48], 1, d, 30, spare=0)
    q = batch.queries(1, G)
    first, many, last = batch.tables[0].tolist()
    tables = torch.full((1, n // BLOCK), many, dtype=torch.int32)
    tables[0, 0], tables[0, -1] = first, last
    got = torch.rand(3, 1, BLOCK, generator=batch.gen).to(dev)
    assert call(mi, dev, batch, q, G, [0, 1], most, got, True, tables=tables, lens=[n]) == 0
    k = batch.tokens(batch.k, 0, 0)
    x = (q[0].double() @ k.T * d ** -0.5).exp()  # [G][48]: the first block, one of the many, the last
    times = torch.ones(48, dtype=torch.float64)
    times[16:32] = n // BLOCK - 2
    w = (x / (x * times).sum(-1, keepdim=True)).sum(0)
    w = torch.cat([w[:16], w[32:]])
    have = torch.cat([got[first, 0], got[last, 0]]).cpu().double()
    # sums in sequence: 2^20 stages over at least 100 blocks, 64 columns, the
    # blocks: fewer than 2^14 roundings
    tol = 2 ** 14 * 2.0 ** -24 + 2 * logit_slack(q[0].double(), k, d ** -0.5) + 2.0 ** -20
    assert torch.all((have - w).abs() <= tol * w), float((have / w - 1).abs().max())
