"""mi_paged_decode_attention_scored: the output, and the weight of every cached
token, against 64 bits; what holds no token keeps its bits."""
import pytest
import torch

from paged_ref import (BLOCK, FP32_HALF, Batch, attention_ref, logit_slack, softmax_parts, weight_tolerance)

pytestmark = pytest.mark.gpu


def _mi():
    import paged_kv_decode_25_gb300 as mi
    return mi


def step(mi, dev, batch, q, Hq, scores, fresh, fp8=None, tables=None, lens=None, width=None, space=None):
    d = batch.d
    B = q.shape[0]
    tables = batch.tables if tables is None else tables
    d_ = mi.dims(B, Hq, batch.Hkv, d, batch.num_blocks, tables.shape[1])
    n = mi.mi_paged_scored_workspace_bytes(d_)
    assert n > 0
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device=dev) if space is None else space
    out = torch.full((B, Hq, d), float("nan"), dtype=torch.bfloat16, device=dev)
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    lens = torch.tensor(batch.lens if lens is None else lens, dtype=torch.int32, device=dev)
    scale = d ** -0.5
    if fp8 is None:
        st = mi.mi_paged_decode_attention_scored(d_, q.to(dev), batch.k.to(dev), batch.v.to(dev), tables.to(dev), lens,
                                                 scale, fresh, out, scores, ws, dev_err=err)
    else:
        st = mi.mi_paged_decode_attention_scored_fp8(d_, q.to(dev), batch.k.to(dev), batch.v.to(dev), fp8[0].to(dev),
                                                     fp8[1].to(dev), tables.to(dev), lens, scale, fresh, out, scores,
                                                     ws, dev_err=err)
    mi.check(st)
    torch.cuda.synchronize()
    return out.cpu(), err.item()


def check(batch, q, Hq, before, got, out, fresh, fp8=None):
    G, scale = Hq // batch.Hkv, batch.d ** -0.5
    want_bits = before.view(torch.int32).clone()
    seen = torch.zeros_like(want_bits, dtype=torch.bool)
    for b, n in enumerate(batch.lens):
        if n == 0:
            assert torch.count_nonzero(out[b].float()) == 0
            continue
        blk, off = batch.rows(b)
        for h in range(batch.Hkv):
            qs = q[b, h * G:(h + 1) * G].double()
            k = batch.tokens(batch.k, b, h) * (1.0 if fp8 is None else fp8[0][h].double())
            v = batch.tokens(batch.v, b, h) * (1.0 if fp8 is None else fp8[1][h].double())
            ref, tol = attention_ref(qs, k, v, scale)
            err = (out[b, h * G:(h + 1) * G].double() - ref).abs()
            assert torch.all(err <= tol), (b, h, float((err / tol).max()))
            w = softmax_parts(qs, k, scale).sum(0)
            old = before[blk, h, off].double()
            if fresh:
                old = torch.zeros_like(old)
            else:
                old[-1] = 0.0
            # fp8: q is converted to f16 (exact for bf16 of this range) and the
            # scale multiplies the logits: one more rounding of each
            slack = logit_slack(qs, k, scale) + float((qs @ k.T).abs().max()) * scale * 4 * FP32_HALF
            tol = weight_tolerance(w, n + G, slack, old)
            err = (got[blk, h, off].double() - (old + w)).abs()
            assert torch.all(err <= tol), (b, h, float((err / tol).max()))
            seen[blk, h, off] = True
    assert torch.equal(got.view(torch.int32)[~seen], want_bits[~seen])


SHAPES = [(4, 2, 64), (8, 8, 64), (3, 1, 128), (16, 8, 128), (28, 4, 128), (8, 1, 128), (10, 2, 64)]


@pytest.mark.parametrize("fresh", [False, True])
@pytest.mark.parametrize("Hq,Hkv,d", SHAPES)
def test_shapes(cuda_device, Hq, Hkv, d, fresh):
    batch = Batch([1, 17, 0, 64, 333, 16, 1200], Hkv, d, 10)
    q = batch.queries(len(batch.lens), Hq)
    before = torch.rand(batch.num_blocks, Hkv, BLOCK, generator=batch.gen)
    got = before.to(cuda_device)
    out, err = step(_mi(), cuda_device, batch, q, Hq, got, fresh)
    assert err == 0
    check(batch, q, Hq, before, got.cpu(), out, fresh)


@pytest.mark.parametrize("Hq,Hkv,d", [(4, 2, 64), (32, 8, 128), (7, 1, 128)])
def test_fp8(cuda_device, Hq, Hkv, d):
    batch = Batch([1, 50, 0, 700], Hkv, d, 11, fp8=True)
    q = batch.queries(4, Hq)
    scales = (0.5 + torch.rand(Hkv, generator=batch.gen), 0.5 + torch.rand(Hkv, generator=batch.gen))
    before = torch.rand(batch.num_blocks, Hkv, BLOCK, generator=batch.gen)
    for fresh in (False, True):
        got = before.to(cuda_device)
        out, err = step(_mi(), cuda_device, batch, q, Hq, got, fresh, fp8=scales)
        assert err == 0
        check(batch, q, Hq, before, got.cpu(), out, fresh, fp8=scales)


@pytest.mark.parametrize("wide", [False, True])
def test_logit_places(cuda_device, wide):
    """Tables much wider than the cache (logits placed by the cache's blocks)
    and as wide as needed (by the batch's order) give the same bits."""
    batch = Batch([100, 2000, 3, 640], 2, 128, 12, width=4096 if wide else None)
    q = batch.queries(4, 8)
    before = torch.rand(batch.num_blocks, 2, BLOCK, generator=batch.gen)
    got = before.to(cuda_device)
    out, err = step(_mi(), cuda_device, batch, q, 8, got, False)
    assert err == 0
    check(batch, q, 8, before, got.cpu(), out, False)


def test_weights_sum_to_group(cuda_device):
    """Every KV head's weights sum to its G query heads."""
    batch = Batch([777, 16, 5000], 4, 64, 13)
    q = batch.queries(3, 12)
    got = torch.zeros(batch.num_blocks, 4, BLOCK, device=cuda_device)
    step(_mi(), cuda_device, batch, q, 12, got, True)
    for b, n in enumerate(batch.lens):
        blk, off = batch.rows(b)
        total = got.cpu()[blk, :, off].double().sum(0)
        assert torch.all((total - 3).abs() <= 3 * (n * FP32_HALF + 2.0 ** -15))


def test_same_output_as_plain_attention(cuda_device):
    mi, dev = _mi(), cuda_device
    batch = Batch([1, 700, 31, 0, 2500], 2, 128, 14)
    q = batch.queries(5, 8)
    scores = torch.zeros(batch.num_blocks, 2, BLOCK, device=dev)
    out, _ = step(mi, dev, batch, q, 8, scores, True)
    d_ = mi.dims(5, 8, 2, 128, batch.num_blocks, batch.width)
    ws = torch.empty(mi.mi_paged_decode_workspace_bytes(d_), dtype=torch.uint8, device=dev)
    plain = torch.empty(5, 8, 128, dtype=torch.bfloat16, device=dev)
    mi.check(mi.mi_paged_decode_attention(d_, q.to(dev), batch.k.to(dev), batch.v.to(dev), batch.tables.to(dev),
                                          torch.tensor(batch.lens, dtype=torch.int32, device=dev), 128 ** -0.5, plain, ws))
    torch.cuda.synchronize()
    # the sums alone differ: by half a bf16 step of their value, then a rounding each
    a, b = out.double(), plain.cpu().double()
    assert torch.all((a - b).abs() <= 3 * 2.0 ** -8 * b.abs() * 1.01 + 1e-30)


def test_bad_blocks_and_lengths(cuda_device):
    """Tokens of a bad block are left out and keep no score; a context longer
    than its table is cut at the table."""
    mi, dev = _mi(), cuda_device
    batch = Batch([64, 48], 1, 64, 15)
    q = batch.queries(2, 2)
    tables = batch.tables.clone()
    tables[0, 1] = -3
    before = torch.rand(batch.num_blocks, 1, BLOCK, generator=batch.gen)
    got = before.to(dev)
    out, err = step(mi, dev, batch, q, 2, got, False, tables=tables, lens=[64, 500])
    assert err == mi.MI_DEVERR_BAD_BLOCK | mi.MI_DEVERR_BAD_CONTEXT
    got = got.cpu()
    assert torch.equal(got[batch.tables[0, 1]], before[batch.tables[0, 1]])
    keep = [t for t in range(64) if not 16 <= t < 32]
    blk, off = batch.rows(0)
    k = batch.tokens(batch.k, 0, 0)[keep]
    w = softmax_parts(q[0].double(), k, 64 ** -0.5).sum(0)
    old = before[blk, 0, off].double()[keep]
    old[-1] = 0
    err = (got[blk, 0, off].double()[keep] - old - w).abs()
    assert torch.all(err <= weight_tolerance(w, 66, logit_slack(q[0].double(), k, 64 ** -0.5), old))


def test_repeat_and_graph(cuda_device):
    """The same bits every time, eager and replayed, also after another batch
    has used the workspace."""
    mi, dev = _mi(), cuda_device
    batch = Batch([900, 33, 16, 4000], 2, 128, 16)
    q = batch.queries(4, 8).to(dev)
    k, v, tables = batch.k.to(dev), batch.v.to(dev), batch.tables.to(dev)
    lens = torch.tensor(batch.lens, dtype=torch.int32, device=dev)
    d_ = mi.dims(4, 8, 2, 128, batch.num_blocks, batch.width)
    ws = torch.empty(mi.mi_paged_scored_workspace_bytes(d_), dtype=torch.uint8, device=dev)
    out = torch.empty(4, 8, 128, dtype=torch.bfloat16, device=dev)
    scores = torch.zeros(batch.num_blocks, 2, BLOCK, device=dev)

    def call(fresh):
        mi.check(mi.mi_paged_decode_attention_scored(d_, q, k, v, tables, lens, 0.1, fresh, out, scores, ws))

    call(True)
    torch.cuda.synchronize()
    first, first_out = scores.clone(), out.clone()
    for _ in range(3):
        call(True)
    torch.cuda.synchronize()
    assert torch.equal(scores, first) and torch.equal(out.view(torch.int16), first_out.view(torch.int16))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        call(True)
        call(False)
    ws.fill_(0x5A)
    for _ in range(2):
        scores.zero_()
        graph.replay()
        torch.cuda.synchronize()
        want = first + first
        at = torch.zeros_like(scores, dtype=torch.bool)
        for b, n in enumerate(batch.lens):
            blk, off = batch.rows(b)
            at[blk.to(dev), :, off.to(dev)] = True
            want[blk[-1].to(dev), :, off[-1].to(dev)] = first[blk[-1].to(dev), :, off[-1].to(dev)]
        assert torch.equal(scores[at], want[at])
        assert torch.equal(out.view(torch.int16), first_out.view(torch.int16))
