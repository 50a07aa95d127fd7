"""mi_paged_prefill_attention_sliding against 64 bits, row by row. Tokens that no new
token of their request sees hold NaN, and table columns of blocks without any
other token hold -1."""
import pytest
import torch

from paged_ref import BLOCK, Batch, attention_ref

pytestmark = pytest.mark.gpu


def _mi():
    import paged_kv_decode_25_gb300 as mi
    return mi


def poison(b, news, window, sinks, hide=True):
    for s, (n, m) in enumerate(zip(b.lens, news)):
        t = torch.arange(n)
        unseen = (t >= sinks) & (t <= n - m - window)
        blk, off = b.rows(s)
        for c in (b.k, b.v):
            c[blk[unseen], :, off[unseen]] = float("nan")
        for j in range(-(-n // BLOCK)):
            if hide and n and unseen[j * BLOCK:(j + 1) * BLOCK].all():
                b.tables[s, j] = -1


def run(dev, b, news, Hq, window, sinks, q, scale=None, lens=None, out=None, err=None, max_q=None, starts=None):
    mi = _mi()
    total = sum(news)
    start = torch.tensor([0] + list(torch.tensor(news).cumsum(0)), dtype=torch.int32) if starts is None else starts
    out = torch.full((total, Hq, b.d), float("nan"), dtype=torch.bfloat16, device=dev) if out is None else out
    err = torch.zeros(1, dtype=torch.int32, device=dev) if err is None else err
    lens = torch.tensor(b.lens, dtype=torch.int32) if lens is None else lens
    mi.check(mi.mi_paged_prefill_attention_sliding(
        mi.dims(len(b.lens), Hq, b.Hkv, b.d, b.num_blocks, b.tables.shape[1]), total,
        max(news + [0]) if max_q is None else max_q, q.to(dev), b.k.to(dev), b.v.to(dev), b.tables.to(dev), lens.to(dev),
        start.to(dev), window, sinks, b.d ** -0.5 if scale is None else scale, out, err))
    torch.cuda.synchronize()
    return out.cpu(), err.item()


def check(b, kv, news, Hq, window, sinks, q, out, rows=None, scale=None):
    """rows: the new tokens that are looked at, of each request (all by default)."""
    G, at = Hq // b.Hkv, 0
    scale = b.d ** -0.5 if scale is None else scale
    for s, (n, m) in enumerate(zip(b.lens, news)):
        for i in range(m) if rows is None else sorted({x % m for x in rows}) if m else ():
            p = n - m + i
            t = torch.arange(p + 1)
            t = t[(t < sinks) | (t > p - window)]
            for h in range(b.Hkv):
                k, v = (x[t] for x in kv[s][h])
                ref, tol = attention_ref(q[at + i, h * G:(h + 1) * G].double(), k, v, scale)
                err = (out[at + i, h * G:(h + 1) * G].double() - ref).abs()
                assert torch.all(err <= tol), (s, i, h, float((err / tol).max()))
        at += m


def make(lens, news, Hq, Hkv, d, window, sinks, seed, hide=True, width=None):
    b = Batch(lens, Hkv, d, seed, width=width)
    q = b.queries(sum(news), Hq)
    kv = [[(b.tokens(b.k, s, h), b.tokens(b.v, s, h)) for h in range(Hkv)] for s in range(len(lens))]
    poison(b, news, window, sinks, hide)
    return b, q, kv


SHAPES = [(4, 2, 64), (8, 8, 64), (3, 1, 128), (16, 8, 128), (28, 4, 128), (8, 1, 128), (10, 2, 64)]


@pytest.mark.parametrize("window,sinks", [(100, 4), (20, 0), (1, 1)])
@pytest.mark.parametrize("Hq,Hkv,d", SHAPES)
def test_shapes(cuda_device, Hq, Hkv, d, window, sinks):
    lens, news = [1, 17, 0, 64, 333, 300, 500], [1, 17, 0, 10, 1, 300, 129]
    b, q, kv = make(lens, news, Hq, Hkv, d, window, sinks, 40)
    out, err = run(cuda_device, b, news, Hq, window, sinks, q)
    assert err == 0
    check(b, kv, news, Hq, window, sinks, q, out, rows=[0, 1, 15, 16, 63, 64, 100, 127, 128, 200, 298, 299])


@pytest.mark.parametrize("window", [1, 2, 15, 16, 17, 33, 64, 128, 129, 250, 2 ** 31 - 1])
@pytest.mark.parametrize("sinks", [0, 1, 16, 17, 140, 2 ** 31 - 1])
def test_windows_and_sinks(cuda_device, window, sinks):
    lens, news = [200, 40, 460, 300], [200, 7, 130, 16]
    b, q, kv = make(lens, news, 4, 1, 64, window, sinks, 41)
    out, err = run(cuda_device, b, news, 4, window, sinks, q)
    assert err == 0
    check(b, kv, news, 4, window, sinks, q, out, rows=[0, 1, 2, 14, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 199])


def test_long_prompts(cuda_device):
    lens, news = [5000, 3500, 4000], [5000, 3500, 100]
    for window, sinks in ((1024, 4), (600, 130)):
        b, q, kv = make(lens, news, 8, 2, 128, window, sinks, 42)
        out, err = run(cuda_device, b, news, 8, window, sinks, q)
        assert err == 0 and torch.all(torch.isfinite(out.float()))
        check(b, kv, news, 8, window, sinks, q, out, rows=[0, 63, 64, 99, 1000, 1023, 1024, 1025, 1090, 2047, 3071, 4444, 4999])


def test_whole_context_is_causal_attention(cuda_device):
    mi = _mi()
    lens, news = [300, 77, 1000], [300, 20, 513]
    b, q, kv = make(lens, news, 8, 2, 128, 1 << 20, 0, 43)
    out, err = run(cuda_device, b, news, 8, 1 << 20, 0, q)
    want = torch.empty_like(out, device=cuda_device)
    start = torch.tensor([0, 300, 320, 833], dtype=torch.int32, device=cuda_device)
    mi.check(mi.mi_paged_prefill_attention(
        mi.dims(3, 8, 2, 128, b.num_blocks, b.width), 833, 513, q.to(cuda_device), b.k.to(cuda_device),
        b.v.to(cuda_device), b.tables.to(cuda_device), torch.tensor(lens, dtype=torch.int32, device=cuda_device), start,
        128 ** -0.5, want))
    assert err == 0
    rows = [0, 1, 19, 63, 64, 127, 128, 299, 512]
    check(b, kv, news, 8, 1 << 20, 0, q, out, rows=rows)
    check(b, kv, news, 8, 1 << 20, 0, q, want.cpu(), rows=rows)


def test_one_new_token_is_the_decode_call(cuda_device):
    mi = _mi()
    lens, news = [300, 77, 1000], [1, 1, 1]
    b, q, kv = make(lens, news, 8, 2, 128, 200, 20, 44)
    out, _ = run(cuda_device, b, news, 8, 200, 20, q)
    check(b, kv, news, 8, 200, 20, q, out)
    d_ = mi.dims(3, 8, 2, 128, b.num_blocks, b.width)
    ws = torch.empty(mi.mi_paged_sliding_workspace_bytes(d_, 200, 20), dtype=torch.uint8, device=cuda_device)
    got = torch.empty(3, 8, 128, dtype=torch.bfloat16, device=cuda_device)
    mi.check(mi.mi_paged_decode_attention_sliding(d_, q.to(cuda_device), b.k.to(cuda_device), b.v.to(cuda_device),
                                                  b.tables.to(cuda_device),
                                                  torch.tensor(lens, dtype=torch.int32, device=cuda_device), 200, 20,
                                                  128 ** -0.5, got, ws))
    check(b, kv, news, 8, 200, 20, q, got.cpu())


def test_window_of_one_is_the_value(cuda_device):
    b, q, kv = make([90], [90], 4, 2, 64, 1, 0, 45)
    out, _ = run(cuda_device, b, [90], 4, 1, 0, q)
    for h in range(2):
        want = kv[0][h][1].to(torch.bfloat16)
        for g in range(2):
            assert torch.equal(out[:, 2 * h + g], want)


def test_scales_and_logits_far_apart(cuda_device):
    for scale in (-0.3, 0.0, 20.0):
        b, q, kv = make([300, 200], [300, 40], 4, 2, 64, 50, 4, 46)
        out, err = run(cuda_device, b, [300, 40], 4, 50, 4, q, scale=scale)
        assert err == 0 and torch.all(torch.isfinite(out.float()))
        check(b, kv, [300, 40], 4, 50, 4, q, out, rows=range(0, 300, 7), scale=scale)


def test_errors(cuda_device):
    mi = _mi()
    # a bad block in sight drops its keys; one out of sight is not looked at
    b, q, kv = make([300], [20], 4, 1, 64, 100, 4, 47, hide=False)
    b.tables[0, 14], b.tables[0, 5] = b.num_blocks, -9
    out, err = run(cuda_device, b, [20], 4, 100, 4, q)
    assert err == mi.MI_DEVERR_BAD_BLOCK
    for i in (0, 10, 19):
        p = 280 + i
        t = torch.arange(p + 1)
        t = t[((t < 4) | (t > p - 100)) & (t // 16 != 14)]
        ref, tol = attention_ref(q[i].double(), *(x[t] for x in kv[0][0]), 64 ** -0.5)
        assert torch.all((out[i].double() - ref).abs() <= tol)
    # more new tokens than context: rows before position 0 are zero
    b, q, kv = make([30], [30], 4, 1, 64, 8, 2, 48)
    out, err = run(cuda_device, b, [30], 4, 8, 2, q, lens=torch.tensor([20], dtype=torch.int32))
    assert err == mi.MI_DEVERR_BAD_QUERY and torch.count_nonzero(out[:10].float()) == 0
    # a length past the table, a request longer than said, starts that do not ascend
    b, q, kv = make([320], [16], 4, 1, 64, 50, 4, 49, hide=False)
    out, err = run(cuda_device, b, [16], 4, 50, 4, q, lens=torch.tensor([5000], dtype=torch.int32))
    assert err == mi.MI_DEVERR_BAD_CONTEXT
    out, err = run(cuda_device, b, [16], 4, 50, 4, q, max_q=8)
    assert err == mi.MI_DEVERR_BAD_QUERY and torch.all(torch.isnan(out.float()))
    out, err = run(cuda_device, b, [16], 4, 50, 4, q, starts=torch.tensor([9, 3], dtype=torch.int32))
    assert err == mi.MI_DEVERR_BAD_QUERY and torch.all(torch.isnan(out.float()))


def test_where_blocks_sit_changes_nothing(cuda_device):
    lens, news = [900, 70, 1500], [900, 3, 200]
    a, q, kv = make(lens, news, 8, 2, 128, 400, 20, 50)
    out, _ = run(cuda_device, a, news, 8, 400, 20, q)
    b, _, _ = make(lens, news, 8, 2, 128, 400, 20, 50, width=2000)
    perm = torch.randperm(b.num_blocks, generator=torch.Generator().manual_seed(1))
    b.k[perm], b.v[perm] = a.k.clone(), a.v.clone()
    b.tables[:, :a.width] = torch.where(a.tables >= 0, perm.to(torch.int32)[a.tables.clamp(min=0).long()], a.tables)
    again, _ = run(cuda_device, b, news, 8, 400, 20, q)
    assert torch.equal(out.view(torch.int16), again.view(torch.int16))


def test_graph_and_streams(cuda_device):
    sets = []
    for seed, (lens, news) in ((51, ([900, 70], [900, 3])), (52, ([1500], [700]))):
        b, q, kv = make(lens, news, 8, 2, 128, 400, 20, seed)
        want, _ = run(cuda_device, b, news, 8, 400, 20, q)
        dev = dict(q=q.to(cuda_device), k=b.k.to(cuda_device), v=b.v.to(cuda_device), t=b.tables.to(cuda_device),
                   n=torch.tensor(lens, dtype=torch.int32, device=cuda_device),
                   s=torch.tensor([0] + list(torch.tensor(news).cumsum(0)), dtype=torch.int32, device=cuda_device),
                   out=torch.empty(want.shape, dtype=want.dtype, device=cuda_device))
        sets.append((b, news, dev, want))
    mi = _mi()

    def call(b, news, x):
        mi.check(mi.mi_paged_prefill_attention_sliding(
            mi.dims(len(b.lens), 8, 2, 128, b.num_blocks, b.width), sum(news), max(news), x["q"], x["k"], x["v"], x["t"],
            x["n"], x["s"], 400, 20, 128 ** -0.5, x["out"]))

    def same():
        torch.cuda.synchronize()
        for _, _, x, want in sets:
            assert torch.equal(x["out"].cpu().view(torch.int16), want.view(torch.int16))
            x["out"].fill_(float("nan"))
        torch.cuda.synchronize()

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for b, news, x, _ in sets:
            call(b, news, x)
    for _ in range(3):
        graph.replay()
        same()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        for (b, news, x, _), st in zip(sets, streams):
            with torch.cuda.stream(st):
                call(b, news, x)
        same()


def test_a_withheld_copy_times_out(cuda_device):
    mi = _mi()
    b, q, kv = make([900, 70], [900, 3], 8, 2, 128, 400, 20, 53)
    want, _ = run(cuda_device, b, [900, 3], 8, 400, 20, q)
    mi.check(mi.mi_test_set_wait_limit(1_000_000))
    mi.check(mi.mi_test_withhold_copy(True))
    try:
        _, err = run(cuda_device, b, [900, 3], 8, 400, 20, q)
    finally:
        mi.mi_test_withhold_copy(False)
        mi.mi_test_set_wait_limit(0)
    assert err & mi.MI_DEVERR_TIMEOUT
    out, err = run(cuda_device, b, [900, 3], 8, 400, 20, q)
    assert err == 0 and torch.equal(out.view(torch.int16), want.view(torch.int16))


@pytest.mark.parametrize("Hq,Hkv,d", [(4, 1, 64), (8, 2, 128), (3, 1, 128)])
def test_rows_wholly_before_position_0(cuda_device, Hq, Hkv, d):
    """Lengths far below the number of new tokens: whole tiles of rows come before
    position 0, around requests that are as they should be."""
    mi = _mi()
    lens, news = [300, 900, 40, 500], [300, 900, 7, 500]
    b, q, kv = make(lens, news, Hq, Hkv, d, 50, 4, 60, hide=False)
    short = torch.tensor([300, 20, 40, 0], dtype=torch.int32)
    b.lens = short.tolist()
    out, err = run(cuda_device, b, news, Hq, 50, 4, q, lens=short)
    assert err == mi.MI_DEVERR_BAD_QUERY
    out = out.double()
    assert torch.count_nonzero(out[300:1180]) == 0   # request 1: 900 rows, 20 of them at a position
    assert torch.count_nonzero(out[1207:]) == 0      # request 3: none
    G = Hq // Hkv
    for at, s, n, rows in ((0, 0, 300, (0, 63, 64, 200, 299)), (1180, 1, 20, (0, 3, 19)), (1200, 2, 40, (33, 39))):
        for p in rows:
            t = torch.arange(p + 1)
            t = t[(t < 4) | (t > p - 50)]
            row = at + p - (33 if s == 2 else 0)
            for h in range(Hkv):
                ref, tol = attention_ref(q[row, h * G:(h + 1) * G].double(), *(x[t] for x in kv[s][h]), d ** -0.5)
                assert torch.all((out[row, h * G:(h + 1) * G] - ref).abs() <= tol), (s, p, h)


def test_many_requests(cuda_device):
    """More requests than one warp lays out, some without new tokens."""
    lens = [(37 * i) % 90 for i in range(1300)]
    news = [min(n, (5 * i) % 12) for i, n in enumerate(lens)]
    b, q, kv = make(lens, news, 4, 2, 64, 24, 2, 61)
    out, err = run(cuda_device, b, news, 4, 24, 2, q)
    assert err == 0 and torch.all(torch.isfinite(out.float()))
    check(b, kv, news, 4, 24, 2, q, out, rows=[0, 1, 7, -1])
