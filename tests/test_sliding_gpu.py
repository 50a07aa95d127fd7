"""mi_paged_decode_attention_sliding (bf16, e4m3, INT8) against 64 bits. Tokens out
of sight hold NaN in the caches (bf16, e4m3), and the table columns of blocks
that are out of sight hold -1."""
import pytest
import torch

from paged_ref import BF16_HALF, BLOCK, FP32_HALF, Batch, attention_ref, logit_slack

pytestmark = pytest.mark.gpu


def _mi():
    import paged_kv_decode_25_gb300 as mi
    return mi


def sight(n, window, sinks):
    t = torch.arange(n)
    return t[(t < sinks) | (t >= n - window)]


def int8_slack(q, v, k_amax, v_amax, scale):
    """What INT8 caches add to attention_ref's tolerance. Codes enter as 1152 + code:
    the bias's products cancel, and what is left of them is their rounding: d (for the
    scores) and n (for the outputs) products of up to 1280, a step of 2^-23 each, times
    the block's factor; the weights are rounded to f16 (half a step 2^-11)."""
    am, vm = float(k_amax) / 127, float(v_amax) / 127
    bias = 1280 * float(q.abs().sum(-1).max()) * am * abs(scale) * 2.0 ** -23 * (q.shape[-1] / 16 + 4)
    return 4 * bias * v.abs().max() + 1280 * vm * 2.0 ** -23 * 64


class Case:
    """A batch in a cache of `kind`, and what its requests see."""

    def __init__(self, lens, Hq, Hkv, d, window, sinks, seed, kind="bf16", width=None, hide=True):
        self.b = Batch(lens, Hkv, d, seed, width=width, fp8=kind == "fp8")
        self.Hq, self.window, self.sinks, self.kind = Hq, window, sinks, kind
        b = self.b
        self.q = b.queries(len(lens), Hq)
        self.scales = None
        if kind == "fp8":
            self.scales = [0.5 + torch.rand(Hkv, generator=b.gen) for _ in range(2)]
        elif kind == "int8":
            self.scales = [1.0 + 3 * torch.rand(b.num_blocks, Hkv, generator=b.gen) for _ in range(2)]
            b.k, b.v = (torch.randint(-127, 128, b.k.shape, generator=b.gen, dtype=torch.int8) for _ in range(2))
        self.kv = [[self.tokens(s, h) for h in range(Hkv)] for s in range(len(lens))]
        if hide:
            for s, n in enumerate(lens):
                t = torch.arange(n)
                seen = (t < sinks) | (t >= n - window)
                blk, off = b.rows(s)
                if kind != "int8":
                    for c in (b.k, b.v):
                        raw = c.view(torch.uint8) if kind == "fp8" else c.view(torch.int16)
                        raw[blk[~seen], :, off[~seen]] = 0x7F if kind == "fp8" else 0x7FC0
                for j in range(-(-n // BLOCK)):
                    if not seen[j * BLOCK:(j + 1) * BLOCK].any():
                        b.tables[s, j] = -1

    def tokens(self, s, h):
        b = self.b
        blk, off = b.rows(s)
        if self.kind == "int8":
            return tuple(c[blk, h, off].double() * m[blk, h].double()[:, None] / 127
                         for c, m in ((b.k, self.scales[0]), (b.v, self.scales[1])))
        f = (1.0, 1.0) if self.scales is None else [x[h].double() for x in self.scales]
        return b.tokens(b.k, s, h) * f[0], b.tokens(b.v, s, h) * f[1]

    def call(self, dev, out=None, ws=None, stream=None, err=None, lens=None, scale=None):
        mi, b = _mi(), self.b
        B = len(b.lens)
        d_ = mi.dims(B, self.Hq, b.Hkv, b.d, b.num_blocks, b.tables.shape[1])
        n = mi.mi_paged_sliding_workspace_bytes(d_, self.window, self.sinks)
        assert n > 0
        if not hasattr(self, "dev"):
            self.dev = dict(q=self.q.to(dev), k=b.k.to(dev), v=b.v.to(dev), tables=b.tables.to(dev),
                            lens=torch.tensor(b.lens, dtype=torch.int32, device=dev),
                            scales=[] if self.scales is None else [x.to(dev) for x in self.scales])
        x = self.dev
        self.ws = torch.full((n,), 0xFF, dtype=torch.uint8, device=dev) if ws is None else ws
        out = torch.full((B, self.Hq, b.d), float("nan"), dtype=torch.bfloat16, device=dev) if out is None else out
        err = torch.zeros(1, dtype=torch.int32, device=dev) if err is None else err
        fn = {"bf16": mi.mi_paged_decode_attention_sliding, "fp8": mi.mi_paged_decode_attention_sliding_fp8,
              "int8": mi.mi_paged_decode_attention_sliding_int8}[self.kind]
        self.scale = b.d ** -0.5 if scale is None else scale
        mi.check(fn(d_, x["q"], x["k"], x["v"], *x["scales"], x["tables"], x["lens"] if lens is None else lens, self.window,
                    self.sinks, self.scale, out, self.ws, dev_err=err, stream=stream))
        return out, err

    def check(self, out, lens=None):
        b, G = self.b, self.Hq // self.b.Hkv
        out = out.cpu()
        for s, n in enumerate(b.lens if lens is None else lens):
            t = sight(n, self.window, self.sinks)
            if len(t) == 0:
                assert torch.count_nonzero(out[s].float()) == 0
                continue
            for h in range(b.Hkv):
                k, v = (x[t] for x in self.kv[s][h])
                q = self.q[s, h * G:(h + 1) * G].double()
                ref, tol = attention_ref(q, k, v, self.scale)
                if self.kind == "int8":
                    tol = tol + int8_slack(q, v, self.scales[0].max(), self.scales[1].max(), self.scale)
                elif self.kind == "fp8":
                    slack = logit_slack(q, k, self.scale) + float((q @ k.T).abs().max()) * abs(self.scale) * 4 * FP32_HALF
                    tol = tol + 4 * slack * v.abs().max()
                err = (out[s, h * G:(h + 1) * G].double() - ref).abs()
                assert torch.all(err <= tol), (s, h, float((err / tol).max()))


SHAPES = [(4, 2, 64), (8, 8, 64), (3, 1, 128), (16, 8, 128), (28, 4, 128), (8, 1, 128), (10, 2, 64)]
KINDS = ["bf16", "fp8", "int8"]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("Hq,Hkv,d", SHAPES)
def test_shapes(cuda_device, Hq, Hkv, d, kind):
    c = Case([1, 17, 0, 64, 333, 16, 1200], Hq, Hkv, d, 100, 4, 20, kind)
    out, err = c.call(cuda_device)
    torch.cuda.synchronize()
    assert err.item() == 0
    c.check(out)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("window", [1, 2, 15, 16, 17, 64, 250, 256, 100000, 2 ** 31 - 1])
@pytest.mark.parametrize("sinks", [0, 1, 16, 17, 100, 2 ** 31 - 1])
def test_windows_and_sinks(cuda_device, window, sinks, kind):
    """Sinks that end inside a block, inside the window, behind the context."""
    lens = [1, 2, 15, 16, 17, 18, 31, 32, 33, 64, 65, 100, 255, 256, 257, 300]
    c = Case(lens, 4, 1, 64, window, sinks, 21, kind)
    out, err = c.call(cuda_device)
    torch.cuda.synchronize()
    assert err.item() == 0
    c.check(out)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("lens,window,sinks", [
    ([30000], 20000, 64),                   # one request over every warp
    ([20000] + [40] * 200, 16384, 0),       # one long among short ones
    ([3000] * 300, 200, 5),                 # more units than warps
    ([700] * 5, 10 ** 9, 0)])               # no window at all
def test_plans(cuda_device, lens, window, sinks, kind):
    c = Case(lens, 8, 2, 64, window, sinks, 22, kind)
    out, err = c.call(cuda_device)
    torch.cuda.synchronize()
    assert err.item() == 0
    c.check(out)
    again, _ = c.call(cuda_device)
    assert torch.equal(out.view(torch.int16), again.view(torch.int16))


@pytest.mark.parametrize("kind", KINDS)
def test_many_requests(cuda_device, kind):
    """Batches past 512 requests plan with the whole block."""
    g = torch.Generator().manual_seed(23)
    lens = torch.randint(0, 60, (700,), generator=g).tolist()
    lens[3], lens[699], lens[350] = 2500, 900, 0
    c = Case(lens, 4, 2, 64, 700, 3, 23, kind)
    out, err = c.call(cuda_device)
    torch.cuda.synchronize()
    assert err.item() == 0
    c.check(out)


def test_whole_context_equals_decode_attention(cuda_device):
    """A window past every context: mi_paged_decode_attention's result, up to fp32
    rounding of the split and its rounding to bf16."""
    mi = _mi()
    c = Case([1, 500, 16, 2000], 8, 2, 128, 1 << 20, 0, 24)
    out, _ = c.call(cuda_device)
    b, x = c.b, c.dev
    d_ = mi.dims(4, 8, 2, 128, b.num_blocks, b.width)
    ws = torch.empty(mi.mi_paged_decode_workspace_bytes(d_), dtype=torch.uint8, device=cuda_device)
    want = torch.empty_like(out)
    mi.check(mi.mi_paged_decode_attention(d_, x["q"], x["k"], x["v"], x["tables"], x["lens"], c.scale, want, ws))
    torch.cuda.synchronize()
    c.check(out)
    c.check(want)


def test_one_token_in_sight_is_its_value(cuda_device):
    for kind in ("bf16",):
        c = Case([1, 5, 16, 100, 999], 8, 2, 128, 1, 0, 25, kind)
        out, _ = c.call(cuda_device)
        out = out.cpu()
        for s, n in enumerate(c.b.lens):
            blk, off = c.b.tables[s, (n - 1) // BLOCK], (n - 1) % BLOCK
            want = c.b.v[blk.long(), :, off].repeat_interleave(4, 0)
            assert torch.equal(out[s].view(torch.int16), want.view(torch.int16))


def test_logits_far_apart_and_scales(cuda_device):
    for scale in (-0.3, 0.0, 20.0):
        c = Case([300, 40, 7], 4, 2, 64, 50, 4, 26)
        out, err = c.call(cuda_device, scale=scale)
        torch.cuda.synchronize()
        assert err.item() == 0
        assert torch.all(torch.isfinite(out.float()))
        c.check(out)


def test_bad_blocks_and_lengths(cuda_device):
    mi = _mi()
    c = Case([100, 300, 50], 8, 2, 64, 64, 4, 27, hide=False)
    c.b.tables[1, 16] = c.b.num_blocks  # in sight
    c.b.tables[1, 8] = -7               # out of sight
    out, err = c.call(cuda_device)
    torch.cuda.synchronize()
    assert err.item() == mi.MI_DEVERR_BAD_BLOCK
    t = sight(300, 64, 4)
    keep = t // 16 != 16
    for h in range(2):
        k, v = (x[t[keep]] for x in c.kv[1][h])
        ref, tol = attention_ref(c.q[1, 4 * h:4 * h + 4].double(), k, v, c.scale)
        assert torch.all((out[1, 4 * h:4 * h + 4].cpu().double() - ref).abs() <= tol)
    # a length past the table is cut to it; a negative one is an empty request
    c = Case([320, 300, 50], 8, 2, 64, 64, 4, 28, hide=False)
    lens = torch.tensor([5000, -3, 50], dtype=torch.int32, device=cuda_device)
    out, err = c.call(cuda_device, lens=lens)
    torch.cuda.synchronize()
    assert err.item() == mi.MI_DEVERR_BAD_CONTEXT
    c.check(out, lens=[320, 0, 50])


def test_tables_wider_than_needed(cuda_device):
    c = Case([33, 500, 0, 64], 4, 2, 64, 100, 16, 29, width=4000)
    out, err = c.call(cuda_device)
    torch.cuda.synchronize()
    assert err.item() == 0
    c.check(out)


def test_where_blocks_sit_changes_nothing(cuda_device):
    a = Case([900, 70, 3000], 8, 2, 128, 400, 20, 30)
    out, _ = a.call(cuda_device)
    b = Case([900, 70, 3000], 8, 2, 128, 400, 20, 30)
    perm = torch.randperm(b.b.num_blocks, generator=torch.Generator().manual_seed(1))
    b.b.k[perm], b.b.v[perm] = a.b.k.clone(), a.b.v.clone()
    b.b.tables = torch.where(a.b.tables >= 0, perm.to(torch.int32)[a.b.tables.clamp(min=0).long()], a.b.tables)
    again, _ = b.call(cuda_device)
    assert torch.equal(out.view(torch.int16), again.view(torch.int16))


def test_graphs_and_streams(cuda_device):
    """One workspace under two captured calls replayed in turn over poisoned
    outputs; two streams at once, each with a workspace of its own."""
    cases = [Case([5000, 40], 8, 2, 128, 4000, 16, 31), Case([3000] * 3, 8, 2, 128, 2500, 0, 32)]
    wants = []
    for c in cases:
        out, _ = c.call(cuda_device)
        c.check(out)
        wants.append(out.clone())
    ws = torch.full((max(c.ws.numel() for c in cases),), 0xFF, dtype=torch.uint8, device=cuda_device)
    outs = [torch.empty_like(w) for w in wants]
    graphs = []
    for c, o in zip(cases, outs):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            c.call(cuda_device, out=o, ws=ws, err=torch.zeros(1, dtype=torch.int32, device=cuda_device))
        graphs.append(graph)
    for _ in range(3):
        for o in outs:
            o.fill_(float("nan"))
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, wants):
            assert torch.equal(o.view(torch.int16), w.view(torch.int16))
    spaces = [torch.full_like(ws, 0xFF) for _ in cases]
    errs = [torch.zeros(1, dtype=torch.int32, device=cuda_device) for _ in cases]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        for o in outs:
            o.fill_(float("nan"))
        torch.cuda.synchronize()
        for c, o, w, e, st in zip(cases, outs, spaces, errs, streams):
            with torch.cuda.stream(st):
                c.call(cuda_device, out=o, ws=w, err=e)
        torch.cuda.synchronize()
        for o, w in zip(outs, wants):
            assert torch.equal(o.view(torch.int16), w.view(torch.int16))


@pytest.mark.parametrize("kind", KINDS)
def test_a_withheld_copy_times_out(cuda_device, kind):
    mi = _mi()
    c = Case([3000, 40, 500], 8, 2, 128, 2000, 16, 33, kind)
    want, _ = c.call(cuda_device)
    torch.cuda.synchronize()
    mi.check(mi.mi_test_set_wait_limit(1_000_000))
    mi.check(mi.mi_test_withhold_copy(True))
    try:
        _, err = c.call(cuda_device)
        torch.cuda.synchronize()
    finally:
        mi.mi_test_withhold_copy(False)
        mi.mi_test_set_wait_limit(0)
    assert err.item() & mi.MI_DEVERR_TIMEOUT
    out, err = c.call(cuda_device, ws=torch.zeros_like(c.ws))
    torch.cuda.synchronize()
    assert err.item() == 0 and torch.equal(out.view(torch.int16), want.view(torch.int16))


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
def test_units_that_end_in_the_same_two_warps(cuda_device, kind):
    """Split units of two pieces as far apart as there are warps: the same two warps
    finish all 20 of them, so one of the two finishes at least 10."""
    mi, dev = _mi(), cuda_device
    warps = 12 * torch.cuda.get_device_properties(dev).multi_processor_count
    g = torch.Generator().manual_seed(70)
    B, d, periods, long_n, pool = 20 * (warps - 1), 64, 20, 12 * BLOCK, 400
    lens = torch.randint(1, BLOCK + 1, (B,), generator=g, dtype=torch.int32)
    tables = torch.full((B, 12), -1, dtype=torch.int32)
    tables[:, 0] = torch.randint(0, pool, (B,), generator=g, dtype=torch.int32)
    long = torch.arange(periods) * (warps - 1)
    lens[long] = long_n
    tables[long] = torch.randint(0, pool, (periods, 12), generator=g, dtype=torch.int32)
    k, v = (torch.randn(pool, 1, BLOCK, d, generator=g).to(torch.bfloat16 if kind == "bf16" else torch.float8_e4m3fn)
            for _ in range(2))
    q = torch.randn(B, 1, d, generator=g).to(torch.bfloat16)
    D = mi.dims(B, 1, 1, d, pool, 12)
    ws = torch.full((mi.mi_paged_sliding_workspace_bytes(D, 1 << 20, 0),), 0xFF, dtype=torch.uint8, device=dev)
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    args = [q.to(dev), k.to(dev), v.to(dev)]
    fn = mi.mi_paged_decode_attention_sliding
    if kind == "fp8":
        fn, args = mi.mi_paged_decode_attention_sliding_fp8, args + [torch.ones(1, device=dev)] * 2
    outs = []
    for _ in range(3):
        out = torch.full((B, 1, d), float("nan"), dtype=torch.bfloat16, device=dev)
        mi.check(fn(D, *args, tables.to(dev), lens.to(dev), 1 << 20, 0, d ** -0.5, out, ws, dev_err=err))
        outs.append(out.cpu())
    assert err.item() == 0
    assert torch.equal(outs[0].view(torch.int16), outs[1].view(torch.int16))
    assert torch.equal(outs[0].view(torch.int16), outs[2].view(torch.int16))
    out, qd, k, v = outs[0][:, 0].double(), q.double(), k[:, 0].double(), v[:, 0].double()

    def fp8_slack(x, slack, v_max):  # as in Case.check
        return 4 * (slack + x.abs().amax(-1) * 4 * FP32_HALF) * v_max if kind == "fp8" else 0 * slack

    for s in long.tolist():
        kk, vv = (x[tables[s].long()].reshape(-1, d) for x in (k, v))
        ref, tol = attention_ref(qd[s], kk, vv, d ** -0.5)
        more = fp8_slack(qd[s] @ kk.T * d ** -0.5, torch.tensor([logit_slack(qd[s], kk, d ** -0.5)]), vv.abs().max())
        assert torch.all((out[s] - ref[0]).abs() <= tol[0] + more), s
    # the short ones all at once, by attention_ref's formula
    short = torch.ones(B, dtype=torch.bool)
    short[long] = False
    seen = torch.arange(BLOCK) < lens[short, None]
    qs, kk, vv = qd[short, 0], k[tables[short, 0].long()], v[tables[short, 0].long()] * seen[..., None]
    x = torch.einsum("bd,btd->bt", qs, kk) * d ** -0.5
    w = torch.softmax(x.masked_fill(~seen, float("-inf")), -1)
    ref, mag = torch.einsum("bt,btd->bd", w, vv), torch.einsum("bt,btd->bd", w, vv.abs())
    slack = (torch.einsum("bd,btd->bt", qs.abs(), kk.abs()) * seen).amax(-1) * d ** -0.5 * d * 2.0 ** -23
    tol = (BF16_HALF * (2 * ref.abs() + mag) + ((2 * slack + 64 * FP32_HALF) * 2)[:, None] * mag) * 1.01 + 1e-30
    more = fp8_slack(x * seen, slack, vv.abs().amax((1, 2)))
    assert torch.all((out[short] - ref).abs() <= tol + more[:, None])


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("Hq,Hkv,d", [(4, 2, 64), (7, 1, 128)])
def test_bad_blocks_on_either_side_of_a_pair(cuda_device, kind, Hq, Hkv, d):
    """One block of a request has a bad id, request by request another one, in windows
    of an odd and an even number of blocks: its tokens alone carry no weight."""
    mi = _mi()
    n, blocks = 16 * 9 + 5, 10
    for window in (16 * 5, 16 * 6, 1 << 20):
        c = Case([n] * blocks, Hq, Hkv, d, window, 4, 71, kind, hide=False)
        for s in range(blocks):
            c.b.tables[s, s] = -1 if s % 2 else c.b.num_blocks
        out, err = c.call(cuda_device)
        assert err.item() == mi.MI_DEVERR_BAD_BLOCK
        assert torch.all(torch.isfinite(out.float()))
        out = out.cpu()
        for s in range(blocks):
            t = sight(n, window, 4)
            t = t[t // BLOCK != s]
            for h in range(Hkv):
                k, v = (x[t] for x in c.kv[s][h])
                q = c.q[s, h * Hq // Hkv:(h + 1) * Hq // Hkv].double()
                ref, tol = attention_ref(q, k, v, c.scale)
                if kind == "int8":
                    tol = tol + int8_slack(q, v, c.scales[0].max(), c.scales[1].max(), c.scale)
                elif kind == "fp8":
                    slack = logit_slack(q, k, c.scale) + float((q @ k.T).abs().max()) * c.scale * 4 * FP32_HALF
                    tol = tol + 4 * slack * v.abs().max()
                got = out[s, h * Hq // Hkv:(h + 1) * Hq // Hkv].double()
                assert torch.all((got - ref).abs() <= tol), (window, s, h)


@pytest.mark.parametrize("spread", [1e2, 1e5])
def test_int8_value_factors_far_apart(cuda_device, spread):
    """Neighbouring blocks whose V factors differ by 1 to `spread`, in either order, zero
    ones among them. Weights times a block's factor over the largest are rounded to
    f16: by half a subnormal step, 2^-25 of the largest factor's values, at least."""
    lens = [1, 16, 17, 32, 33, 100, 500, 900]
    c = Case(lens, 4, 2, 64, 300, 20, 72, "int8")
    g = torch.Generator().manual_seed(73)
    c.scales[1] = torch.exp(torch.rand(c.b.num_blocks, 2, generator=g) * torch.log(torch.tensor(spread)))
    c.scales[1][torch.rand(c.b.num_blocks, 2, generator=g) < 0.1] = 0.0
    c.kv = [[c.tokens(s, h) for h in range(2)] for s in range(len(lens))]
    out, err = c.call(cuda_device)
    assert err.item() == 0
    out = out.cpu()
    for s, n in enumerate(lens):
        t = sight(n, 300, 20)
        for h in range(2):
            k, v = (x[t] for x in c.kv[s][h])
            q = c.q[s, 2 * h:2 * h + 2].double()
            ref, tol = attention_ref(q, k, v, c.scale)
            top = c.scales[1].max()
            tol = tol + int8_slack(q, v, c.scales[0].max(), top, c.scale) + len(t) * 2.0 ** -25 * float(top)
            assert torch.all((out[s, 2 * h:2 * h + 2].double() - ref).abs() <= tol), (s, h)
