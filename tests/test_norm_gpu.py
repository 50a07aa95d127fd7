"""mi_paged_kv_append_norm against the formula in 64 bits; what no token names
keeps its bits.

Tolerances: the result is rounded once (half a step: 2^-8 of a bf16 value, 2^-4
of an e4m3 one or 2^-10 below its normal range). Before that, in fp32, with
magnitudes m = |y c| + |y' s|: a sum of d squares (each value off by at most
d 2^-24 of itself in all, half of that in the root), r and the products (the
root within 2^-22, four more roundings), two products and their sum: below
(d / 2 + 16) 2^-24 m."""
import pytest
import torch

from paged_ref import BF16_HALF, FP32_HALF

pytestmark = pytest.mark.gpu
EPS, MAX_POS = 1e-6, 5000


def _mi():
    import paged_kv_decode_25_gb300 as mi
    return mi


def table(d, theta=1e6):
    a = torch.arange(MAX_POS, dtype=torch.float64)[:, None] * theta ** (-2 * torch.arange(d // 2, dtype=torch.float64) / d)
    return torch.stack([torch.cos(a), torch.sin(a)], -1).float()


def inputs(T, Hq, Hkv, d, seed, fused=False, gap=0):
    g = torch.Generator().manual_seed(seed)
    H = Hq + 2 * Hkv
    x = torch.randn(T, H, d, generator=g) * torch.exp(2 * torch.randn(T, H, 1, generator=g))
    x = x.to(torch.bfloat16).reshape(T, H * d)
    if fused:
        wide = torch.full((T, H * d + gap), float("nan"), dtype=torch.bfloat16)
        wide[:, :H * d] = x
        x = wide[:, :H * d]
    blocks = T // 8 + 4
    s = dict(q=x[:, :Hq * d], k=x[:, Hq * d:(Hq + Hkv) * d], v=x[:, (Hq + Hkv) * d:], blocks=blocks,
             qw=(1 + 0.3 * torch.randn(d, generator=g)).to(torch.bfloat16),
             kw=(1 + 0.3 * torch.randn(d, generator=g)).to(torch.bfloat16),
             pos=torch.randint(0, MAX_POS, (T,), generator=g, dtype=torch.int32),
             slot=torch.randperm(blocks * 16, generator=g)[:T].to(torch.int32), g=g)
    if not fused:
        s.update({n: s[n].contiguous() for n in "qkv"})
    return s


def heads(x, w, rope, pos, d):
    """(normed and rotated heads [T][H][d], magnitudes) in 64 bits."""
    x = x.double().reshape(x.shape[0], -1, d)
    y = x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS) * w.double()
    cs = rope.double()[pos.long()][:, None]
    c, s = cs[..., 0], cs[..., 1]
    a, b = y[..., :d // 2], y[..., d // 2:]
    return (torch.cat([a * c - b * s, b * c + a * s], -1),
            torch.cat([(a * c).abs() + (b * s).abs(), (b * c).abs() + (a * s).abs()], -1))


def close(got, want, mag, d, half=BF16_HALF, least=2.0 ** -134):
    err = (got.double() - want).abs()
    early = (d / 2 + 16) * FP32_HALF * mag
    tol = (half * (want.abs() + early) + early) * 1.01 + least
    assert torch.all(err <= tol), float((err / tol).max())


def to_dev(x, dev):
    """On the device with the row stride it has here."""
    if x.dim() == 2 and x.shape[0] > 1 and x.stride(0) != x.shape[1]:
        return torch.empty_strided((x.shape[0], x.stride(0)), (x.stride(0), 1), dtype=x.dtype,
                                   device=dev)[:, :x.shape[1]].copy_(x)
    return x.to(dev)


def run(dev, s, Hq, Hkv, d, scales=None, stream=None, in_place=False):
    mi = _mi()
    T = s["q"].shape[0]
    kind = torch.bfloat16 if scales is None else torch.float8_e4m3fn
    kc = torch.randn(s["blocks"], Hkv, 16, d, generator=s["g"]).to(kind)
    vc = torch.randn(s["blocks"], Hkv, 16, d, generator=s["g"]).to(kind)
    before = kc.clone(), vc.clone()
    q, k, v = (to_dev(s[n], dev) for n in "qkv")
    q_out = q if in_place else torch.full((T, Hq, d), float("nan"), dtype=torch.bfloat16, device=dev)
    rope = table(d).to(dev)
    kc, vc = kc.to(dev), vc.to(dev)
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    args = [mi.dims(T, Hq, Hkv, d, s["blocks"], 1), q, k, v, s["qw"].to(dev), s["kw"].to(dev), EPS, s["pos"].to(dev),
            s["slot"].to(dev), rope, MAX_POS, q_out, kc, vc]
    if scales is None:
        mi.check(mi.mi_paged_kv_append_norm(*args, dev_err=err, stream=stream))
    else:
        mi.check(mi.mi_paged_kv_append_norm_fp8(*args, scales[0].to(dev), scales[1].to(dev), dev_err=err, stream=stream))
    torch.cuda.synchronize()
    return q_out.cpu().reshape(T, Hq, d), kc.cpu(), vc.cpu(), before, err.item()


def bits(x):
    return x.view(torch.uint8) if x.element_size() == 1 else x.view(torch.int16)


def check(s, Hq, Hkv, d, got, scales=None, rows=None, k_heads=None, v_heads=None):
    """rows: those that were appended (default all); *_heads: KV heads that were stored."""
    q_out, kc, vc, before, _ = got
    T = s["q"].shape[0]
    rows = torch.arange(T) if rows is None else rows
    rope = table(d)
    want, mag = heads(s["q"], s["qw"], rope, s["pos"].clamp(0, MAX_POS - 1), d)
    close(q_out[rows], want[rows], mag[rows], d)
    want, mag = heads(s["k"], s["kw"], rope, s["pos"].clamp(0, MAX_POS - 1), d)
    slot = s["slot"].long()[rows]
    keep = (slot >= 0) & (slot < s["blocks"] * 16)
    rows, slot = rows[keep], slot[keep]
    blk, off = slot // 16, slot % 16
    for cache, old, ref, m, hs, i in ((kc, before[0], want, mag, k_heads, 0),
                                      (vc, before[1], s["v"].double().reshape(T, Hkv, d), None, v_heads, 1)):
        hs = list(range(Hkv)) if hs is None else hs
        touched = torch.zeros(s["blocks"], Hkv, 16, dtype=torch.bool)
        for h in hs:
            x = cache.float()[blk, h, off] if scales is not None else cache[blk, h, off]
            r, mm = ref[rows, h], torch.zeros_like(ref[rows, h]) if m is None else m[rows, h]
            if scales is not None:
                f = scales[i][h].double()
                r, mm = (r / f).clamp(-448, 448), mm / f + (r / f).abs() * (2 / (d / 2 + 16))
                close(x, r, mm, d, half=2.0 ** -4, least=2.0 ** -10)
            elif m is None:
                assert torch.equal(bits(x), bits(s["v"].reshape(T, Hkv, d)[rows, h].contiguous()))
            else:
                close(x, r, mm, d)
            touched[blk, h, off] = True
        assert torch.equal(bits(cache)[~touched], bits(old)[~touched])


SHAPES = [(4, 2, 64), (8, 8, 64), (3, 1, 128), (16, 8, 128), (28, 4, 128), (8, 1, 128), (10, 2, 64), (1, 1, 128),
          (40, 5, 64)]


@pytest.mark.parametrize("T", [1, 2, 7, 64, 700])
@pytest.mark.parametrize("Hq,Hkv,d", SHAPES)
def test_shapes(cuda_device, Hq, Hkv, d, T):
    s = inputs(T, Hq, Hkv, d, 1)
    got = run(cuda_device, s, Hq, Hkv, d)
    assert got[4] == 0
    check(s, Hq, Hkv, d, got)


@pytest.mark.parametrize("T,gap", [(1, 0), (5, 0), (33, 8), (3000, 64)])
@pytest.mark.parametrize("Hq,Hkv,d", [(4, 2, 64), (32, 8, 128)])
def test_rows_of_one_projection(cuda_device, Hq, Hkv, d, T, gap):
    s = inputs(T, Hq, Hkv, d, 2, fused=True, gap=gap)
    got = run(cuda_device, s, Hq, Hkv, d)
    assert got[4] == 0
    check(s, Hq, Hkv, d, got)


@pytest.mark.parametrize("T", [1, 50, 900])
@pytest.mark.parametrize("Hq,Hkv,d", [(4, 2, 64), (32, 8, 128), (7, 1, 128)])
def test_fp8(cuda_device, Hq, Hkv, d, T):
    s = inputs(T, Hq, Hkv, d, 3, fused=T > 1)
    # scales that clamp some values and push others below the normal range
    scales = [torch.exp(torch.linspace(-6, 3, Hkv)), torch.exp(torch.linspace(4, -5, Hkv))]
    got = run(cuda_device, s, Hq, Hkv, d, scales)
    assert got[4] == 0
    check(s, Hq, Hkv, d, got, scales)


def test_in_place(cuda_device):
    for T in (1, 40, 2000):
        s = inputs(T, 8, 2, 128, 4)
        got = run(cuda_device, s, 8, 2, 128, in_place=True)
        check(s, 8, 2, 128, got)


def test_edge_values(cuda_device):
    """Zero heads, tiny and huge ones, one value among zeros; position 0 and the last."""
    s = inputs(40, 4, 2, 128, 5)
    for n, per in (("q", 4), ("k", 2)):
        x = s[n].reshape(40, per, 128)
        x[0] = 0
        x[1] *= 2.0 ** -60
        x[2] *= 2.0 ** 50
        x[3] = 0
        x[3, :, 77] = 3.0
        x[4] = -1.0
    s["pos"][:6] = torch.tensor([0, MAX_POS - 1, 0, 17, 0, 1])
    got = run(cuda_device, s, 4, 2, 128)
    check(s, 4, 2, 128, got)
    assert torch.count_nonzero(got[0][0].float()) == 0


@pytest.mark.parametrize("T", [6, 2500])
def test_bad_positions_and_slots(cuda_device, T):
    mi = _mi()
    for bad, bit in (((-1, MAX_POS), mi.MI_DEVERR_BAD_POS), (None, mi.MI_DEVERR_BAD_SLOT)):
        s = inputs(T, 8, 2, 64, 6)
        rows = torch.ones(T, dtype=torch.bool)
        if bad:
            s["pos"][1], s["pos"][4] = bad
            rows[1] = rows[4] = False
        else:
            s["slot"][2], s["slot"][5] = -1, s["blocks"] * 16
        got = run(cuda_device, s, 8, 2, 64)
        assert got[4] == bit
        check(s, 8, 2, 64, got, rows=torch.nonzero(rows)[:, 0])
        assert torch.all(torch.isnan(got[0][~rows].float()))


def test_bad_scales_skip_their_heads(cuda_device):
    s = inputs(30, 8, 4, 128, 7)
    scales = [torch.tensor([0.1, 0.0, 0.2, float("nan")]), torch.tensor([float("inf"), 0.3, -1.0, 0.1])]
    got = run(cuda_device, s, 8, 4, 128, scales)
    assert got[4] == _mi().MI_DEVERR_BAD_SCALE
    check(s, 8, 4, 128, got, scales, k_heads=[0, 2], v_heads=[1, 3])


def test_same_as_the_plain_append_of_normed_heads(cuda_device):
    """With the norm done before, in 64 bits, and rounded to bf16, the append
    gives what this call gives up to that rounding."""
    mi = _mi()
    T, Hq, Hkv, d = 20, 8, 2, 128
    s = inputs(T, Hq, Hkv, d, 8)
    got = run(cuda_device, s, Hq, Hkv, d)
    q = s["q"].double().reshape(T, Hq, d)
    q = (q / torch.sqrt((q * q).mean(-1, keepdim=True) + EPS) * s["qw"].double()).to(torch.bfloat16).to(cuda_device)
    kc = torch.zeros(s["blocks"], Hkv, 16, d, dtype=torch.bfloat16, device=cuda_device)
    out = torch.empty_like(q)
    mi.check(mi.mi_paged_kv_append(mi.dims(T, Hq, Hkv, d, s["blocks"], 1), q, s["k"].to(cuda_device),
                                   s["v"].to(cuda_device), s["pos"].to(cuda_device), s["slot"].to(cuda_device),
                                   table(d).to(cuda_device), MAX_POS, out, kc, kc.clone()))
    # two roundings of bf16, the first one rotated: half a step of both terms
    want, mag = heads(s["q"], s["qw"], table(d), s["pos"], d)
    err = (out.cpu().double() - got[0].double()).abs()
    assert torch.all(err <= 2 * BF16_HALF * want.abs() + 1.02 * BF16_HALF * mag + 1e-30)


def test_graph_and_streams(cuda_device):
    """Captured and replayed over poisoned outputs, and on two streams at once."""
    mi = _mi()
    T, Hq, Hkv, d = 100, 8, 2, 128
    calls, want = [], []
    for seed in (11, 12):
        s = inputs(T, Hq, Hkv, d, seed)
        want.append(run(cuda_device, s, Hq, Hkv, d)[:3])
        dev = {n: s[n].to(cuda_device) for n in ("q", "k", "v", "qw", "kw", "pos", "slot")}
        dev.update(rope=table(d).to(cuda_device), q_out=torch.empty(T, Hq, d, dtype=torch.bfloat16, device=cuda_device),
                   blocks=s["blocks"], kc=torch.zeros(s["blocks"], Hkv, 16, d, dtype=torch.bfloat16, device=cuda_device))
        dev["vc"] = dev["kc"].clone()
        dev["at"] = (s["slot"].long() // 16, s["slot"].long() % 16)
        calls.append(dev)

    def call(x):
        mi.check(mi.mi_paged_kv_append_norm(mi.dims(T, Hq, Hkv, d, x["blocks"], 1), x["q"], x["k"], x["v"], x["qw"],
                                            x["kw"], EPS, x["pos"], x["slot"], x["rope"], MAX_POS, x["q_out"], x["kc"],
                                            x["vc"]))

    def same():
        torch.cuda.synchronize()
        for x, w in zip(calls, want):
            b, o = x["at"]
            assert torch.equal(bits(x["q_out"].cpu()), bits(w[0]))
            for got, ref in ((x["kc"], w[1]), (x["vc"], w[2])):
                assert torch.equal(bits(got.cpu()[b, :, o].contiguous()), bits(ref[b, :, o].contiguous()))

    def poison():
        for x in calls:
            for n in ("q_out", "kc", "vc"):
                x[n].fill_(float("nan"))
        torch.cuda.synchronize()

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for x in calls:
            call(x)
    for _ in range(3):
        poison()
        graph.replay()
        same()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        poison()
        for x, st in zip(calls, streams):
            with torch.cuda.stream(st):
                call(x)
        same()


@pytest.mark.parametrize("seed", range(4))
def test_e4m3_quotients_bit_for_bit(cuda_device, seed):
    """Every bf16 value over scales of all sizes (ones with all bits set, powers of two,
    denormal and near the largest): the code of the IEEE single precision quotient."""
    mi, dev = _mi(), cuda_device
    g = torch.Generator().manual_seed(seed)
    Hkv, d, T, NB = 32, 128, 512, 32
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    # a head has 512 x 128 values: each of them once
    v = torch.stack([bits[torch.randperm(65536, generator=g)].view(T, d) for _ in range(Hkv)], 1).contiguous()
    mant = 1 + torch.rand(Hkv, generator=g)
    scale = torch.ldexp(mant, torch.randint(-12, 4, (Hkv,), generator=g))
    scale[:12] = torch.ldexp(mant[:12], torch.randint(-126, 127, (12,), generator=g))
    scale[12:24] = torch.tensor([2 - 2.0 ** -23, 1.0, 2.0 ** -60, 2.0 ** -60 * (1 - 2.0 ** -24), 2.0 ** 60,
                                 2.0 ** 60 * (1 + 2.0 ** -23), 1 + 2.0 ** -23, 3.0, 1 / 3, 448.0, 1e-40, 3e38])
    q = torch.zeros(T, Hkv, d, dtype=torch.bfloat16, device=dev)
    w = torch.ones(d, dtype=torch.bfloat16, device=dev)
    rope = torch.zeros(1, d // 2, 2, device=dev)
    kc, vc = (torch.zeros(NB, Hkv, 16, d, dtype=torch.uint8, device=dev) for _ in range(2))
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    mi.check(mi.mi_paged_kv_append_norm_fp8(
        mi.dims(T, Hkv, Hkv, d, NB, 1), q, torch.zeros_like(q), v.to(dev), w, w, 1e-6,
        torch.zeros(T, dtype=torch.int32, device=dev), torch.arange(T, dtype=torch.int32, device=dev), rope, 1,
        torch.empty_like(q), kc, vc, torch.ones(Hkv, device=dev), scale.to(dev), dev_err=err))
    assert err.item() == 0
    got = vc.cpu().view(NB, Hkv, 16, d).transpose(1, 2).reshape(T, Hkv, d)
    want = (v.float() / scale[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    nan = torch.isnan(v.float())
    assert torch.all((got[nan] & 0x7F) == 0x7F)
    bad = (got != want) & ~nan
    assert not bad.any(), (int(bad.sum()), v[bad][:4].tolist(), got[bad][:4].tolist(), want[bad][:4].tolist())
