"""mi_paged_decode_attention_prefix against softmax attention over prefix and
own tokens in 64 bits, and against the plain decode call over joined tables."""
import numpy as np
import pytest
import torch

from paged_ref import Batch, attention_ref, blocks_of

pytestmark = pytest.mark.gpu


def _mi():
    import paged_kv_decode_25_gb300 as mi
    return mi


def make(prefixes, own, Hkv, d, seed):
    """One pool of blocks: sequences 0..P-1 are the prefixes, the rest the requests."""
    both = Batch(list(prefixes) + list(own), Hkv, d, seed)
    P = len(prefixes)
    pw = max([1] + [blocks_of(n) for n in prefixes])
    return both, both.tables[:P, :pw].contiguous(), both.tables[P:].contiguous()


def call(mi, dev, both, ptab, plens, starts, tables, lens, q, scale, space=None):
    B, Hq, d = q.shape
    d_ = mi.dims(B, Hq, both.Hkv, d, both.num_blocks, tables.shape[1])
    pw = max(ptab.shape[1], 1)
    n = mi.mi_paged_prefix_workspace_bytes(d_, len(plens), pw)
    assert n > 0
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device=dev) if space is None else space
    out = torch.full((B, Hq, d), float("nan"), dtype=torch.bfloat16, device=dev)
    err = torch.zeros(1, dtype=torch.int32, device=dev)

    def i32(x):
        return torch.tensor(x, dtype=torch.int32, device=dev)

    mi.check(mi.mi_paged_decode_attention_prefix(d_, len(plens), pw, q.to(dev), both.k.to(dev), both.v.to(dev),
                                                 ptab.to(dev) if len(plens) else None, i32(plens) if len(plens) else None,
                                                 i32(starts), tables.to(dev), i32(lens), scale, out, ws, dev_err=err))
    torch.cuda.synchronize()
    return out.cpu(), err.item()


def check(both, P, starts, lens, q, out, scale, drop=None):
    """drop(g): indices of the prefix's tokens that do not count."""
    B, Hq, d = q.shape
    G = Hq // both.Hkv
    worst = 0.0
    for b in range(B):
        g = next((i for i in range(P) if starts[i] <= b < starts[i + 1]), None)
        for h in range(both.Hkv):
            k, v = both.tokens(both.k, P + b, h)[:lens[b]], both.tokens(both.v, P + b, h)[:lens[b]]
            if g is not None:
                pk, pv = both.tokens(both.k, g, h), both.tokens(both.v, g, h)
                if drop is not None:
                    keep = [t for t in range(len(pk)) if t not in drop(g)]
                    pk, pv = pk[keep], pv[keep]
                k, v = torch.cat([pk, k]), torch.cat([pv, v])
            ref, tol = attention_ref(q[b, h * G:(h + 1) * G].double(), k, v, scale)
            err = (out[b, h * G:(h + 1) * G].double() - ref).abs()
            assert torch.all(err <= tol), (b, h, float((err / tol.clamp(min=1e-30)).max()))
            worst = max(worst, float(err.max()))
    return worst


@pytest.mark.parametrize("Hq,Hkv,d", [(4, 2, 64), (8, 8, 64), (3, 1, 128), (16, 8, 128), (28, 4, 128), (8, 1, 128), (10, 2, 64)])
def test_shapes(cuda_device, Hq, Hkv, d):
    """Groups of all sizes (one of them empty), prefixes that end inside a
    block, an empty prefix, empty own contexts, requests outside every group."""
    prefixes, starts = [100, 0, 333, 16, 1], [1, 8, 11, 11, 29, 30]
    own = [int(x) for x in np.random.default_rng(3).integers(0, 70, 33)]
    own[0], own[2], own[9], own[32] = 0, 0, 0, 5
    both, ptab, tables = make(prefixes, own, Hkv, d, 30)
    q = both.queries(len(own), Hq)
    out, err = call(_mi(), cuda_device, both, ptab, prefixes, starts, tables, own, q, d ** -0.5)
    assert err == 0
    check(both, 5, starts, own, q, out, d ** -0.5)


@pytest.mark.parametrize("n", [1, 15, 16, 17, 63, 64, 65, 127, 128, 129, 500, 4099])
@pytest.mark.parametrize("B", [1, 5, 40])
def test_prefix_lengths(cuda_device, n, B):
    own = [1 + (7 * b) % 20 for b in range(B)]
    both, ptab, tables = make([n], own, 2, 128, 31)
    q = both.queries(B, 8)
    out, err = call(_mi(), cuda_device, both, ptab, [n], [0, B], tables, own, q, 128 ** -0.5)
    assert err == 0
    check(both, 1, [0, B], own, q, out, 128 ** -0.5)


@pytest.mark.parametrize("B", [16, 31, 32, 33, 64, 65, 130, 300])
def test_group_sizes(cuda_device, B):
    own = [b % 3 for b in range(B)]
    both, ptab, tables = make([210], own, 1, 64, 32)
    q = both.queries(B, 4)
    out, err = call(_mi(), cuda_device, both, ptab, [210], [0, B], tables, own, q, 0.125)
    assert err == 0
    check(both, 1, [0, B], own, q, out, 0.125)


def test_many_groups(cuda_device):
    """More prefixes than a block has threads, some without requests."""
    rng = np.random.default_rng(4)
    P, sizes = 700, rng.integers(0, 4, 700)
    starts = [0] + np.cumsum(sizes).tolist()
    prefixes = [int(x) for x in rng.integers(0, 40, P)]
    own = [int(x) for x in rng.integers(0, 20, starts[-1])]
    both, ptab, tables = make(prefixes, own, 1, 64, 33)
    q = both.queries(len(own), 2)
    out, err = call(_mi(), cuda_device, both, ptab, prefixes, starts, tables, own, q, 0.125)
    assert err == 0
    check(both, P, starts, own, q, out, 0.125)


def test_many_requests_in_few_groups(cuda_device):
    """More requests than one warp plans for, lengths from none to many blocks."""
    rng = np.random.default_rng(5)
    B = 700
    own = [int(x) for x in rng.integers(0, 60, B)]
    own[3], own[699], own[350] = 900, 500, 0
    starts = [0, 0, 300, 640]
    both, ptab, tables = make([90, 700, 33], own, 1, 64, 35)
    q = both.queries(B, 4)
    out, err = call(_mi(), cuda_device, both, ptab, [90, 700, 33], starts, tables, own, q, 0.125)
    assert err == 0
    check(both, 3, starts, own, q, out, 0.125)


@pytest.mark.parametrize("prefix,own", [(5, [9000, 0, 3, 17000, 40]), (9000, [1, 0, 17, 40, 3]), (3000, [3000] * 9),
                                        (0, [700, 16, 0, 33])])
def test_parts_of_unequal_length(cuda_device, prefix, own):
    """Own tokens that outweigh the prefix, the reverse, and a prefix without tokens."""
    both, ptab, tables = make([prefix], own, 2, 128, 36)
    q = both.queries(len(own), 8)
    out, err = call(_mi(), cuda_device, both, ptab, [prefix], [0, len(own)], tables, own, q, 0.08)
    assert err == 0
    check(both, 1, [0, len(own)], own, q, out, 0.08)


def test_no_prefixes_is_plain_decode(cuda_device):
    """Without prefixes the call is plain decode attention up to the split: both
    lie within the roundings of the 64-bit value."""
    mi, dev = _mi(), cuda_device
    own = [1, 200, 0, 3333]
    both, ptab, tables = make([], own, 2, 128, 34)
    q = both.queries(4, 8)
    out, err = call(mi, dev, both, ptab, [], [0], tables, own, q, 0.1)
    assert err == 0
    d_ = mi.dims(4, 8, 2, 128, both.num_blocks, tables.shape[1])
    ws = torch.empty(mi.mi_paged_decode_workspace_bytes(d_), dtype=torch.uint8, device=dev)
    plain = torch.empty(4, 8, 128, dtype=torch.bfloat16, device=dev)
    mi.check(mi.mi_paged_decode_attention(d_, q.to(dev), both.k.to(dev), both.v.to(dev), tables.to(dev),
                                          torch.tensor(own, dtype=torch.int32, device=dev), 0.1, plain, ws))
    torch.cuda.synchronize()
    check(both, 0, [0], own, q, out, 0.1)
    check(both, 0, [0], own, q, plain.cpu(), 0.1)


def test_large_values_and_far_parts(cuda_device):
    """One part's keys outweigh the other's by far, both ways; infinite and NaN
    values in blocks that no row reads."""
    for lift in (0, 1):
        both, ptab, tables = make([300], [40, 40], 1, 128, 35)
        blk, off = both.rows(0) if lift == 0 else both.rows(1)
        q = both.queries(2, 4)
        both.k[blk, 0, off] = (both.k[blk, 0, off].float() * 6).to(torch.bfloat16)
        out, err = call(_mi(), cuda_device, both, ptab, [300], [0, 2], tables, [40, 40], q, 0.5)
        assert err == 0
        check(both, 1, [0, 2], [40, 40], q, out, 0.5)


@pytest.mark.parametrize("scale", [0.0, -0.2, 1.0])
def test_scales(cuda_device, scale):
    own = [40, 0, 3, 129]
    both, ptab, tables = make([700], own, 2, 64, 38)
    q = both.queries(4, 8)
    out, err = call(_mi(), cuda_device, both, ptab, [700], [0, 4], tables, own, q, scale)
    assert err == 0
    check(both, 1, [0, 4], own, q, out, scale)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("step", [60.0, -60.0, 6.0])
def test_logits_far_apart(cuda_device, d, step):
    """Logits that climb or fall along a prefix by hundreds: the reference of a
    row's sums moves many times, not at all, or once in a while."""
    own = [5, 200] + [1] * 40
    both, ptab, tables = make([3000], own, 1, d, 39)
    q = both.queries(len(own), 8)
    q[:, :, 0] = 2.0
    blk, off = both.rows(0)
    both.k[blk, 0, off, 0] = (torch.arange(3000) // 100 * step).to(torch.bfloat16)
    out, err = call(_mi(), cuda_device, both, ptab, [3000], [0, len(own)], tables, own, q, 0.5)
    assert err == 0
    check(both, 1, [0, len(own)], own, q, out, 0.5)


def test_device_errors(cuda_device):
    mi, dev = _mi(), cuda_device
    own = [10, 20, 30]
    both, ptab, tables = make([100, 64], own, 2, 64, 36)
    q = both.queries(3, 4)
    # groups out of order or out of range: own tokens only
    for starts in ([2, 1, 3], [0, 4, 4], [-1, 2, 3], [0, 2, -1], [0, 2, 4]):
        out, err = call(mi, dev, both, ptab, [100, 64], starts, tables, own, q, 0.125)
        assert err == mi.MI_DEVERR_BAD_QUERY
        check(both, 2, [0, 0, 0], own, q, out, 0.125)
    # a bad block of the prefix drops its keys
    bad = ptab.clone()
    bad[0, 2], bad[1, 0] = both.num_blocks, -2
    out, err = call(mi, dev, both, bad, [100, 64], [0, 2, 3], tables, own, q, 0.125)
    assert err == mi.MI_DEVERR_BAD_BLOCK
    check(both, 2, [0, 2, 3], own, q, out, 0.125, drop=lambda g: range(32, 48) if g == 0 else range(16))
    # a prefix of bad blocks only
    out, err = call(mi, dev, both, torch.full_like(ptab, -1), [100, 64], [0, 2, 3], tables, own, q, 0.125)
    assert err == mi.MI_DEVERR_BAD_BLOCK
    check(both, 2, [0, 0, 0], own, q, out, 0.125)
    # a prefix length past its table is cut (here the table's blocks are full)
    out, err = call(mi, dev, both, ptab[1:, :4].contiguous(), [1000], [2, 3], tables, own, q, 0.125)
    assert err == mi.MI_DEVERR_BAD_CONTEXT
    want, tol = zip(*[attention_ref(q[2, 2 * h:2 * h + 2].double(),
                                    torch.cat([both.tokens(both.k, 1, h), both.tokens(both.k, 4, h)]),
                                    torch.cat([both.tokens(both.v, 1, h), both.tokens(both.v, 4, h)]), 0.125)
                      for h in range(2)])
    assert torch.all((out[2].double() - torch.cat(want)).abs() <= torch.cat(tol))


@pytest.mark.parametrize("P", [3, 32, 33, 60])
def test_last_group_ends_before_it_starts(cuda_device, P):
    """It is empty; the groups before it are as given."""
    B = P + 2
    own, prefixes = [b % 7 for b in range(B)], [20 + g % 50 for g in range(P)]
    both, ptab, tables = make(prefixes, own, 1, 64, 37)
    q = both.queries(B, 2)
    for end in (0, 1, P - 2, P - 1):
        starts = list(range(P)) + [end]
        out, err = call(_mi(), cuda_device, both, ptab, prefixes, starts, tables, own, q, 0.125)
        assert err == 0
        check(both, P, starts, own, q, out, 0.125)


def test_paging_does_not_matter_and_repeat(cuda_device):
    """The same bits wherever the blocks sit, run after run and replayed."""
    mi, dev = _mi(), cuda_device
    own = [33, 1, 0, 500]
    both, ptab, tables = make([700], own, 2, 128, 37)
    q = both.queries(4, 8)
    out, _ = call(mi, dev, both, ptab, [700], [0, 3], tables, own, q, 0.09)
    move = torch.randperm(both.num_blocks)
    back = torch.empty_like(move)
    back[move] = torch.arange(both.num_blocks)
    both.k, both.v = both.k[back], both.v[back]
    ptab2, tables2 = (torch.where(t >= 0, move[t.clamp(min=0).long()].to(torch.int32), t) for t in (ptab, tables))
    again, _ = call(mi, dev, both, ptab2, [700], [0, 3], tables2, own, q, 0.09)
    assert torch.equal(out.view(torch.int16), again.view(torch.int16))

    def i32(x):
        return torch.tensor(x, dtype=torch.int32, device=dev)

    d_ = mi.dims(4, 8, 2, 128, both.num_blocks, tables.shape[1])
    ws = torch.empty(mi.mi_paged_prefix_workspace_bytes(d_, 1, ptab.shape[1]), dtype=torch.uint8, device=dev)
    args = (d_, 1, ptab.shape[1], q.to(dev), both.k.to(dev), both.v.to(dev), ptab2.to(dev), i32([700]), i32([0, 3]),
            tables2.to(dev), i32(own), 0.09)
    res = torch.empty(4, 8, 128, dtype=torch.bfloat16, device=dev)
    mi.check(mi.mi_paged_decode_attention_prefix(*args, res, ws))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        mi.check(mi.mi_paged_decode_attention_prefix(*args, res, ws))
    for _ in range(3):
        res.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out.view(torch.int16), res.cpu().view(torch.int16))


def test_shared_blocks(cuda_device):
    """The same block in a prefix, in two requests and twice in one table."""
    mi, dev = _mi(), cuda_device
    both, ptab, tables = make([48], [48, 48], 1, 64, 38)
    tables = ptab[0].repeat(2, 1)
    tables[1, 1] = tables[1, 0]
    q = both.queries(2, 2)
    out, err = call(mi, dev, both, ptab, [48], [0, 2], tables, [48, 40], q, 0.125)
    assert err == 0
    both.tables[1], both.tables[2] = tables[0], tables[1]
    check(both, 1, [0, 2], [48, 40], q, out, 0.125)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("step", [1.0, 5.0, 30.0, -5.0])
@pytest.mark.parametrize("size", [0, 80, 110, -110])
def test_large_and_small_values(cuda_device, d, step, size):
    """Values of 2^size while the logits climb or fall by `step` every 100
    tokens (24 prefixes of 8 heads, so that one block takes many keys): sums of
    weights times values stay in range wherever one softmax over both parts has
    them there."""
    P, prefixes, own = 24, [700] * 24, [30] + [0] * 23
    both, ptab, tables = make(prefixes, own, 8, d, 32)
    q = both.queries(P, 16)
    q[:, :, 0] = 2.0
    for s in range(P):
        blk, off = both.rows(s, 700)
        both.k[blk, :, off, 0] = (torch.arange(700) // 100 * step).to(torch.bfloat16)[:, None]
    plain = both.v
    both.v = both.v * 2.0 ** size  # (exact)
    out, err = call(_mi(), cuda_device, both, ptab, prefixes, list(range(P + 1)), tables, own, q, 0.5)
    assert err == 0
    both.v = plain
    check(both, P, list(range(P + 1)), own, q, out.double() * 2.0 ** -size, 0.5)
