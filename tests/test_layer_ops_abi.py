"""Argument checks of the normed append and of the page moves, made before
anything is queued: no GPU, no device pointer is followed."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def mi():
    import paged_kv_decode_25_gb300 as m
    from paged_kv_decode_25_gb300 import build
    build.build()
    return m


P = 1 << 32  # stands for device buffers far apart: aligned, never read
BAD, UNSUPPORTED = 1, 4


def dims(mi, **kw):
    a = dict(B=2, Hq=8, Hkv=2, head_dim=128, num_blocks=64, max_blocks_per_seq=8, block_size=16)
    a.update(kw)
    return mi.dims(**a)


def norm(mi, fp8=False, d=None, q=P, k=2 * P, v=3 * P, qw=4 * P, kw=5 * P, eps=1e-6, pos=6 * P, slot=7 * P, rope=8 * P,
         max_pos=100, q_out=9 * P, kc=10 * P, vc=11 * P, ks=12 * P, vs=13 * P, strides=(1024, 256, 256)):
    fn = mi.mi_paged_kv_append_norm_fp8 if fp8 else mi.mi_paged_kv_append_norm
    args = (dims(mi) if d is None else d, q, k, v, qw, kw, eps, pos, slot, rope, max_pos, q_out, kc, vc)
    return fn(*args, *((ks, vs) if fp8 else ()), stream=0, strides=strides)


@pytest.mark.parametrize("fp8", [False, True])
def test_norm_refusals(mi, fp8):
    for change, st in [(dict(B=-1), BAD), (dict(B=(1 << 24) + 1), BAD), (dict(Hq=0), BAD), (dict(Hkv=0), BAD),
                       (dict(num_blocks=0), BAD), (dict(head_dim=96), UNSUPPORTED), (dict(block_size=32), UNSUPPORTED),
                       (dict(Hq=7), UNSUPPORTED), (dict(num_blocks=1 << 27), BAD),
                       (dict(Hq=1 << 25, Hkv=1 << 25), BAD)]:
        assert norm(mi, fp8, d=dims(mi, **change)) == st, change
    assert norm(mi, fp8, d=dims(mi, B=0)) == 0
    names = "q k v qw kw pos slot rope q_out kc vc".split() + (["ks", "vs"] if fp8 else [])
    for name in names:
        assert norm(mi, fp8, **{name: 0}) == BAD, name
    for name in "q k v qw kw rope q_out kc vc".split():
        assert norm(mi, fp8, **{name: 20 * P + 8}) == BAD, name
    for eps in (0.0, -1e-6, float("nan"), float("inf")):
        assert norm(mi, fp8, eps=eps) == BAD, eps
    assert norm(mi, fp8, max_pos=0) == BAD
    for strides in ((1023, 256, 256), (1016, 256, 256), (1024, 248, 256), (1024, 256, 0), (1024, -256, 256),
                    (1028, 256, 256), (1 << 40, 256, 256)):
        assert norm(mi, fp8, strides=strides) == BAD, strides


def test_norm_overlaps(mi):
    """q_out may be q row for row, nothing else that is read."""
    for at in (P + 2048, P + 16, P - 16):  # 2 rows of 1,024 elements
        assert norm(mi, q_out=at) == BAD
    for name in "k v".split():
        assert norm(mi, q_out=3 * P, **{name: 3 * P + 4096 - 16}) == BAD
        assert norm(mi, q_out=3 * P, **{name: 3 * P}) == BAD
    assert norm(mi, q_out=P, strides=(1032, 256, 256)) == BAD  # q's rows lie apart, q_out's do not
    assert norm(mi, q_out=P + 4096, strides=(1 << 20, 256, 256)) == BAD  # between q's rows


def planes(mi, rows=((P, 4, 16),), src=2 * P, dst=3 * P, n=1, count=None):
    a = (mi.MiKvPlane * max(1, len(rows)))(*(mi.MiKvPlane(*r) for r in rows))
    return mi.mi_kv_copy_planes((a, len(rows) if count is None else count), src, dst, n, stream=0)


def test_plane_refusals(mi):
    assert planes(mi, n=0) == 0 and planes(mi, rows=()) == 0
    assert planes(mi, n=-1) == BAD and planes(mi, count=-1) == BAD
    assert mi.load().mi_kv_copy_planes(None, 1, 2 * P, 3 * P, 1, None, None) == BAD
    assert mi.load().mi_kv_copy_planes(None, 0, 2 * P, 3 * P, 1, None, None) == 0
    for row in ((0, 4, 16), (P + 2, 4, 16), (P, 0, 16), (P, -1, 16), (P, 1 << 31, 16), (P, 4, 0), (P, 4, 2), (P, 4, 18),
                (P, 4, -4), (P, 1 << 20, 1 << 21), (P, 1, 1 << 62)):
        assert planes(mi, rows=((P, 4, 16), row)) == BAD, row
        assert planes(mi, rows=((P, 4, 16), row), n=0) == BAD, row
    for name in ("src", "dst"):
        assert planes(mi, **{name: 0}) == BAD and planes(mi, **{name: P + 2}) == BAD


def test_planes_of_tensors(mi):
    torch = pytest.importorskip("torch")
    x = torch.zeros(7, 2, 16, 64, dtype=torch.bfloat16)
    y = torch.zeros(7, 2)
    a, n = mi.kv_planes([x, y])
    assert n == 2 and ctypes.sizeof(mi.MiKvPlane) == 24
    assert (a[0].base, a[0].rows, a[0].row_bytes) == (x.data_ptr(), 7, 2 * 16 * 64 * 2)
    assert (a[1].base, a[1].rows, a[1].row_bytes) == (y.data_ptr(), 7, 8)
    with pytest.raises(AssertionError):
        mi.kv_planes([x.transpose(1, 2)])


def sliding(mi, kind="bf16", d=None, q=P, k=2 * P, v=3 * P, ks=4 * P, vs=5 * P, tab=6 * P, lens=7 * P, window=10, sinks=2,
            scale=0.1, out=8 * P, ws=9 * P, nbytes=1 << 40):
    fn = {"bf16": mi.mi_paged_decode_attention_sliding, "fp8": mi.mi_paged_decode_attention_sliding_fp8,
          "int8": mi.mi_paged_decode_attention_sliding_int8}[kind]
    return fn(dims(mi) if d is None else d, q, k, v, *(() if kind == "bf16" else (ks, vs)), tab, lens, window, sinks, scale,
              out, ws, workspace_bytes=nbytes, stream=0)


BAD_DIMS = [(dict(B=-1), 1), (dict(B=65536), 1), (dict(Hq=0), 1), (dict(Hkv=0), 1), (dict(num_blocks=0), 1),
            (dict(max_blocks_per_seq=0), 1), (dict(head_dim=96), 4), (dict(head_dim=256), 4), (dict(block_size=32), 4),
            (dict(Hq=7, Hkv=2), 4), (dict(Hq=9, Hkv=1), 4), (dict(num_blocks=1 << 27, Hkv=8, Hq=8), 1),
            (dict(max_blocks_per_seq=(1 << 27) - 127), 1), (dict(B=65535, Hkv=1 << 15, Hq=1 << 15, num_blocks=1), 1)]


@pytest.mark.parametrize("kind", ["bf16", "fp8", "int8"])
def test_sliding_refusals(mi, kind):
    for change, st in BAD_DIMS:
        assert sliding(mi, kind, d=dims(mi, **change)) == st, change
    assert sliding(mi, kind, d=dims(mi, B=0)) == 0
    for kw in (dict(window=0), dict(window=-1), dict(sinks=-1), dict(scale=float("nan")), dict(scale=float("inf"))):
        assert sliding(mi, kind, **kw) == BAD, kw
    for name in "q k v tab lens out ws".split() + (["ks", "vs"] if kind != "bf16" else []):
        assert sliding(mi, kind, **{name: 0}) == BAD, name
    for name in "q k v out ws".split():
        assert sliding(mi, kind, **{name: 20 * P + 8}) == BAD, name
    if kind != "bf16":
        assert sliding(mi, kind, ks=20 * P + 2) == BAD and sliding(mi, kind, vs=20 * P + 1) == BAD
    for change, _ in BAD_DIMS:
        assert mi.mi_paged_sliding_workspace_bytes(dims(mi, **change), 10, 2) == 0
    assert mi.mi_paged_sliding_workspace_bytes(dims(mi), 0, 2) == 0
    assert mi.mi_paged_sliding_workspace_bytes(dims(mi), 1, -1) == 0


def sliding_prefill(mi, d=None, total=4, most=4, q=P, k=2 * P, v=3 * P, tab=4 * P, lens=5 * P, starts=6 * P, window=10,
                    sinks=2, scale=0.1, out=7 * P):
    return mi.mi_paged_prefill_attention_sliding(dims(mi) if d is None else d, total, most, q, k, v, tab, lens, starts,
                                                 window, sinks, scale, out, stream=0)


def test_sliding_prefill_refusals(mi):
    for change, st in BAD_DIMS:
        if change.get("B", 0) <= 0:  # (any number of requests, and they need not fit 2^30 heads)
            assert sliding_prefill(mi, d=dims(mi, **change)) == st, change
    for kw in (dict(window=0), dict(window=-1), dict(sinks=-1), dict(scale=float("nan")), dict(scale=float("inf")),
               dict(total=-1), dict(most=-1), dict(total=1 << 30), dict(most=1 << 30)):
        assert sliding_prefill(mi, **kw) == BAD, kw
    for kw in (dict(total=0), dict(most=0), dict(d=dims(mi, B=0))):
        assert sliding_prefill(mi, **kw) == 0, kw
    for name in "q k v tab lens starts out".split():
        assert sliding_prefill(mi, **{name: 0}) == BAD, name
    for name in "q k v out".split():
        assert sliding_prefill(mi, **{name: 20 * P + 8}) == BAD, name
    assert mi.load().mi_paged_prefill_attention_sliding(None, 4, 4, P, P, P, P, P, P, 1, 0, 0.1, P, None, None) == BAD


def test_pieces_stay_within_the_places():
    """The plan's cuts, in fp32 as every block of the launch computes them: pieces of split
    units never outnumber the workspace's places (8 per warp and 64)."""
    import random

    import numpy as np
    f, r = np.float32, random.Random(74)
    for _ in range(300):
        warps = f(r.choice((12, 1776, 1824)))
        units = int(np.exp(r.uniform(0, np.log(60000))))
        hi = int(np.exp(r.uniform(0, np.log(20000))))
        nb = np.random.default_rng(r.randrange(1 << 30)).integers(r.choice((1, max(1, hi // 2), hi)), hi + 1, units)
        least = max(f(1), np.ceil(f(2) * f(nb.sum()) / (f(8) * warps)))
        for step in (least, least + 1, 2 * least):  # no cut is finer than the first
            pieces = -(-nb // int(step))
            assert pieces[pieces > 1].sum() <= 8 * warps + 64
