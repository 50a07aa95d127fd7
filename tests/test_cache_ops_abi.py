"""Argument checks of the cache operators (made before anything is queued, so
they need no GPU and never follow a device pointer), workspace sizes, and
mi_kv_pool_shrink."""
import numpy as np
import pytest


@pytest.fixture(scope="module")
def mi():
    import paged_kv_decode_25_gb300 as m
    from paged_kv_decode_25_gb300 import build
    build.build()
    return m


P = 1 << 20  # stands for device buffers: aligned, never read
BIG = 1 << 40
BAD_DIMS = [(dict(B=-1), 1), (dict(B=65536), 1), (dict(Hq=0), 1), (dict(Hkv=0), 1), (dict(num_blocks=0), 1),
            (dict(max_blocks_per_seq=0), 1), (dict(head_dim=96), 4), (dict(head_dim=256), 4), (dict(block_size=32), 4),
            (dict(Hq=7, Hkv=2), 4), (dict(Hq=9, Hkv=1), 4), (dict(num_blocks=1 << 27, Hkv=8, Hq=8), 1),
            (dict(max_blocks_per_seq=1 << 27), 1)]


def dims(mi, **kw):
    a = dict(B=2, Hq=8, Hkv=2, head_dim=128, num_blocks=64, max_blocks_per_seq=8, block_size=16)
    a.update(kw)
    return mi.dims(**a)


def prefix(mi, d=None, P_=1, width=4, q=P, k=P, v=P, ptab=P, plens=P, starts=P, tab=P, lens=P, scale=0.1, out=P, ws=P,
           nbytes=BIG):
    return mi.mi_paged_decode_attention_prefix(dims(mi) if d is None else d, P_, width, q, k, v, ptab, plens, starts, tab,
                                               lens, scale, out, ws, workspace_bytes=nbytes, stream=0)


def scored(mi, d=None, q=P, k=P, v=P, tab=P, lens=P, scale=0.1, out=P, scores=P, ws=P, nbytes=BIG):
    return mi.mi_paged_decode_attention_scored(dims(mi) if d is None else d, q, k, v, tab, lens, scale, 0, out, scores, ws,
                                               workspace_bytes=nbytes, stream=0)


def window(mi, d=None, total=4, most=4, q=P, k=P, tab=P, lens=P, starts=P, scale=0.1, scores=P, ws=P, nbytes=BIG):
    return mi.mi_paged_prefill_scores(dims(mi) if d is None else d, total, most, q, k, tab, lens, starts, scale, 0, scores,
                                      ws, workspace_bytes=nbytes, stream=0)


def evict(mi, d=None, k=P, v=P, scores=P, tab=P, lens=2 * P, budgets=3 * P, recent=1, dst=4 * P, new=5 * P, ws=P,
          nbytes=BIG, fp8=False):
    fn = mi.mi_paged_kv_evict_fp8 if fp8 else mi.mi_paged_kv_evict
    return fn(dims(mi) if d is None else d, k, v, scores, tab, lens, budgets, recent, dst, new, ws, workspace_bytes=nbytes,
              stream=0)


@pytest.mark.parametrize("call", [prefix, scored, window, evict])
@pytest.mark.parametrize("change,status", BAD_DIMS)
def test_dims(mi, call, change, status):
    assert call(mi, d=dims(mi, **change)) == status


@pytest.mark.parametrize("call", [prefix, scored, window, evict])
def test_empty_batch(mi, call):
    assert call(mi, d=dims(mi, B=0)) == mi.MI_OK


@pytest.mark.parametrize("call,names", [
    (prefix, "q k v ptab plens starts tab lens out ws"), (scored, "tab lens scores ws"),
    (window, "q k tab lens starts scores ws"), (evict, "k v scores tab lens budgets dst new ws")])
def test_null(mi, call, names):
    for name in names.split():
        assert call(mi, **{name: 0}) == mi.MI_ERR_INVALID_ARG, name


@pytest.mark.parametrize("call,names", [(prefix, "q k v out ws"), (scored, "scores ws"), (window, "q k scores ws"),
                                        (evict, "k v scores ws")])
def test_misaligned(mi, call, names):
    for name in names.split():
        assert call(mi, **{name: P + 8}) == mi.MI_ERR_INVALID_ARG, name


def test_sizes(mi):
    bad = mi.MI_ERR_INVALID_ARG
    for kw in (dict(P_=-1), dict(P_=65536), dict(width=0), dict(width=1 << 27), dict(scale=float("nan")),
               dict(scale=float("inf"))):
        assert prefix(mi, **kw) == bad, kw
    for kw in (dict(total=-1), dict(most=-1), dict(total=1 << 30), dict(most=1 << 30), dict(scale=float("nan")),
               dict(nbytes=0)):
        assert window(mi, **kw) == bad, kw
    for kw in (dict(recent=-1), dict(nbytes=0), dict(lens=2 * P + 2), dict(new=5 * P + 1)):
        assert evict(mi, **kw) == bad, kw
        assert evict(mi, fp8=True, **kw) == bad, kw


def test_evict_overlaps(mi):
    bad = mi.MI_ERR_INVALID_ARG
    assert evict(mi, new=2 * P) == bad             # the lengths
    assert evict(mi, new=2 * P + 4) == bad
    assert evict(mi, new=3 * P) == bad             # the budgets
    assert evict(mi, new=P + 4 * 15) == bad        # the last table entry (2 x 8)
    assert evict(mi, new=4 * P - 4) == bad         # the first destination entry
    assert evict(mi, dst=P + 4) == bad             # a table shifted over the source's


def test_workspace_sizes(mi):
    assert mi.mi_paged_kv_evict_workspace_bytes(dims(mi)) >= 2 * 2 * 8 * 16 * 4
    assert mi.mi_paged_kv_evict_workspace_bytes(dims(mi, head_dim=96)) == 0
    assert mi.mi_paged_prefill_scores_workspace_bytes(dims(mi), 10, 10) >= 10 * 8 * 4
    assert mi.mi_paged_prefill_scores_workspace_bytes(dims(mi), -1, 10) == 0
    assert mi.mi_paged_prefill_scores_workspace_bytes(dims(mi, Hq=7), 10, 10) == 0
    assert mi.mi_paged_prefix_workspace_bytes(dims(mi), -1, 4) == 0
    assert mi.mi_paged_prefix_workspace_bytes(dims(mi), 1, 0) == 0
    assert mi.mi_paged_scored_workspace_bytes(dims(mi, head_dim=80)) == 0


# ------------------------------------------------------------------ shrink --

def test_shrink_returns_the_tail(mi):
    pool = mi.Pool(20, 4, 10)
    assert pool.alloc(0, 100) == 0 and pool.alloc(1, 17) == 0  # blocks 0..6 and 7, 8
    assert pool.shrink(0, 40) == 0
    bt, cl, sl = pool.batch_meta([0])
    assert cl[0] == 40 and bt[0].tolist() == [0, 1, 2] + [-1] * 7 and sl[0] == 2 * 16 + 7
    assert pool.num_free() == 20 - 9 + 4
    # pushed in table order 3, 4, 5, 6: the next pop is 6
    assert pool.alloc(2, 33) == 0
    assert pool.batch_meta([2])[0][0, :3].tolist() == [6, 5, 4]
    # growing again takes new blocks
    assert pool.alloc(0, 49) == 0
    assert pool.batch_meta([0])[0][0, :4].tolist() == [0, 1, 2, 3]


@pytest.mark.parametrize("n,blocks", [(100, 7), (97, 7), (96, 6), (17, 2), (16, 1), (1, 1), (0, 0)])
def test_shrink_sizes(mi, n, blocks):
    pool = mi.Pool(8, 1, 8)
    assert pool.alloc(0, 100) == 0
    assert pool.shrink(0, n) == 0
    assert pool.num_free() == 8 - blocks
    assert len(mi.mi_kv_pool_seq_blocks(pool.handle, 0)) == blocks
    assert pool.shrink(0, n) == 0 and pool.num_free() == 8 - blocks
    assert pool.free(0) == 0 and pool.num_free() == 8


def test_shrink_refusals(mi):
    pool = mi.Pool(8, 3, 8)
    assert pool.shrink(0, 0) == mi.MI_ERR_UNKNOWN_SEQ
    assert pool.shrink(-1, 0) == mi.MI_ERR_UNKNOWN_SEQ and pool.shrink(3, 0) == mi.MI_ERR_UNKNOWN_SEQ
    assert pool.alloc(0, 30) == 0
    assert pool.shrink(0, 31) == mi.MI_ERR_INVALID_ARG and pool.shrink(0, -1) == mi.MI_ERR_INVALID_ARG
    assert mi.mi_kv_pool_shrink(None, 0, 0) == mi.MI_ERR_INVALID_ARG
    assert pool.swap_out(0)[0] == 0
    assert pool.shrink(0, 10) == mi.MI_ERR_UNKNOWN_SEQ
    assert pool.swap_in(0)[0] == 0 and pool.shrink(0, 10) == 0 and pool.num_free() == 7


def test_shrink_among_other_calls(mi):
    """Blocks are never lost, doubled or shared over a random run of calls."""
    r = np.random.default_rng(8)
    pool, held = mi.Pool(60, 6, 20), {}
    for _ in range(3000):
        s = int(r.integers(6))
        if r.random() < 0.4:
            n = int(r.integers(0, 300))
            st = pool.shrink(s, n)
            assert (st == 0) == (s in held and n <= held[s])
            if st == 0:
                held[s] = n
        elif r.random() < 0.2:
            if pool.free(s) == 0:
                held.pop(s)
        else:
            n = held.get(s, 0) + int(r.integers(0, 60))
            if pool.alloc(s, n) == 0:
                held[s] = n
        blocks = [b for q in held for b in mi.mi_kv_pool_seq_blocks(pool.handle, q)]
        assert len(blocks) == len(set(blocks)) and len(blocks) + pool.num_free() == 60
        assert all(len(mi.mi_kv_pool_seq_blocks(pool.handle, q)) == -(-n // 16) for q, n in held.items())


def test_longest_tables(mi):
    """Tables of 2^27 - 128 blocks at most: the kernels look up to 1,024 tokens
    past a sequence's end, in 32 bits."""
    top = (1 << 27) - 128
    for call in (prefix, scored, window, evict):
        for width in (top + 1, (1 << 27) - 1):
            assert call(mi, d=dims(mi, max_blocks_per_seq=width)) == mi.MI_ERR_INVALID_ARG
    for size in (mi.mi_paged_kv_evict_workspace_bytes, lambda d: mi.mi_paged_prefill_scores_workspace_bytes(d, 4, 4)):
        assert size(dims(mi, max_blocks_per_seq=top)) > 0 and size(dims(mi, max_blocks_per_seq=top + 1)) == 0
    assert prefix(mi, width=top + 1) == mi.MI_ERR_INVALID_ARG
