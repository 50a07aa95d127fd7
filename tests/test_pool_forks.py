"""mi_kv_pool_fork, _slide, _compact and _block_refs against a plain model of
tables and counts, and their refusals (CPU)."""
import numpy as np
import pytest


@pytest.fixture(scope="module")
def mi():
    import paged_kv_decode_25_gb300 as m
    from paged_kv_decode_25_gb300 import build
    build.build()
    return m


BAD, FULL, UNKNOWN = 1, 2, 3


class Model:
    """Tables as lists (None: given back), the free stack, tokens; blocks are
    counted by looking through the tables."""

    def __init__(self, blocks, seqs, width):
        self.blocks, self.seqs, self.width = blocks, seqs, width
        self.free_ids, self.tab, self.n, self.out = list(range(blocks))[::-1], {}, {}, {}

    def refs(self, b):
        return sum(t.count(b) for t in self.tab.values())

    def _drop(self, ids):
        """`ids` just left a table, in order."""
        for b in ids:
            if b is not None and self.refs(b) == 0:
                self.free_ids.append(b)

    def alloc(self, s, n):
        t = self.tab.get(s, [])
        if s in self.out or n < self.n.get(s, 0) or -(-n // 16) > self.width:
            return BAD
        extra = -(-n // 16) - len(t)
        if extra > len(self.free_ids):
            return FULL
        self.tab[s] = t + [self.free_ids.pop() for _ in range(extra)]
        self.n[s] = n
        return 0

    def free(self, s):
        if s in self.out:
            del self.out[s], self.n[s]
            return 0
        if s not in self.tab:
            return UNKNOWN
        self._drop(self.tab.pop(s))
        del self.n[s]
        return 0

    def shrink(self, s, n):
        if s not in self.tab:
            return UNKNOWN
        t, keep = self.tab[s], -(-n // 16)
        if n > self.n[s] or (n and t[keep - 1] is None) or (n % 16 and self.refs(t[keep - 1]) > 1):
            return BAD
        self.tab[s] = t[:keep]
        self._drop(t[keep:])
        self.n[s] = n
        return 0

    def fork(self, a, b, n, group):
        if a not in self.tab:
            return UNKNOWN, [], []
        if b in self.tab or b in self.out or n > self.n[a]:
            return BAD, [], []
        t, shared, every = self.tab[a], n // group * (group // 16), -(-n // 16)
        if None in t[shared:every] or (n and t[every - 1] is None):
            return BAD, [], []
        if every - shared > len(self.free_ids):
            return FULL, [], []
        new = [self.free_ids.pop() for _ in range(every - shared)]
        self.tab[b], self.n[b] = t[:shared] + new, n
        return 0, t[shared:every], new

    def slide(self, s, window, sinks, group):
        if s not in self.tab:
            return UNKNOWN, 0
        t, n, gone = self.tab[s], self.n[s], []
        for j in range(len(t)):
            tokens = range(16 * j, 16 * j + 16)
            unseen = all(x >= sinks and x < n - window for x in tokens) and tokens[-1] < n
            if unseen and tokens[-1] < n // group * group and t[j] is not None:
                gone.append(t[j])
                t[j] = None
        self._drop(gone)
        return 0, len(gone)

    def compact(self):
        used = self.blocks - len(self.free_ids)
        src = [b for b in range(used, self.blocks) if self.refs(b)]
        dst = [b for b in range(used) if not self.refs(b)]
        to = dict(zip(src, dst))
        for s, t in self.tab.items():
            self.tab[s] = [to.get(b, b) for b in t]
        self.free_ids = list(range(used, self.blocks))[::-1]
        return src, dst

    def swap_out(self, s):
        if s not in self.tab:
            return UNKNOWN, []
        t = self.tab.pop(s)
        self._drop(t)
        self.out[s] = [b is None for b in t]
        return 0, [b for b in t if b is not None]

    def swap_in(self, s):
        if s not in self.out:
            return UNKNOWN, []
        if self.out[s].count(False) > len(self.free_ids):
            return FULL, []
        self.tab[s] = [None if hole else self.free_ids.pop() for hole in self.out.pop(s)]
        return 0, [b for b in self.tab[s] if b is not None]


def same(mi, pool, model):
    assert pool.num_free() == len(model.free_ids)
    for s in range(model.seqs):
        got = mi.mi_kv_pool_seq_blocks(pool.handle, s)
        if s not in model.tab:
            assert got is None
            continue
        want = [-1 if b is None else b for b in model.tab[s]]
        assert got.tolist() == want
        bt, cl, sl = pool.batch_meta([s])
        n = model.n[s]
        assert bt[0].tolist() == want + [-1] * (model.width - len(want)) and cl[0] == n
        assert sl[0] == (want[(n - 1) // 16] * 16 + (n - 1) % 16 if n else -1)
    for b in range(model.blocks):
        assert pool.block_refs(b) == model.refs(b)


@pytest.mark.parametrize("seed", range(4))
def test_random_calls_match_the_model(mi, seed):
    r = np.random.default_rng(seed)
    blocks, seqs, width = 90, 9, 24
    pool, model = mi.Pool(blocks, seqs, width), Model(blocks, seqs, width)
    done = dict.fromkeys("alloc free shrink fork slide compact out in".split(), 0)
    for step in range(2500):
        a, b = (int(x) for x in r.integers(0, seqs, 2))
        what = r.choice(list(done), p=[0.36, 0.1, 0.1, 0.18, 0.12, 0.02, 0.06, 0.06])
        n = int(r.integers(0, 1 + max(1, model.n.get(a, 0))))
        group = int(r.choice([16, 64]))
        if what == "alloc":
            n = model.n.get(a, 0) + int(r.integers(0, 50))
            got = pool.alloc(a, n), model.alloc(a, n)
        elif what == "free":
            got = pool.free(a), model.free(a)
        elif what == "shrink":
            got = pool.shrink(a, n), model.shrink(a, n)
        elif what == "fork":
            st, src, dst = pool.fork(a, b, n, group)
            got = (st, src.tolist(), dst.tolist()), model.fork(a, b, n, group)
        elif what == "slide":
            w, k = int(r.integers(1, 200)), int(r.choice([0, 1, 16, 20, 64]))
            got = pool.slide(a, w, k, group), model.slide(a, w, k, group)
        elif what == "compact":
            st, src, dst = pool.compact()
            got = (src.tolist(), dst.tolist()), model.compact()
            assert st == 0 and not set(got[0][0]) & set(got[0][1])
        elif what == "out":
            got = pool.swap_out(a), model.swap_out(a)
        else:
            got = pool.swap_in(a), model.swap_in(a)
        assert got[0] == got[1], (step, what)
        done[what] += (got[0] if isinstance(got[0], int) else got[0][0]) in (0, [])
        if step % 40 == 0:
            same(mi, pool, model)
    same(mi, pool, model)
    assert all(done[k] > 10 for k in done if k != "compact"), done
    for s in range(seqs):
        pool.free(s)
    assert pool.num_free() == blocks and all(pool.block_refs(b) == 0 for b in range(blocks))


def test_fork_shares_whole_groups(mi):
    pool = mi.Pool(20, 6, 10)
    assert pool.alloc(0, 70) == 0  # blocks 0 .. 4
    st, src, dst = pool.fork(0, 1, 70)
    assert st == 0 and src.tolist() == [4] and dst.tolist() == [5]
    st, src, dst = pool.fork(0, 2, 70, 64)
    assert st == 0 and src.tolist() == [4] and dst.tolist() == [6]
    st, src, dst = pool.fork(0, 3, 50, 64)  # the open group whole
    assert st == 0 and src.tolist() == [0, 1, 2, 3] and dst.tolist() == [7, 8, 9, 10]
    st, src, dst = pool.fork(0, 4, 64)
    assert st == 0 and len(src) == 0
    st, src, dst = pool.fork(0, 5, 0)
    assert st == 0 and len(src) == 0 and pool.batch_meta([5])[1][0] == 0
    assert [pool.block_refs(b) for b in range(6)] == [4, 4, 4, 4, 1, 1]
    # each writes its own last block
    assert len({int(pool.batch_meta([s])[2][0]) // 16 for s in (0, 1, 2)}) == 3
    assert pool.free(0) == 0 and [pool.block_refs(b) for b in range(5)] == [3, 3, 3, 3, 0]
    assert pool.num_free() == 20 - 10


def test_fork_refusals(mi):
    pool = mi.Pool(8, 4, 8)
    assert pool.fork(0, 1, 0)[0] == UNKNOWN
    assert pool.alloc(0, 100) == 0 and pool.alloc(2, 1) == 0  # all eight blocks
    for src, dst, n in ((0, 0, 10), (0, 2, 10), (0, -1, 10), (0, 4, 10), (0, 1, 101), (0, 1, -1)):
        assert pool.fork(src, dst, n)[0] == BAD, (src, dst, n)
    for src in (-1, 4, 3):
        assert pool.fork(src, 1, 0)[0] == UNKNOWN
    for group in (0, -16, 8, 24):
        assert pool.fork(0, 1, 10, group)[0] == BAD
    assert pool.num_free() == 0 and pool.fork(0, 1, 10)[0] == FULL
    assert pool.fork(0, 1, 96)[0] == 0
    # no place for the copies
    assert pool.free(2) == 0
    assert mi.mi_kv_pool_fork(pool.handle, 0, 3, 20, 16, max_copies=0)[0] == BAD
    assert mi.mi_kv_pool_fork(pool.handle, 0, 3, 20, 16, max_copies=1)[0] == 0
    assert mi.mi_kv_pool_fork(None, 0, 3, 20)[0] == BAD
    lib, h = mi.load(), pool.handle
    buf = np.empty(8, np.int32)
    assert lib.mi_kv_pool_fork(h, 0, 2, 20, 16, None, buf.ctypes.data, 1, buf.ctypes.data) == BAD
    assert lib.mi_kv_pool_fork(h, 0, 2, 20, 16, buf.ctypes.data, buf.ctypes.data, 1, None) == BAD
    assert pool.swap_out(3)[0] == 0
    assert pool.fork(3, 2, 0)[0] == UNKNOWN and pool.fork(0, 3, 16)[0] == BAD


def test_shared_or_released_ends_are_not_shrunk_to(mi):
    pool = mi.Pool(20, 4, 12)
    assert pool.alloc(0, 100) == 0 and pool.fork(0, 1, 96)[0] == 0
    assert pool.shrink(0, 50) == BAD and pool.shrink(1, 95) == BAD
    assert pool.shrink(0, 97) == 0 and pool.shrink(0, 64) == 0  # its own block; a block's end
    assert pool.alloc(2, 150) == 0 and pool.slide(2, 20, 16) == (0, 7)
    assert mi.mi_kv_pool_seq_blocks(pool.handle, 2).tolist()[1:8] == [-1] * 7
    assert pool.shrink(2, 100) == BAD and pool.shrink(2, 112) == BAD and pool.shrink(2, 128) == BAD
    assert pool.fork(2, 3, 100)[0] == BAD and pool.fork(2, 3, 112)[0] == BAD
    assert pool.shrink(2, 16) == 0 and pool.batch_meta([2])[1][0] == 16


def test_slots_of_released_tokens(mi):
    pool = mi.Pool(20, 4, 12)
    assert pool.alloc(0, 150) == 0 and pool.slide(0, 20, 16) == (0, 7)
    assert mi.mi_kv_pool_token_slots(pool.handle, 0, 10, 4)[0] == 0
    assert mi.mi_kv_pool_token_slots(pool.handle, 0, 10, 7)[0] == BAD
    assert mi.mi_kv_pool_token_slots(pool.handle, 0, 128, 22)[0] == 0
    assert pool.slide(0, 20, 16) == (0, 0)
    assert pool.slide(0, 1, 0) == (0, 2)  # the sinks' block and one more; the last block stays
    assert pool.batch_meta([0])[2][0] >= 0


@pytest.mark.parametrize("n,window,sinks,group,kept", [
    (160, 32, 0, 16, [8, 9]), (160, 33, 0, 16, [7, 8, 9]), (161, 33, 0, 16, [8, 9, 10]), (160, 31, 4, 16, [0, 8, 9]),
    (160, 1, 0, 16, [9]), (161, 1, 0, 16, [10]), (160, 160, 0, 16, list(range(10))), (160, 400, 0, 16, list(range(10))),
    (160, 10, 500, 16, list(range(10))), (160, 10, 17, 16, [0, 1, 9]), (160, 1, 0, 64, [8, 9]), (192, 1, 0, 64, [11]),
    (191, 1, 0, 64, [8, 9, 10, 11]), (0, 1, 0, 16, []), (5, 1, 0, 16, [0])])
def test_slide_keeps_what_is_seen(mi, n, window, sinks, group, kept):
    pool = mi.Pool(40, 1, 40)
    assert pool.alloc(0, n) == 0
    st, gone = pool.slide(0, window, sinks, group)
    blocks = mi.mi_kv_pool_seq_blocks(pool.handle, 0)
    assert st == 0 and np.flatnonzero(blocks >= 0).tolist() == kept and gone == len(blocks) - len(kept)
    assert pool.num_free() == 40 - len(kept)
    assert pool.alloc(0, n + 40) == 0 and pool.free(0) == 0 and pool.num_free() == 40


def test_slide_refusals(mi):
    pool = mi.Pool(8, 2, 8)
    assert pool.slide(0, 1, 0)[0] == UNKNOWN and pool.slide(-1, 1, 0)[0] == UNKNOWN
    assert pool.alloc(0, 100) == 0
    for w, s, g in ((0, 0, 16), (-1, 0, 16), (1, -1, 16), (1, 0, 0), (1, 0, 17)):
        assert pool.slide(0, w, s, g)[0] == BAD
    assert mi.mi_kv_pool_slide(None, 0, 1, 0)[0] == BAD
    assert pool.slide(0, 1 << 30, 2 ** 31 - 1) == (0, 0)
    assert pool.swap_out(0)[0] == 0 and pool.slide(0, 1, 0)[0] == UNKNOWN


def test_compact_order_and_room(mi):
    pool = mi.Pool(12, 5, 6, [11, 0, 7, 3, 9, 1, 2, 4, 5, 6, 8, 10])
    assert pool.alloc(0, 33) == 0 and pool.alloc(1, 17) == 0  # 11 0 7 | 3 9
    assert pool.free(1) == 0 and pool.fork(0, 2, 40)[0] == BAD and pool.fork(0, 2, 32)[0] == 0
    n = np.zeros(1, np.int32)
    lib, h = mi.load(), pool.handle
    assert lib.mi_kv_pool_compact(h, None, None, 0, n.ctypes.data) == BAD and n[0] == 2
    assert mi.mi_kv_pool_seq_blocks(h, 0).tolist() == [11, 0, 7]  # unchanged
    st, src, dst = pool.compact()
    assert st == 0 and src.tolist() == [7, 11] and dst.tolist() == [1, 2]
    assert mi.mi_kv_pool_seq_blocks(h, 0).tolist() == [2, 0, 1] and mi.mi_kv_pool_seq_blocks(h, 2).tolist() == [2, 0]
    assert [pool.block_refs(b) for b in range(12)] == [2, 1, 2] + [0] * 9
    assert pool.compact()[1].tolist() == []
    assert pool.alloc(3, 20) == 0 and mi.mi_kv_pool_seq_blocks(h, 3).tolist() == [3, 4]
    assert lib.mi_kv_pool_compact(None, None, None, 0, n.ctypes.data) == BAD
    assert lib.mi_kv_pool_compact(h, None, None, 0, None) == BAD
    assert lib.mi_kv_pool_compact(h, None, None, -1, n.ctypes.data) == BAD
    assert lib.mi_kv_pool_compact(h, None, None, 3, n.ctypes.data) == BAD
    assert pool.block_refs(-1) == -1 and pool.block_refs(12) == -1 and mi.mi_kv_pool_block_refs(None, 0) == -1


def test_compact_empty_and_full(mi):
    pool = mi.Pool(4, 2, 4)
    st, src, dst = pool.compact()
    assert st == 0 and len(src) == 0
    assert pool.alloc(0, 64) == 0
    st, src, dst = pool.compact()
    assert st == 0 and len(src) == 0 and pool.num_free() == 0


def test_a_slid_sequence_that_shrinks_keeps_its_window():
    """Slid with window + k, a sequence that takes k tokens back still has all its
    window; slid with the window alone its table shows what is missing."""
    import paged_kv_decode_25_gb300 as mi
    for k, whole in ((20, True), (0, False)):
        pool = mi.Pool(32, 2, 16)
        assert pool.alloc(0, 150) == 0
        assert pool.slide(0, 40 + k, 3)[0] == 0
        assert mi.mi_kv_pool_shrink(pool.handle, 0, 130) == 0
        blocks = mi.mi_kv_pool_seq_blocks(pool.handle, 0)
        assert (blocks[(130 - 40) // 16:] >= 0).all() == whole


def test_token_slots_over_released_blocks():
    import paged_kv_decode_25_gb300 as mi
    pool = mi.Pool(32, 2, 16)
    assert pool.alloc(0, 150) == 0 and pool.slide(0, 40, 3)[0] == 0  # columns 1 .. 5 are gone
    for first, count in ((96, 54), (0, 16), (15, 1), (149, 1)):
        assert mi.mi_kv_pool_token_slots(pool.handle, 0, first, count)[0] == 0
    for first in (16, 95, 150):
        assert mi.mi_kv_pool_token_slots(pool.handle, 0, first, 0)[0] == 0
    for first, count in ((95, 55), (0, 17), (15, 2), (16, 1), (50, 60)):
        assert mi.mi_kv_pool_token_slots(pool.handle, 0, first, count)[0] == mi.MI_ERR_INVALID_ARG
