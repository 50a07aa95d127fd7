"""Forks of slid sequences: which columns of their windows are there (CPU)."""
import pytest


@pytest.fixture(scope="module")
def mi():
    import paged_kv_decode_25_gb300 as m
    from paged_kv_decode_25_gb300 import build
    build.build()
    return m


def window_columns(mi, pool, seq, n, window):
    """The blocks that the newest of n tokens sees without sinks."""
    return mi.mi_kv_pool_seq_blocks(pool.handle, seq)[max(0, n - window) // 16:]


@pytest.mark.parametrize("back", [0, 1, 16, 90, 400])
@pytest.mark.parametrize("sinks", [0, 20])
def test_slid_with_the_tokens_that_forks_go_back(mi, back, sinks):
    """A fork `back` tokens behind a source slid with window + back has its whole window."""
    pool = mi.Pool(100, 3, 82)
    assert pool.alloc(0, 1000) == 0
    st, gone = pool.slide(0, 100 + back, sinks)
    assert st == 0 and gone > 0
    assert pool.fork(0, 1, 1000 - back)[0] == 0
    assert (window_columns(mi, pool, 1, 1000 - back, 100) >= 0).all()
    # the source's later tokens push its window on; the fork keeps its own blocks
    assert pool.alloc(0, 1300) == 0 and pool.slide(0, 100, sinks)[0] == 0
    assert (window_columns(mi, pool, 1, 1000 - back, 100) >= 0).all()
    assert pool.free(0) == 0 and pool.free(1) == 0 and pool.num_free() == 100


def test_a_fork_further_back_shows_what_is_missing(mi):
    """Slid with the window alone: the fork is made, and its table says which blocks
    attention will not find (columns of -1, which it reports as bad blocks)."""
    pool = mi.Pool(100, 3, 82)
    assert pool.alloc(0, 1000) == 0 and pool.slide(0, 100, 0) == (0, 56)  # tokens below 896
    st, src, dst = pool.fork(0, 1, 910)
    assert st == 0 and len(src) == 1
    assert window_columns(mi, pool, 1, 910, 100).tolist()[:-1] == [-1] * 6  # tokens 800 .. 895
    assert window_columns(mi, pool, 0, 1000, 100).min() >= 0
    assert pool.fork(0, 2, 896)[0] == mi.MI_ERR_INVALID_ARG  # its last block is gone
