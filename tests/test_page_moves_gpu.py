"""mi_kv_copy_planes: every plane's rows, bit for bit, and nothing else."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def _mi():
    import paged_kv_decode_25_gb300 as mi
    return mi


def fill(rows, nbytes, g):
    return torch.randint(0, 256, (rows, nbytes), generator=g, dtype=torch.uint8)


def move(dev, planes, src, dst, err=None):
    mi = _mi()
    mi.check(mi.mi_kv_copy_planes(mi.kv_planes(planes), torch.tensor(src, dtype=torch.int32, device=dev),
                                  torch.tensor(dst, dtype=torch.int32, device=dev), len(src), err))
    torch.cuda.synchronize()


# rows of a bf16 and an e4m3 cache, scores, maxima, and lengths around an item's
SIZES = [4, 12, 32, 512, 1000, 4096, 16384, 32764, 32768, 32772, 65536, 100000]


@pytest.mark.parametrize("n", [1, 3, 70])
@pytest.mark.parametrize("nbytes", SIZES)
def test_one_plane(cuda_device, nbytes, n):
    g = torch.Generator().manual_seed(nbytes + n)
    x = fill(2 * n + 3, nbytes, g)
    ids = torch.randperm(2 * n + 3, generator=g)
    want = x.clone()
    want[ids[n:2 * n]] = x[ids[:n]]
    y = x.to(cuda_device)
    move(cuda_device, [y], ids[:n].tolist(), ids[n:2 * n].tolist())
    assert torch.equal(y.cpu(), want)


@pytest.mark.parametrize("planes", [1, 8, 143, 144, 145, 300])
def test_many_planes(cuda_device, planes):
    """Planes of different row lengths, more than one launch holds."""
    g = torch.Generator().manual_seed(planes)
    xs = [fill(40, (4, 512, 2048, 40000)[i % 4], g) for i in range(planes)]
    src, dst = [1, 7, 7, 39, 0], [30, 31, 32, 2, 38]
    wants = []
    for x in xs:
        w = x.clone()
        w[dst] = x[src]
        wants.append(w)
    ys = [x.to(cuda_device) for x in xs]
    move(cuda_device, ys, src, dst)
    for y, w in zip(ys, wants):
        assert torch.equal(y.cpu(), w)


def test_bases_off_16_bytes(cuda_device):
    g = torch.Generator().manual_seed(5)
    whole = fill(1, 4 + 20 * 64, g).to(cuda_device)
    x = whole[0, 4:].reshape(20, 64)
    want = x.cpu().clone()
    want[[3, 4]] = want[[10, 11]]
    move(cuda_device, [x], [10, 11], [3, 4])
    assert torch.equal(x.cpu(), want)


def test_bad_ids_skip_their_rows(cuda_device):
    mi = _mi()
    g = torch.Generator().manual_seed(6)
    for nbytes in (32, 32768, 70000):
        x, small = fill(10, nbytes, g), fill(8, 16, g)
        want, want_small = x.clone(), small.clone()
        want[[1, 2, 3]] = x[[5, 9, 6]]
        want_small[[1, 3]] = small[[5, 6]]  # row 9 lies behind this plane
        err = torch.zeros(1, dtype=torch.int32, device=cuda_device)
        y, ys = x.to(cuda_device), small.to(cuda_device)
        move(cuda_device, [y, ys], [5, 9, 6, -1, 4, 10, 4], [1, 2, 3, 0, -1, 0, 10], err)
        assert err.item() == mi.MI_DEVERR_BAD_BLOCK
        assert torch.equal(y.cpu(), want) and torch.equal(ys.cpu(), want_small)


def test_offsets_past_32_bits(cuda_device):
    """A plane of more than 4 GB."""
    rows, nbytes = 70000, 65536
    x = torch.zeros(rows, nbytes, dtype=torch.uint8, device=cuda_device)
    x[5] = 3
    x[rows - 1] = 7
    x[40000] = 9
    move(cuda_device, [x], [5, rows - 1, 40000], [rows - 2, 6, 32768])
    for i, v in ((5, 3), (rows - 2, 3), (6, 7), (32768, 9), (rows - 1, 7), (rows - 3, 0), (4, 0), (7, 0)):
        assert bool(torch.all(x[i] == v)), i


def test_compaction_and_forks_of_a_pool(cuda_device):
    """What every sequence holds stays what it was while a pool forks, slides
    and compacts, in every layer."""
    mi = _mi()
    g = torch.Generator().manual_seed(9)
    import numpy as np
    r = np.random.default_rng(9)
    blocks, seqs, layers, Hkv, d = 60, 8, 3, 2, 64
    pool = mi.Pool(blocks, seqs, 20)
    caches = [torch.zeros(blocks, Hkv, 16, d, dtype=torch.bfloat16, device=cuda_device) for _ in range(2 * layers)]
    planes = mi.kv_planes(caches)
    held = {}  # sequence: list of [planes] token values, None where given back

    def ids(x):
        return torch.from_numpy(np.ascontiguousarray(x, np.int32)).to(cuda_device)

    def move_ids(src, dst):
        mi.check(mi.mi_kv_copy_planes(planes, ids(src), ids(dst), len(src)))

    for step in range(300):
        a, b = (int(x) for x in r.integers(0, seqs, 2))
        what = r.choice(["grow", "free", "fork", "slide", "compact"], p=[0.45, 0.12, 0.25, 0.12, 0.06])
        if what == "grow":
            have = held.get(a, [])
            n = len(have) + int(r.integers(1, 30))
            if pool.alloc(a, n) == 0:
                new = torch.randn(n - len(have), 2 * layers, Hkv, d, generator=g).to(torch.bfloat16)
                slots = torch.from_numpy(pool.token_slots(a, len(have), n - len(have))).long().to(cuda_device)
                for i, c in enumerate(caches):
                    c[slots // 16, :, slots % 16] = new[:, i].to(cuda_device)
                held[a] = have + list(new)
        elif what == "free":
            if pool.free(a) == 0:
                held.pop(a)
        elif what == "fork" and a in held:
            n = int(r.integers(0, len(held[a]) + 1))
            st, src, dst = pool.fork(a, b, n)
            if st == 0:
                move_ids(src, dst)
                held[b] = list(held[a][:n])
        elif what == "slide" and a in held:
            st, gone = pool.slide(a, 20, 4)
            table = mi.mi_kv_pool_seq_blocks(pool.handle, a)
            for t in range(len(held[a])):
                if table[t // 16] < 0:
                    assert 4 <= t < len(held[a]) - 20
                    held[a][t] = None
        elif what == "compact":
            st, src, dst = pool.compact()
            move_ids(src, dst)
        if step % 30 == 29:
            torch.cuda.synchronize()
            host = [c.cpu() for c in caches]
            for s, tokens in held.items():
                table = mi.mi_kv_pool_seq_blocks(pool.handle, s)
                for t, v in enumerate(tokens):
                    if v is not None:
                        for i in range(2 * layers):
                            assert torch.equal(host[i][table[t // 16], :, t % 16], v[i]), (step, s, t)
    assert len(held) > 2


def test_graph(cuda_device):
    mi = _mi()
    g = torch.Generator().manual_seed(10)
    x = fill(50, 8192, g)
    y = x.to(cuda_device)
    src, dst = (torch.tensor(v, dtype=torch.int32, device=cuda_device) for v in ([1, 2, 3], [10, 11, 12]))
    planes = mi.kv_planes([y])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mi.check(mi.mi_kv_copy_planes(planes, src, dst, 3))
    for _ in range(3):
        y.copy_(x)
        src.copy_(torch.tensor([4, 5, 6], dtype=torch.int32))  # the lists are read when the graph runs
        graph.replay()
        want = x.clone()
        want[[10, 11, 12]] = x[[4, 5, 6]]
        assert torch.equal(y.cpu(), want)
