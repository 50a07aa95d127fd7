"""The calls for layers with norms and windows as a serving loop uses them: prompts
and chunks appended with their norms, sliding prefill, forked sequences, decode
steps, pages given back and moved together, over bf16 and e4m3 caches (and an
INT8 one by itself). Every layer's outputs against 64 bits over what the caches
were given."""
import numpy as np
import pytest
import torch

from paged_ref import attention_ref
from test_sliding_gpu import int8_slack

pytestmark = pytest.mark.gpu
EPS, MAX_POS, LAYERS = 1e-6, 4096, 2


def _mi():
    import paged_kv_decode_25_gb300 as mi
    return mi


class Loop:
    """Two layers' caches, one pool, and for every sequence and layer what its
    tokens' K and V rows held when they were appended."""

    def __init__(self, dev, kind, Hq, Hkv, d, window, sinks, seed):
        self.mi, self.dev, self.kind = _mi(), dev, kind
        self.Hq, self.Hkv, self.d, self.window, self.sinks = Hq, Hkv, d, window, sinks
        self.blocks, self.width, self.seqs = 60, 30, 6
        self.pool = self.mi.Pool(self.blocks, self.seqs, self.width, np.random.default_rng(seed).permutation(self.blocks))
        self.g = torch.Generator().manual_seed(seed)
        dt = {"bf16": torch.bfloat16, "fp8": torch.float8_e4m3fn}[kind]
        self.k, self.v = ([torch.full((self.blocks, Hkv, 16, d), float("nan"), device=dev).to(dt) for _ in range(LAYERS)]
                          for _ in range(2))
        self.planes = self.mi.kv_planes(self.k + self.v)
        self.scales = [(0.02 + 0.02 * torch.rand(Hkv, generator=self.g)) for _ in range(2)]
        a = torch.arange(MAX_POS, dtype=torch.float64)[:, None] * 1e4 ** (-2 * torch.arange(d // 2, dtype=torch.float64) / d)
        self.rope = torch.stack([torch.cos(a), torch.sin(a)], -1).float().to(dev)
        self.weights = [[(1 + 0.2 * torch.randn(d, generator=self.g)).to(torch.bfloat16).to(dev) for _ in range(2)]
                        for _ in range(LAYERS)]
        self.held = {}  # sequence: [layer] -> list of (k, v) rows [Hkv][d] in 64 bits
        self.err = torch.zeros(1, dtype=torch.int32, device=dev)
        n = max(self.mi.mi_paged_sliding_workspace_bytes(self.dims(B), window, sinks) for B in range(1, self.seqs + 1))
        self.space = torch.empty(n, dtype=torch.uint8, device=dev)

    def dims(self, B):
        return self.mi.dims(B, self.Hq, self.Hkv, self.d, self.blocks, self.width)

    def i32(self, x):
        return torch.from_numpy(np.ascontiguousarray(x, np.int32)).to(self.dev)

    def append(self, seqs, news):
        """Random new tokens of `seqs` into every layer; their rotated queries."""
        mi, dev = self.mi, self.dev
        pos, slot = [], []
        for s, m in zip(seqs, news):
            n = len(self.held.get(s, [[]])[0])
            assert self.pool.alloc(s, n + m) == 0
            self.held.setdefault(s, [[] for _ in range(LAYERS)])
            pos += range(n, n + m)
            slot += self.pool.token_slots(s, n, m).tolist()
        T, queries = len(pos), []
        pos_d, slot_d = self.i32(pos), self.i32(slot)
        for layer in range(LAYERS):
            H = self.Hq + 2 * self.Hkv
            x = torch.randn(T, H * self.d, generator=self.g).to(torch.bfloat16).to(dev)
            q, k, v = x.split([self.Hq * self.d, self.Hkv * self.d, self.Hkv * self.d], 1)
            out = torch.empty(T, self.Hq, self.d, dtype=torch.bfloat16, device=dev)
            args = (self.dims(T), q, k, v, *self.weights[layer], EPS, pos_d, slot_d, self.rope, MAX_POS, out,
                    self.k[layer], self.v[layer])
            if self.kind == "fp8":
                mi.check(mi.mi_paged_kv_append_norm_fp8(*args, *(s.to(dev) for s in self.scales), dev_err=self.err))
            else:
                mi.check(mi.mi_paged_kv_append_norm(*args, dev_err=self.err))
            queries.append(out)
            rows = []
            for c, f in ((self.k[layer], self.scales[0]), (self.v[layer], self.scales[1])):
                got = c.float()[slot_d.long() // 16, :, slot_d.long() % 16].cpu().double()
                rows.append(got * f.double()[:, None] if self.kind == "fp8" else got)
            at = 0
            for s, m in zip(seqs, news):
                self.held[s][layer] += [(rows[0][at + i], rows[1][at + i]) for i in range(m)]
                at += m
        return queries

    def check(self, seqs, news, layer, q, out):
        G, at = self.Hq // self.Hkv, 0
        q, out = q.cpu(), out.cpu()
        for s, m in zip(seqs, news):
            n = len(self.held[s][layer])
            for i in range(m):
                p = n - m + i
                t = [x for x in range(p + 1) if x < self.sinks or x > p - self.window]
                k, v = (torch.stack([self.held[s][layer][x][j] for x in t]) for j in (0, 1))
                for h in range(self.Hkv):
                    rows = slice(h * G, h * G + G)
                    ref, tol = attention_ref(q[at + i, rows].double(), k[:, h], v[:, h], self.d ** -0.5)
                    assert torch.all((out[at + i, rows].double() - ref).abs() <= tol), (s, i, h)
            at += m

    def prefill(self, seqs, news):
        for layer, q in enumerate(self.append(seqs, news)):
            bt, cl, _ = self.pool.batch_meta(seqs)
            out = torch.empty_like(q)
            self.mi.check(self.mi.mi_paged_prefill_attention_sliding(
                self.dims(len(seqs)), sum(news), max(news), q, self.k[layer], self.v[layer], self.i32(bt), self.i32(cl),
                self.i32(np.concatenate([[0], np.cumsum(news)])), self.window, self.sinks, self.d ** -0.5, out, self.err))
            self.check(seqs, news, layer, q, out)

    def decode(self, seqs):
        for layer, q in enumerate(self.append(seqs, [1] * len(seqs))):
            bt, cl, _ = self.pool.batch_meta(seqs)
            out = torch.empty_like(q)
            args = (self.i32(bt), self.i32(cl), self.window, self.sinks, self.d ** -0.5, out, self.space)
            if self.kind == "fp8":
                self.mi.check(self.mi.mi_paged_decode_attention_sliding_fp8(
                    self.dims(len(seqs)), q, self.k[layer], self.v[layer], *(s.to(self.dev) for s in self.scales), *args,
                    dev_err=self.err))
            else:
                self.mi.check(self.mi.mi_paged_decode_attention_sliding(self.dims(len(seqs)), q, self.k[layer],
                                                                        self.v[layer], *args, dev_err=self.err))
            self.check(seqs, [1] * len(seqs), layer, q, out)

    def move(self, src, dst):
        self.mi.check(self.mi.mi_kv_copy_planes(self.planes, self.i32(src), self.i32(dst), len(src), self.err))

    def fork(self, a, b):
        n = len(self.held[a][0])
        st, src, dst = self.pool.fork(a, b, n)
        assert st == 0
        self.move(src, dst)
        self.held[b] = [list(x) for x in self.held[a]]

    def slide(self, seqs):
        for s in seqs:
            assert self.pool.slide(s, self.window, self.sinks)[0] == 0

    def compact(self):
        st, src, dst = self.pool.compact()
        assert st == 0
        self.move(src, dst)
        return len(src)


@pytest.mark.parametrize("kind,Hq,Hkv,d", [("bf16", 8, 2, 64), ("bf16", 7, 1, 128), ("fp8", 8, 2, 64)])
def test_serving_loop(cuda_device, kind, Hq, Hkv, d):
    loop = Loop(cuda_device, kind, Hq, Hkv, d, window=40, sinks=3, seed=7)
    if kind == "bf16":
        loop.prefill([0, 1], [70, 33])
        loop.prefill([1, 2], [50, 5])          # a chunk behind a prompt, and a new one
    else:                                      # prefill attention takes bf16 caches
        loop.append([0, 1, 2], [70, 83, 5])
    loop.fork(0, 3)
    loop.slide([0, 1, 2, 3])
    free = loop.pool.num_free()
    for _ in range(3):
        loop.decode([0, 1, 2, 3])
    assert loop.pool.free(1) == 0
    del loop.held[1]
    assert loop.compact() > 0
    loop.decode([3, 0, 2])
    loop.fork(3, 1)
    for _ in range(14):
        loop.decode([0, 1, 2, 3])
    loop.slide([0, 1, 2, 3])
    loop.compact()
    loop.decode([2, 1, 3, 0])
    assert loop.pool.num_free() >= free - 2
    torch.cuda.synchronize()
    assert loop.err.item() == 0


def test_int8_cache_slides_and_forks(cuda_device):
    """INT8 appends quantise a sequence's open group again: forks copy it, slides keep
    it, and a fork's appends leave the other sequence's codes as they were."""
    mi, dev = _mi(), cuda_device
    Hq, Hkv, d, window, sinks, blocks, width = 4, 2, 64, 30, 3, 40, 20
    g = torch.Generator().manual_seed(3)
    pool = mi.Pool(blocks, 4, width)
    kc, vc = (torch.zeros(blocks, Hkv, 16, d, dtype=torch.int8, device=dev) for _ in range(2))
    ka, va = (torch.zeros(blocks, Hkv, device=dev) for _ in range(2))
    ko, vo = (torch.zeros(4, Hkv, 64, d, dtype=torch.bfloat16, device=dev) for _ in range(2))
    st, table = mi.mi_rope_table(1e4, d, 500)
    mi.check(st)
    rope = torch.from_numpy(table).to(dev)
    err = torch.zeros(1, dtype=torch.int32, device=dev)

    def i32(x):
        return torch.from_numpy(np.ascontiguousarray(x, np.int32)).to(dev)

    def step(seqs, news):
        T = sum(news)
        q, k, v = (torch.randn(T, h, d, generator=g).to(torch.bfloat16).to(dev) for h in (Hq, Hkv, Hkv))
        for s, m in zip(seqs, news):
            n = pool.batch_meta([s])[1][0] if mi.mi_kv_pool_seq_blocks(pool.handle, s) is not None else 0
            assert pool.alloc(s, int(n) + m) == 0
        bt, cl, _ = pool.batch_meta(seqs)
        out = torch.empty_like(q)
        dims = mi.dims(len(seqs), Hq, Hkv, d, blocks, width)
        mi.check(mi.mi_paged_kv_append_int8_tokens(dims, T, q, k, v, rope, 500, i32(bt), i32(cl),
                                                   i32(np.concatenate([[0], np.cumsum(news)])), i32(seqs), out, kc, vc, ka, va,
                                                   ko, vo, err))
        return out, bt, cl

    def attend(seqs, q, bt, cl):
        dims = mi.dims(len(seqs), Hq, Hkv, d, blocks, width)
        ws = torch.empty(mi.mi_paged_sliding_workspace_bytes(dims, window, sinks), dtype=torch.uint8, device=dev)
        out = torch.empty_like(q)
        mi.check(mi.mi_paged_decode_attention_sliding_int8(dims, q, kc, vc, ka, va, i32(bt), i32(cl), window, sinks,
                                                           d ** -0.5, out, ws, dev_err=err))
        for i, s in enumerate(seqs):
            n = int(cl[i])
            t = torch.tensor([x for x in range(n) if x < sinks or x >= n - window])
            blk, off = torch.from_numpy(bt[i]).long()[t // 16].to(dev), (t % 16).to(dev)
            for h in range(Hkv):
                k, v = (c[blk, h, off].double().cpu() * a[blk, h].double().cpu()[:, None] / 127 for c, a in ((kc, ka), (vc, va)))
                ref, tol = attention_ref(q[i, 2 * h:2 * h + 2].double().cpu(), k, v, d ** -0.5)
                # (the codes' bias of 1152 leaves its rounding: see test_sliding_gpu)
                assert torch.all((out[i, 2 * h:2 * h + 2].cpu().double() - ref).abs() <= tol + 2e-3)

    step([0], [89])
    before = [x.clone() for x in (kc, vc, ka, va)]
    st, src, dst = pool.fork(0, 1, 89, 64)
    assert st == 0 and len(src) == 2  # the open group: tokens 64 .. 88
    mi.check(mi.mi_kv_copy_planes(mi.kv_planes([kc, vc, ka, va]), i32(src), i32(dst), 2))
    mi.check(mi.mi_kv_copy_planes(mi.kv_planes([ko, vo]), i32([0]), i32([1]), 1))
    for s in (0, 1):
        assert pool.slide(s, window, sinks, 64)[0] == 0
        assert (mi.mi_kv_pool_seq_blocks(pool.handle, s) >= 0).tolist() == [True, False, False, True, True, True]
    q, bt, cl = step([1], [5])  # the fork alone goes on
    attend([1], q[4:], bt, cl)
    own = mi.mi_kv_pool_seq_blocks(pool.handle, 0)
    for x, y in zip((kc, vc, ka, va), before):
        for b in own[own >= 0]:
            assert torch.equal(x[int(b)], y[int(b)])
    for _ in range(45):  # past the group's end
        q, bt, cl = step([0, 1], [1, 1])
    attend([0, 1], q, bt, cl)
    torch.cuda.synchronize()
    assert err.item() == 0
