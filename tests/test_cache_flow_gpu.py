"""The cache operators together, as a serving loop uses them: prompts through
prefill, their scores from the last tokens, eviction in place with the blocks
given back to the pool, decode steps that keep scoring (the next token at its
true position), another eviction; and a shared prefix cut down once, out of
place, for all requests behind it. Every step against 64 bits over the tokens
that the step before left."""
import numpy as np
import pytest
import torch

from paged_ref import BLOCK, attention_ref, blocks_of, evict_ref, logit_slack, softmax_parts

pytestmark = pytest.mark.gpu
Hq, Hkv, D = 8, 2, 64
G, SCALE = Hq // Hkv, D ** -0.5


def _mi():
    import paged_kv_decode_25_gb300 as mi
    return mi


class Loop:
    """One layer's caches, scores and pool, with the library's calls on them."""

    def __init__(self, dev, num_blocks, max_seqs, width, seed):
        self.mi, self.dev, self.width, self.nb = _mi(), dev, width, num_blocks
        rng = np.random.default_rng(seed)
        self.pool = self.mi.Pool(num_blocks, max_seqs, width, rng.permutation(num_blocks))
        self.gen = torch.Generator().manual_seed(seed)
        shape = (num_blocks, Hkv, BLOCK, D)
        self.k = torch.full(shape, float("nan"), dtype=torch.bfloat16, device=dev)
        self.v = self.k.clone()
        self.scores = torch.full((num_blocks, Hkv, BLOCK), float("nan"), device=dev)
        _, table = self.mi.mi_rope_table(1e6, D, 4096)
        self.rope = torch.from_numpy(table).to(dev)
        self.err = torch.zeros(1, dtype=torch.int32, device=dev)

    def i32(self, x):
        return torch.as_tensor(np.ascontiguousarray(x, np.int32)).to(self.dev)

    def dims(self, B):
        return self.mi.dims(B, Hq, Hkv, D, self.nb, self.width)

    def space(self, n):
        assert n > 0
        return torch.empty(n, dtype=torch.uint8, device=self.dev)

    def normal(self, *shape):
        return torch.randn(*shape, generator=self.gen).to(torch.bfloat16).to(self.dev)

    def append(self, rows, positions, slots):
        """New q / k / v rows; returns the rotated q."""
        q, k, v = self.normal(rows, Hq, D), self.normal(rows, Hkv, D), self.normal(rows, Hkv, D)
        out = torch.empty_like(q)
        self.mi.check(self.mi.mi_paged_kv_append(self.dims(rows), q, k, v, self.i32(positions), self.i32(slots), self.rope,
                                                 4096, out, self.k, self.v, dev_err=self.err))
        return out

    def meta(self, seqs):
        return self.pool.batch_meta(seqs)

    def held(self, seq):
        """(k, v, scores) of a sequence's rows, [Hkv][n][..] fp64 on the host."""
        bt, cl, _ = self.meta([seq])
        t = torch.arange(int(cl[0]))
        blk = torch.from_numpy(bt[0]).long()[t // BLOCK]
        k, v, s = self.k.cpu(), self.v.cpu(), self.scores.cpu()
        return (k[blk, :, t % BLOCK].transpose(0, 1).double(), v[blk, :, t % BLOCK].transpose(0, 1).double(),
                s[blk, :, t % BLOCK].T.contiguous())

    def evict(self, seqs, budget, recent):
        mi = self.mi
        bt, cl, _ = self.meta(seqs)
        tables, new = self.i32(bt), torch.zeros(len(seqs), dtype=torch.int32, device=self.dev)
        d = self.dims(len(seqs))
        mi.check(mi.mi_paged_kv_evict(d, self.k, self.v, self.scores, tables, self.i32(cl),
                                      self.i32([budget] * len(seqs)), recent, tables, new,
                                      self.space(mi.mi_paged_kv_evict_workspace_bytes(d)), dev_err=self.err))
        torch.cuda.synchronize()
        for s, n in zip(seqs, new.tolist()):
            assert self.pool.shrink(s, n) == 0


def assert_close(got, ref, tol):
    assert torch.all((got.double() - ref).abs() <= tol), float(((got.double() - ref).abs() / tol.clamp(min=1e-30)).max())


def test_prompt_evict_decode_evict(cuda_device):
    loop = Loop(cuda_device, 200, 4, 40, 60)
    mi, seqs, prompts, window = loop.mi, [0, 1, 2], [300, 45, 517], 32
    total, starts, q_all = sum(prompts), np.concatenate([[0], np.cumsum(prompts)]), None
    for s, n in zip(seqs, prompts):
        assert loop.pool.alloc(s, n) == 0
    positions = np.concatenate([np.arange(n) for n in prompts])
    slots = np.concatenate([loop.pool.token_slots(s, 0, n) for s, n in zip(seqs, prompts)])
    q_all = loop.append(total, positions, slots)
    bt, cl, _ = loop.meta(seqs)
    out = torch.empty_like(q_all)
    mi.check(mi.mi_paged_prefill_attention(loop.dims(3), total, max(prompts), q_all, loop.k, loop.v, loop.i32(bt),
                                           loop.i32(cl), loop.i32(starts), SCALE, out, dev_err=loop.err))
    # the scores of the prompts, from their last tokens
    m = [min(window, n) for n in prompts]
    q_win = torch.cat([q_all[e - w:e] for e, w in zip(starts[1:], m)])
    d = loop.dims(3)
    mi.check(mi.mi_paged_prefill_scores(d, sum(m), window, q_win, loop.k, loop.i32(bt), loop.i32(cl),
                                        loop.i32(np.concatenate([[0], np.cumsum(m)])), SCALE, True, loop.scores,
                                        loop.space(mi.mi_paged_prefill_scores_workspace_bytes(d, sum(m), window)),
                                        dev_err=loop.err))
    torch.cuda.synchronize()
    first = np.concatenate([[0], np.cumsum(m)])
    for s, n in zip(seqs, prompts):
        k, _, sc = loop.held(s)
        keep = torch.arange(n) <= (n - m[s] + torch.arange(m[s]))[:, None]
        for h in range(Hkv):
            qs = [q_win[first[s]:first[s + 1], j].double().cpu() for j in range(h * G, (h + 1) * G)]
            w = sum(softmax_parts(x, k[h], SCALE, keep).sum(0) for x in qs)
            slack = max(logit_slack(x, k[h], SCALE) for x in qs)
            assert_close(sc[h], w, w * (2 * slack + 2.0 ** -18 + (n + m[s] * G) * 2.0 ** -24) + 1e-30)

    true_pos = list(prompts)
    for phase in range(2):
        before = [loop.held(s) for s in seqs]
        lens = [x[0].shape[1] for x in before]
        free = loop.pool.num_free()
        loop.evict(seqs, 100 - 30 * phase, 16)
        assert loop.pool.num_free() == free + sum(blocks_of(n) - blocks_of(min(n, 100 - 30 * phase)) for n in lens)
        for s in seqs:
            k, v, sc = loop.held(s)
            for h in range(Hkv):
                src = evict_ref(before[s][2][h].numpy(), lens[s], 100 - 30 * phase, 16)
                for have, old in zip((k, v, sc), before[s]):
                    assert torch.equal(have[h], old[h][src])
        for _ in range(5):
            old = [loop.held(s) for s in seqs]
            now = [x[0].shape[1] + 1 for x in old]
            assert loop.pool.alloc_batch(seqs, now) == 0
            bt, cl, sl = loop.meta(seqs)
            q = loop.append(3, true_pos, sl)
            true_pos = [p + 1 for p in true_pos]
            out = torch.empty_like(q)
            mi.check(mi.mi_paged_decode_attention_scored(d, q, loop.k, loop.v, loop.i32(bt), loop.i32(cl), SCALE, False,
                                                         out, loop.scores,
                                                         loop.space(mi.mi_paged_scored_workspace_bytes(d)),
                                                         dev_err=loop.err))
            torch.cuda.synchronize()
            for s in seqs:
                k, v, sc = loop.held(s)
                for h in range(Hkv):
                    qs = q[s, h * G:(h + 1) * G].double().cpu()
                    ref, tol = attention_ref(qs, k[h], v[h], SCALE)
                    assert_close(out[s, h * G:(h + 1) * G].cpu(), ref, tol)
                    w = softmax_parts(qs, k[h], SCALE).sum(0)
                    w[:-1] += old[s][2][h].double()
                    tol = w * (2 * logit_slack(qs, k[h], SCALE) + 2.0 ** -18 + (len(w) + G) * 2.0 ** -24) + 1e-30
                    assert_close(sc[h], w, tol)
    assert loop.err.item() == 0


def test_shared_prefix_cut_down(cuda_device):
    """A prefix scored and evicted out of place; the requests behind it attend
    to what is left and to their own tokens; the source stays whole."""
    loop = Loop(cuda_device, 120, 8, 40, 61)
    mi, n = loop.mi, 400
    assert loop.pool.alloc(0, n) == 0
    q_all = loop.append(n, np.arange(n), loop.pool.token_slots(0, 0, n))
    bt, cl, _ = loop.meta([0])
    d1 = loop.dims(1)
    mi.check(mi.mi_paged_prefill_scores(d1, n, n, q_all, loop.k, loop.i32(bt), loop.i32(cl), loop.i32([0, n]), SCALE, True,
                                        loop.scores, loop.space(mi.mi_paged_prefill_scores_workspace_bytes(d1, n, n)),
                                        dev_err=loop.err))
    torch.cuda.synchronize()
    whole = loop.held(0)
    keep = 101
    assert loop.pool.alloc(1, keep) == 0
    dst, _, _ = loop.meta([1])
    new = torch.zeros(1, dtype=torch.int32, device=cuda_device)
    mi.check(mi.mi_paged_kv_evict(d1, loop.k, loop.v, loop.scores, loop.i32(bt), loop.i32(cl), loop.i32([keep]), 20,
                                  loop.i32(dst), new, loop.space(mi.mi_paged_kv_evict_workspace_bytes(d1)),
                                  dev_err=loop.err))
    torch.cuda.synchronize()
    assert new.item() == keep
    for a, b in zip(loop.held(0), whole):
        assert torch.equal(a, b)
    cut = loop.held(1)
    for h in range(Hkv):
        src = evict_ref(whole[2][h].numpy(), n, keep, 20)
        for have, old in zip(cut, whole):
            assert torch.equal(have[h], old[h][src])
    # five requests behind the prefix, one without
    seqs, own = [2, 3, 4, 5, 6, 7], [0, 0, 0, 0, 0, 0]
    d = loop.dims(6)
    for step in range(4):
        own = [x + 1 for x in own]
        assert loop.pool.alloc_batch(seqs, own) == 0
        bt, cl, sl = loop.meta(seqs)
        q = loop.append(6, [n + step] * 5 + [step], sl)
        out = torch.empty_like(q)
        ptab, plen, _ = loop.meta([1])
        mi.check(mi.mi_paged_decode_attention_prefix(d, 1, loop.width, q, loop.k, loop.v, loop.i32(ptab), loop.i32(plen),
                                                     loop.i32([0, 5]), loop.i32(bt), loop.i32(cl), SCALE, out,
                                                     loop.space(mi.mi_paged_prefix_workspace_bytes(d, 1, loop.width)),
                                                     dev_err=loop.err))
        torch.cuda.synchronize()
        for i, s in enumerate(seqs):
            k, v, _ = loop.held(s)
            for h in range(Hkv):
                kk = torch.cat([cut[0][h], k[h]]) if i < 5 else k[h]
                vv = torch.cat([cut[1][h], v[h]]) if i < 5 else v[h]
                ref, tol = attention_ref(q[i, h * G:(h + 1) * G].double().cpu(), kk, vv, SCALE)
                assert_close(out[i, h * G:(h + 1) * G].cpu(), ref, tol)
    assert loop.err.item() == 0
