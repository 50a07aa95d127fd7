"""Paged batches with poisoned unused rows, and plain 64-bit forms of the
cache operators (shared-prefix attention, attention weights, eviction).

Tolerances count roundings: half a step of bf16 is 2^-8 of the value, of fp32
2^-24. `logit_slack` bounds an fp32 dot product accumulated in any order:
d products, each sum off by at most 2^-23 (tensor cores may truncate) of the
sum of magnitudes.
"""
import numpy as np
import torch

BLOCK = 16
BF16_HALF, FP32_HALF = 2.0 ** -8, 2.0 ** -24


def blocks_of(n):
    return -(-n // BLOCK)


class Batch:
    """Sequences of the given lengths in a shuffled block pool: `tables`
    [S][width] int32 (-1 past each), `k` / `v` [num_blocks][Hkv][16][d] bf16
    with NaN in every row that holds no token."""

    def __init__(self, lens, Hkv, d, seed, spare=3, width=None, fp8=False):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.Hkv, self.d = list(lens), Hkv, d
        used = sum(blocks_of(n) for n in lens)
        self.num_blocks = used + spare
        order = torch.randperm(self.num_blocks, generator=g).to(torch.int32)
        self.free = order[used:]
        self.width = max([1] + [blocks_of(n) for n in lens]) if width is None else width
        self.tables = torch.full((len(lens), self.width), -1, dtype=torch.int32)
        at = 0
        self.k = torch.full((self.num_blocks, Hkv, BLOCK, d), float("nan"), dtype=torch.bfloat16)
        self.v = self.k.clone()
        for s, n in enumerate(lens):
            nb = blocks_of(n)
            self.tables[s, :nb] = order[at:at + nb]
            at += nb
            if n:
                blk, off = self.rows(s, n)
                self.k[blk, :, off] = torch.randn(n, Hkv, d, generator=g).to(torch.bfloat16)
                self.v[blk, :, off] = torch.randn(n, Hkv, d, generator=g).to(torch.bfloat16)
        if fp8:
            self.k, self.v = self.k.to(torch.float8_e4m3fn), self.v.to(torch.float8_e4m3fn)
        self.gen = g

    def rows(self, s, n=None, tables=None):
        n = self.lens[s] if n is None else n
        t = torch.arange(n)
        return (self.tables if tables is None else tables)[s].long()[t // BLOCK], t % BLOCK

    def tokens(self, cache, s, h):
        """[n][d] in fp64."""
        blk, off = self.rows(s)
        if cache.element_size() == 1:
            return cache.view(torch.uint8)[blk, h, off].view(cache.dtype).double()
        return cache[blk, h, off].double()

    def queries(self, rows, Hq):
        return torch.randn(rows, Hq, self.d, generator=self.gen).to(torch.bfloat16)


def logit_slack(q, k, scale):
    """Largest error of scale * <q, k> in fp32, natural units."""
    if not q.numel() or not k.numel():
        return 0.0
    return float((q.abs() @ k.abs().T).max()) * abs(scale) * q.shape[-1] * 2.0 ** -23


def softmax_parts(q, k, scale, keep=None):
    """Weights [rows][n] of q [rows][d] over k [n][d] in fp64 (zero rows where nothing is kept)."""
    x = q @ k.T * scale
    if keep is not None:
        x = x.masked_fill(~keep, float("-inf"))
    if x.shape[-1] == 0:
        return x
    top = x.amax(-1, keepdim=True)
    w = torch.exp(x - torch.where(torch.isfinite(top), top, torch.zeros_like(top)))
    total = w.sum(-1, keepdim=True)
    return torch.where(total > 0, w / total.clamp(min=1e-300), torch.zeros_like(w))


def attention_ref(q, k, v, scale):
    """(out, tolerance) of bf16 decode attention of q [G][d] over k, v [n][d].

    The weights enter the second product rounded to bf16 (half a step of each
    weight, so of sum w|v|), the sum that normalises them may hold the rounded
    ones (another half step of |out|), the output is rounded once more; the
    logits' error multiplies every weight by at most e^(2 slack)."""
    w = softmax_parts(q, k, scale)
    if k.shape[0] == 0:
        z = torch.zeros_like(q)
        return z, z
    out, mag = w @ v, w @ v.abs()
    slack = 2 * logit_slack(q, k, scale) + 64 * FP32_HALF
    return out, (BF16_HALF * (out.abs() + mag + out.abs()) + slack * 2 * mag) * 1.01 + 1e-30


def weight_tolerance(w_sum, terms, slack, before=None):
    """Of a sum of fp32 weights: each off by e^(2 slack) and the roundings of
    an exponential, a logarithm and a sum of `terms` values (fp32 each)."""
    tol = w_sum * (2 * slack + 2.0 ** -20 + terms * FP32_HALF) * 1.01 + 1e-30
    return tol if before is None else tol + 2 * FP32_HALF * before.abs()


def evict_ref(scores, n, budget, recent):
    """Source indices of the kept tokens of one (request, head), in order."""
    k = min(n, max(budget, 0))
    if k == n:
        return np.arange(n)
    r = min(recent, k)
    s = np.where(np.isnan(scores), -np.inf, scores.astype(np.float64))
    nan = np.isnan(scores)
    old = n - r
    # heaviest first, NaN after everything, equal scores by index
    order = np.lexsort((np.arange(old), -s[:old], nan[:old]))
    return np.concatenate([np.sort(order[:k - r]), np.arange(old, n)]).astype(np.int64)
