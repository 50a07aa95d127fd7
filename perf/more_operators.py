"""Normed appends, sliding windows and page moves of a paged decode: cases, plain forms, exact values.

Four operators of a serving loop whose layers norm their queries and keys and
attend to a window:

  norm   append of new tokens with the RMS norm of each query and key head, the
         rotation and the scatter into the paged cache in one pass
  slide  decode attention that sees a sequence's first tokens (sinks) and its
         newest ones (the window), over bf16, e4m3 and INT8 caches
  chunk  the same for many new tokens per request (prompts, chunks of prompts)
  pages  one list of pages moved in every layer's cache (forks, compaction)

`own` chooses between the plain form (torch operations in fp32) and the
library's calls.
"""
import math
import random

import numpy as np
import torch

own = False

BLOCK, GROUP = 16, 64
NEG = float("-inf")
EPS, THETA, MAX_POS = 1e-6, 1e6, 65536
SHAPES = ((32, 8, 128), (16, 8, 128), (28, 4, 128), (4, 2, 64), (8, 8, 64), (8, 1, 128))  # Hq, Hkv, head_dim
BYTES = {"bf16": 2, "fp8": 1, "int8": 1}  # of a cached element


# ------------------------------------------------------------------ cases --

def listed():
    return [
        # a decode step's new tokens, one per request: latency
        dict(name="norm_step", op="norm", Hq=32, Hkv=8, d=128, T=64, seqs=64, kind="bf16", fused=True, lens=1),
        # the new tokens of a prefill step, as its projection left them (q, k and v in one row)
        dict(name="norm_prompts", op="norm", Hq=32, Hkv=8, d=128, T=12821, seqs=16, kind="bf16", fused=True, lens=2),
        # a prompt into an e4m3 cache, q, k and v apart; seven query heads per KV head
        dict(name="norm_fp8", op="norm", Hq=28, Hkv=4, d=128, T=5000, seqs=3, kind="fp8", fused=False, lens=3),
        # one long chat behind a short window: the latency of the smallest call
        dict(name="slide_single", op="slide", B=1, Hq=32, Hkv=8, d=128, kind="bf16", window=1024, sinks=4, lo=20000,
             hi=20000, held=False, lens=4),
        # a serving batch, some contexts still shorter than the window, no page given back yet
        dict(name="slide_batch", op="slide", B=64, Hq=32, Hkv=8, d=128, kind="bf16", window=1024, sinks=4, lo=512,
             hi=8192, held=True, lens=5),
        # long contexts in an e4m3 cache that keeps the pages in sight only
        dict(name="slide_fp8_long", op="slide", B=128, Hq=28, Hkv=4, d=128, kind="fp8", window=4096, sinks=64, lo=2000,
             hi=60000, held=False, lens=6),
        # many short windows without sinks in an INT8 cache
        dict(name="slide_int8_short", op="slide", B=256, Hq=16, Hkv=8, d=128, kind="int8", window=128, sinks=0, lo=50,
             hi=2000, held=True, lens=7),
        # one short prompt
        dict(name="chunk_one", op="chunk", B=1, Hq=32, Hkv=8, d=128, window=256, sinks=4, q_lo=0, q_hi=0, lo=700, hi=700,
             lens=8),
        # a chunked-prefill batch: 512 new tokens each behind what was there
        dict(name="chunk_batch", op="chunk", B=16, Hq=32, Hkv=8, d=128, window=1024, sinks=4, q_lo=512, q_hi=512,
             lo=1024, hi=8192, lens=9),
        # whole prompts several windows long
        dict(name="chunk_prompts", op="chunk", B=2, Hq=28, Hkv=4, d=128, window=4096, sinks=0, q_lo=0, q_hi=0, lo=12000,
             hi=16000, lens=10),
        # eight forked sequences get their last page of 36 layers
        dict(name="pages_fork", op="pages", Hkv=8, d=128, kind="bf16", layers=36, blocks=64, moves=8, lens=11),
        # a cache moved together after many frees
        dict(name="pages_compact", op="pages", Hkv=8, d=128, kind="bf16", layers=4, blocks=4000, moves=1300, lens=12),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _cost(case):
    w = work(case)
    return max(w["bytes"], w["flops"] / 50)


def draw(rng):
    most = {}
    for c in listed():
        most[c["op"]] = max(most.get(c["op"], 0), _cost(c))
    while True:
        op = rng.choice(("norm", "slide", "slide", "chunk", "pages"))
        Hq, Hkv, d = rng.choice(SHAPES)
        c = dict(op=op, Hq=Hq, Hkv=Hkv, d=d, lens=rng.randrange(1 << 30))
        if op == "norm":
            T = _log(rng, 1, 12821)
            c.update(T=T, seqs=rng.choice((T, _log(rng, 1, min(T, 64)))), kind=rng.choice(("bf16", "fp8")),
                     fused=rng.random() < 0.5)
        elif op == "slide":
            a, b = _log(rng, 1, 60000), _log(rng, 1, 60000)
            c.update(B=_log(rng, 1, 256), kind=rng.choice(("bf16", "fp8", "int8")), window=_log(rng, 1, 8192),
                     sinks=rng.choice((0, 1, 4, 17, 64, 200)), lo=min(a, b), hi=max(a, b), held=rng.random() < 0.3)
        elif op == "chunk":
            a, b = _log(rng, 20, 16000), _log(rng, 20, 16000)
            m = 0 if rng.random() < 0.4 else _log(rng, 1, 1024)
            c.update(B=_log(rng, 1, 16), window=_log(rng, 1, 8192), sinks=rng.choice((0, 1, 4, 17, 64, 200)), q_lo=m,
                     q_hi=m + m // 2, lo=min(a, b), hi=max(a, b))
        else:
            blocks = _log(rng, 8, 8000)
            c.update(kind=rng.choice(("bf16", "int8")), layers=_log(rng, 1, 40), blocks=blocks,
                     moves=_log(rng, 1, blocks // 2))
            del c["Hq"]
        big = op == "slide" and c["held"] and sum(_lengths(c)) * Hkv * d > 5e8
        big |= op == "pages" and c["blocks"] * c["layers"] * Hkv * d > 4e6
        if not big and _cost(c) <= most[op]:
            return c


# ---------------------------------------------------------------- lengths --

def _lengths(case):
    """Tokens each request holds (log-uniform over the case's range)."""
    r = random.Random(case["lens"])
    lo, hi = case["lo"], case["hi"]
    return [min(hi, max(lo, int(math.exp(r.uniform(math.log(lo + 1), math.log(hi + 2)))) - 1)) for _ in range(case["B"])]


def _queries(case):
    """New tokens per request (`q_lo` 0: the whole prompt)."""
    r = random.Random(case["lens"] + 2)
    return [min(x, r.randint(case["q_lo"], case["q_hi"])) if case["q_lo"] else x for x in _lengths(case)]


def _seen(n, case):
    """Tokens that the newest of n tokens sees."""
    return min(n, case["window"]) + min(case["sinks"], max(0, n - case["window"]))


def _pairs(case):
    """(query token, key) pairs of the new tokens."""
    total = 0
    for m, n in zip(_queries(case), _lengths(case)):
        x = np.arange(n - m + 1, n + 1)
        total += int((np.minimum(x, case["window"]) + np.minimum(case["sinks"], np.maximum(0, x - case["window"]))).sum())
    return total


def _reach(m, n, case):
    """Tokens that any of the last m of n tokens sees."""
    return min(n, m + case["window"] - 1) + min(case["sinks"], max(0, n - m - case["window"] + 1))


def _planes(case):
    """(bytes of a page's row) of every plane: K and V of each layer, and an INT8 cache's maxima."""
    row = case["Hkv"] * BLOCK * case["d"] * BYTES[case["kind"]]
    return [row, row] * case["layers"] + ([4 * case["Hkv"]] * 2 * case["layers"] if case["kind"] == "int8" else [])


def work(case):
    Hkv, d = case["Hkv"], case["d"]
    if case["op"] == "pages":
        return dict(bytes=2 * case["moves"] * sum(_planes(case)) + 8 * case["moves"], flops=0)
    Hq = case["Hq"]
    e = BYTES[case.get("kind", "bf16")]
    if case["op"] == "norm":
        T = case["T"]
        return dict(bytes=T * (2 * (2 * Hq + 2 * Hkv) * d + 2 * e * Hkv * d + 8) + min(T, MAX_POS) * d * 4,
                    flops=T * (Hq + Hkv) * d * 8)
    if case["op"] == "slide":
        seen = sum(_seen(n, case) for n in _lengths(case))
        return dict(bytes=2 * e * d * Hkv * seen + 2 * 2 * case["B"] * Hq * d, flops=4 * d * Hq * seen)
    m = _queries(case)
    reach = sum(_reach(a, n, case) for a, n in zip(m, _lengths(case)))
    return dict(bytes=2 * 2 * d * Hkv * reach + 2 * 2 * d * Hq * sum(m), flops=4 * d * Hq * _pairs(case))


# ----------------------------------------------------------------- inputs --

def _i32(x):
    return torch.as_tensor(np.asarray(x, np.int32)).to("cuda")


def _i64(x):
    return torch.as_tensor(np.asarray(x, np.int64)).to("cuda")


def _tables(n, order, hide=None):
    """Block tables [B][width] over `order`; `hide(b, j)`: columns whose pages were given back."""
    width = max([-(-x // BLOCK) for x in n] + [1])
    t = np.full((len(n), width), -1, np.int32)
    at = 0
    for b, x in enumerate(n):
        cols = np.arange(-(-x // BLOCK))
        if hide is not None:
            cols = cols[~hide(b, cols)]
        t[b, cols] = order[at:at + len(cols)]
        at += len(cols)
    return t, at


def prepare(case, seed):
    return {"norm": _prepare_norm, "slide": _prepare_attention, "chunk": _prepare_attention, "pages": _prepare_pages}[
        case["op"]](case, seed)


def _prepare_norm(case, seed):
    dev = "cuda"
    Hq, Hkv, d, T, seqs = case["Hq"], case["Hkv"], case["d"], case["T"], case["seqs"]
    g = torch.Generator(dev).manual_seed(seed)
    rng = np.random.default_rng(seed)
    shape = random.Random(case["lens"])
    # T new tokens of `seqs` sequences, each behind what it holds already
    cuts = sorted(shape.sample(range(1, T), seqs - 1)) if seqs > 1 else []
    m = np.diff([0] + cuts + [T])
    first = np.array([_log(shape, 1, MAX_POS - int(x)) - 1 if shape.random() < 0.7 else 0 for x in m])
    pages = [(f + x - 1) // BLOCK - f // BLOCK + 1 for f, x in zip(first, m)]
    num_blocks = int(sum(pages)) + 3
    order = rng.permutation(num_blocks)
    pos = np.concatenate([np.arange(f, f + x) for f, x in zip(first, m)])
    base = np.repeat(np.concatenate([[0], np.cumsum(pages)[:-1]]) - first // BLOCK, m)
    slot = order[base + pos // BLOCK] * BLOCK + pos % BLOCK
    s = dict(case=case, num_blocks=num_blocks, pos=_i32(pos), slot=_i32(slot))
    # heads of very different magnitudes, as projections leave them
    heads = Hq + 2 * Hkv
    size = torch.exp(1.5 * torch.randn(heads, 1, generator=g, device=dev))
    x = (torch.randn(T, heads, d, generator=g, device=dev) * size).to(torch.bfloat16).reshape(T, heads * d)
    q, k, v = x.split([Hq * d, Hkv * d, Hkv * d], dim=1)
    s.update(q=q, k=k, v=v) if case["fused"] else s.update(q=q.contiguous(), k=k.contiguous(), v=v.contiguous())
    s.update(q_w=(1 + 0.2 * torch.randn(d, generator=g, device=dev)).to(torch.bfloat16),
             k_w=(1 + 0.2 * torch.randn(d, generator=g, device=dev)).to(torch.bfloat16))
    angle = torch.arange(MAX_POS, device=dev, dtype=torch.float64)[:, None] * THETA ** (
        -2 * torch.arange(d // 2, device=dev, dtype=torch.float64) / d)
    s["rope"] = torch.stack([torch.cos(angle), torch.sin(angle)], -1).float()  # [max_pos][d / 2][2]
    s["q_out"] = torch.empty(T, Hq, d, dtype=torch.bfloat16, device=dev)
    kc = torch.randn(num_blocks, Hkv, BLOCK, d, generator=g, device=dev, dtype=torch.bfloat16)
    vc = torch.randn(num_blocks, Hkv, BLOCK, d, generator=g, device=dev, dtype=torch.bfloat16)
    if case["kind"] == "fp8":
        kc, vc = kc.to(torch.float8_e4m3fn), vc.to(torch.float8_e4m3fn)
        s.update(ks=0.01 + 0.02 * torch.rand(Hkv, generator=g, device=dev),
                 vs=0.01 + 0.02 * torch.rand(Hkv, generator=g, device=dev))
    s.update(kc=kc, vc=vc)
    return s


def _prepare_attention(case, seed):
    dev = "cuda"
    B, Hq, Hkv, d = case["B"], case["Hq"], case["Hkv"], case["d"]
    g = torch.Generator(dev).manual_seed(seed)
    rng = np.random.default_rng(seed)
    n = _lengths(case)
    m = _queries(case) if case["op"] == "chunk" else [1] * B
    hide = None
    if not case.get("held", False):  # pages between the sinks and the first window are the pool's again

        def hide(b, j):
            return (j * BLOCK >= case["sinks"]) & ((j + 1) * BLOCK <= n[b] - m[b] + 1 - case["window"])

    num_blocks = _tables(n, np.zeros(sum(-(-x // BLOCK) for x in n), np.int32), hide)[1] + 3
    tables, _ = _tables(n, rng.permutation(num_blocks).astype(np.int32), hide)
    s = dict(case=case, n=_i32(n), tables=_i32(tables), num_blocks=num_blocks, width=tables.shape[1],
             scale=1 / math.sqrt(d), lens=n, news=m)
    lean = torch.randn(Hkv, d, generator=g, device=dev)  # what a head's queries have in common
    k = torch.randn(num_blocks, Hkv, BLOCK, d, generator=g, device=dev, dtype=torch.bfloat16)
    v = torch.randn(num_blocks, Hkv, BLOCK, d, generator=g, device=dev, dtype=torch.bfloat16)
    firsts = _i64([row[0] for row in tables if row[0] >= 0])
    k[firsts, :, :4] += lean[:, None].to(torch.bfloat16)  # the first tokens of a context draw attention
    kind = case.get("kind", "bf16")
    if kind == "fp8":
        k, v = k.to(torch.float8_e4m3fn), v.to(torch.float8_e4m3fn)
        s.update(ks=0.5 + torch.rand(Hkv, generator=g, device=dev), vs=0.5 + torch.rand(Hkv, generator=g, device=dev))
    elif kind == "int8":
        # quantised by groups of 64 tokens and head
        b, j = np.nonzero(tables >= 0)
        group = b.astype(np.int64) * (-(-tables.shape[1] * BLOCK // GROUP)) + j * BLOCK // GROUP
        blk, group = _i64(tables[b, j]), _i64(group)
        for name in ("k", "v"):
            x = (k if name == "k" else v).float()
            top = x.abs().amax((2, 3))  # [num_blocks][Hkv]
            most = torch.zeros(int(group.max()) + 1, Hkv, device=dev)
            most.scatter_reduce_(0, group[:, None].expand(-1, Hkv), top[blk], "amax")
            top[blk] = most[group]
            s[name + "_max"] = top
            code = (x * (127 / top)[..., None, None]).clamp_(-128, 127).trunc_().to(torch.int8)
            k, v = (code, v) if name == "k" else (k, code)
    s.update(k=k, v=v)
    rows = sum(m)
    s["q"] = (torch.randn(rows, Hkv, Hq // Hkv, d, generator=g, device=dev) + 0.5 * lean[:, None]).reshape(
        rows, Hq, d).to(torch.bfloat16)
    s["out"] = torch.empty(rows, Hq, d, dtype=torch.bfloat16, device=dev)
    if case["op"] == "chunk":
        s.update(start=_i32(np.concatenate([[0], np.cumsum(m)])), total=rows, most=max(m))
    return s


def _prepare_pages(case, seed):
    dev = "cuda"
    Hkv, d, blocks, moves = case["Hkv"], case["d"], case["blocks"], case["moves"]
    g = torch.Generator(dev).manual_seed(seed)
    rng = np.random.default_rng(seed)
    # every layer's K and V, [2 * layers][page][...]
    shape = (2 * case["layers"], blocks, Hkv, BLOCK, d)
    if case["kind"] == "bf16":
        whole = {"kv": torch.randn(shape, generator=g, device=dev, dtype=torch.bfloat16)}
    else:
        whole = {"kv": torch.randint(-127, 128, shape, generator=g, device=dev, dtype=torch.int8),
                 "max": 3.5 + torch.rand(shape[:3], generator=g, device=dev)}
    planes = [x for stack in whole.values() for x in stack]
    # pages that hold something move to pages that hold nothing
    order = rng.permutation(blocks)
    return dict(case=case, whole=whole, planes=planes, src=_i32(np.sort(order[:moves])), dst=_i32(np.sort(order[moves:2 * moves])),
                src64=_i64(np.sort(order[:moves])), dst64=_i64(np.sort(order[moves:2 * moves])))


# ------------------------------------------------------------- plain forms --

def _normed(x, weight, s):
    """Normed and rotated heads [T][H][d] in fp32."""
    x = x.float().unflatten(1, (-1, s["case"]["d"]))
    y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * weight.float()
    table = s["rope"][s["pos"].long()]
    c, sn = table[:, None, :, 0], table[:, None, :, 1]
    lo, hi = y.chunk(2, dim=-1)
    return torch.cat([lo * c - hi * sn, hi * c + lo * sn], -1)


def _plain_norm(s):
    c = s["case"]
    s["q_out"].copy_(_normed(s["q"], s["q_w"], s))
    k, v = _normed(s["k"], s["k_w"], s), s["v"].unflatten(1, (-1, c["d"]))
    slot = s["slot"].long()
    blk, off = slot // BLOCK, slot % BLOCK
    if c["kind"] == "fp8":
        top = torch.finfo(torch.float8_e4m3fn).max
        for cache, x, scale in ((s["kc"], k, s["ks"]), (s["vc"], v.float(), s["vs"])):
            cache.view(torch.uint8)[blk, :, off] = (x / scale[:, None]).clamp(-top, top).to(
                torch.float8_e4m3fn).view(torch.uint8)
    else:
        s["kc"][blk, :, off] = k.to(torch.bfloat16)
        s["vc"][blk, :, off] = v
    return _appended(s)


def _appended(s):
    return {"q_out": s["q_out"], "k_cache": s["kc"], "v_cache": s["vc"]}


def _pages_of(s, name, blk):
    """Pages `blk` of K or V in fp32: [..][Hkv][16][d]."""
    kind = s["case"].get("kind", "bf16")
    x = s[name][blk].float()
    if kind == "fp8":
        return x * s[name + "s"][:, None, None]
    if kind == "int8":
        return x * (s[name + "_max"][blk] / 127)[..., None, None]
    return x


def _plain_slide(s):
    c = s["case"]
    B, Hq, Hkv, d, W, sinks = c["B"], c["Hq"], c["Hkv"], c["d"], c["window"], c["sinks"]
    n = s["n"].long()
    # the sinks' pages and the window's, page by page
    few = min(-(-sinks // BLOCK), s["width"])
    many = min(-(-W // BLOCK) + 1, s["width"])
    head = torch.arange(few, device=n.device).expand(B, few)
    tail = torch.clamp((n - W).div(BLOCK, rounding_mode="floor"), min=few)[:, None] + torch.arange(many, device=n.device)
    cols = torch.cat([head, tail], 1)
    t = (cols[..., None] * BLOCK + torch.arange(BLOCK, device=n.device)).flatten(1)
    keep = (t < n[:, None]) & ((t < sinks) | (t >= (n - W)[:, None]))
    blk = s["tables"].long().gather(1, cols.clamp(max=s["width"] - 1)).clamp(min=0)
    k, v = (_pages_of(s, name, blk).transpose(1, 2).flatten(2, 3) for name in ("k", "v"))  # [B][Hkv][tokens][d]
    q = s["q"].float().reshape(B, Hkv, Hq // Hkv, d)
    x = (q @ k.transpose(-1, -2) * s["scale"]).masked_fill(~keep[:, None, None], NEG)
    w = torch.exp(x - x.amax(-1, keepdim=True))
    return {"out": (w @ v / w.sum(-1, keepdim=True)).reshape(B, Hq, d).to(torch.bfloat16)}


def _plain_chunk(s):
    c = s["case"]
    Hq, Hkv, d, W, sinks = c["Hq"], c["Hkv"], c["d"], c["window"], c["sinks"]
    dev = s["q"].device
    row = 0
    for b, (m, n) in enumerate(zip(s["news"], s["lens"])):
        for i in range(0, m, 1024):  # rows of at most 1,024 tokens against the keys they reach
            rows = min(1024, m - i)
            p = torch.arange(n - m + i, n - m + i + rows, device=dev)
            lo, hi = max(0, n - m + i - W + 1), n - m + i + rows
            t = torch.cat([torch.arange(min(sinks, lo), device=dev), torch.arange(lo, hi, device=dev)])
            blk, off = s["tables"][b].long()[t // BLOCK], t % BLOCK
            k, v = s["k"][blk, :, off].float().transpose(0, 1), s["v"][blk, :, off].float().transpose(0, 1)
            q = s["q"][row + i:row + i + rows].float().reshape(rows, Hkv, Hq // Hkv, d).permute(1, 2, 0, 3)
            keep = (t <= p[:, None]) & ((t < sinks) | (t > p[:, None] - W))
            x = (q @ k[:, None].transpose(-1, -2)).mul_(s["scale"]).masked_fill_(~keep, NEG)
            x.sub_(x.amax(-1, keepdim=True)).exp_()
            out = x @ v[:, None] / x.sum(-1, keepdim=True)
            s["out"][row + i:row + i + rows] = out.permute(2, 0, 1, 3).reshape(rows, Hq, d).to(torch.bfloat16)
        row += m
    return {"out": s["out"]}


def _plain_pages(s):
    for x in s["planes"]:
        x[s["dst64"]] = x[s["src64"]]
    return dict(s["whole"])


# --------------------------------------------------------------- the calls --

_space = {}


def _workspace(nbytes):
    """One workspace for all calls, as a program on one stream keeps it."""
    if _space.get("bytes", -1) < nbytes:
        _space.update(bytes=nbytes, buf=torch.empty(max(nbytes, 16), dtype=torch.uint8, device="cuda"))
    return _space["buf"]


def _own(s):
    import paged_kv_decode_25_gb300 as mi
    c = s["case"]
    if c["op"] == "pages":
        if "list" not in s:
            s["list"] = mi.kv_planes(s["planes"])
        mi.check(mi.mi_kv_copy_planes(s["list"], s["src"], s["dst"], c["moves"]))
        return dict(s["whole"])
    if c["op"] == "norm":
        if "dims" not in s:
            s["dims"] = mi.dims(c["T"], c["Hq"], c["Hkv"], c["d"], s["num_blocks"], 1)
        if c["kind"] == "fp8":
            mi.check(mi.mi_paged_kv_append_norm_fp8(s["dims"], s["q"], s["k"], s["v"], s["q_w"], s["k_w"], EPS, s["pos"],
                                                    s["slot"], s["rope"], MAX_POS, s["q_out"], s["kc"], s["vc"], s["ks"],
                                                    s["vs"]))
        else:
            mi.check(mi.mi_paged_kv_append_norm(s["dims"], s["q"], s["k"], s["v"], s["q_w"], s["k_w"], EPS, s["pos"],
                                                s["slot"], s["rope"], MAX_POS, s["q_out"], s["kc"], s["vc"]))
        return _appended(s)
    if "dims" not in s:
        s["dims"] = mi.dims(c["B"], c["Hq"], c["Hkv"], c["d"], s["num_blocks"], s["width"])
        if c["op"] == "slide":
            s["bytes"] = mi.mi_paged_sliding_workspace_bytes(s["dims"], c["window"], c["sinks"])
    dims, W, sinks = s["dims"], c["window"], c["sinks"]
    if c["op"] == "chunk":
        mi.check(mi.mi_paged_prefill_attention_sliding(dims, s["total"], s["most"], s["q"], s["k"], s["v"], s["tables"],
                                                       s["n"], s["start"], W, sinks, s["scale"], s["out"]))
        return {"out": s["out"]}
    space = _workspace(s["bytes"])
    if c["kind"] == "bf16":
        mi.check(mi.mi_paged_decode_attention_sliding(dims, s["q"], s["k"], s["v"], s["tables"], s["n"], W, sinks,
                                                      s["scale"], s["out"], space))
    elif c["kind"] == "fp8":
        mi.check(mi.mi_paged_decode_attention_sliding_fp8(dims, s["q"], s["k"], s["v"], s["ks"], s["vs"], s["tables"],
                                                          s["n"], W, sinks, s["scale"], s["out"], space))
    else:
        mi.check(mi.mi_paged_decode_attention_sliding_int8(dims, s["q"], s["k"], s["v"], s["k_max"], s["v_max"],
                                                           s["tables"], s["n"], W, sinks, s["scale"], s["out"], space))
    return {"out": s["out"]}


def run(state):
    if own:
        return _own(state)
    return {"norm": _plain_norm, "slide": _plain_slide, "chunk": _plain_chunk, "pages": _plain_pages}[
        state["case"]["op"]](state)


# ------------------------------------------------------------------- exact --

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "pages":
        out = {name: x.double() for name, x in s["whole"].items()}
        for src, dst in zip(s["src"].tolist(), s["dst"].tolist()):
            for x in out.values():
                x[:, dst] = x[:, src]
        return out
    return _exact_norm(s) if case["op"] == "norm" else _exact_attention(s)


def _exact_norm(s):
    c = s["case"]
    d, T = c["d"], c["T"]
    pos, slot = s["pos"].long(), s["slot"].long()
    z = torch.view_as_complex(s["rope"].double())[pos]  # the rotation as a complex factor

    def head(x, w):
        x = x.double()
        y = x / torch.sqrt(x.square().sum(-1, keepdim=True) / d + EPS) * w.double()
        y = torch.complex(y[:, :d // 2], y[:, d // 2:]) * z
        return torch.cat([y.real, y.imag], -1)

    q_out = torch.stack([head(s["q"][:, j * d:(j + 1) * d], s["q_w"]) for j in range(c["Hq"])], 1)
    kc, vc = s["kc"].double(), s["vc"].double()
    at = (slot // BLOCK, slot % BLOCK)
    for h in range(c["Hkv"]):
        k, v = head(s["k"][:, h * d:(h + 1) * d], s["k_w"]), s["v"][:, h * d:(h + 1) * d].double()
        if c["kind"] == "fp8":
            k, v = ((x / scale[h].double()).clamp(-448, 448) for x, scale in ((k, s["ks"]), (v, s["vs"])))
        kc[at[0], h, at[1]], vc[at[0], h, at[1]] = k, v
    return {"q_out": q_out, "k_cache": kc, "v_cache": vc}


def _exact_attention(s):
    """Row by row of a KV head: every key of the context, most of them masked."""
    c = s["case"]
    Hq, Hkv, d = c["Hq"], c["Hkv"], c["d"]
    G, kind, dev = Hq // Hkv, c.get("kind", "bf16"), s["q"].device
    out = torch.zeros(sum(s["news"]), Hq, d, dtype=torch.float64, device=dev)
    step, row = 2048, 0
    for b, (m, n) in enumerate(zip(s["news"], s["lens"])):
        for i in range(0, m, step):
            p = torch.arange(n - m + i, min(n - m + i + step, n), device=dev)
            # keys nobody in these rows sees carry no weight: left out
            t = torch.arange(int(p[-1]) + 1, device=dev)
            t = t[(t < c["sinks"]) | (t > int(p[0]) - c["window"])]
            blk, off = s["tables"][b].long()[t // BLOCK], t % BLOCK
            hidden = ~((t <= p[:, None]) & ((t < c["sinks"]) | (p[:, None] - t < c["window"])))
            for h in range(Hkv):
                k, v = s["k"][blk, h, off].double(), s["v"][blk, h, off].double()
                if kind == "fp8":
                    k, v = k * s["ks"][h].double(), v * s["vs"][h].double()
                elif kind == "int8":
                    k, v = (x * s[a][blk, h].double()[:, None] / 127 for x, a in ((k, "k_max"), (v, "v_max")))
                for j in range(h * G, h * G + G):
                    x = s["q"][row + i:row + i + len(p), j].double() @ k.T * s["scale"]
                    out[row + i:row + i + len(p), j] = torch.softmax(x.masked_fill(hidden, NEG), -1) @ v
        row += m
    return {"out": out}
