"""The cache-saving operators of a paged decode: their cases, plain forms and exact values.

Four operators that belong to one serving loop over a paged KV cache:

  prefix  decode attention of a batch whose requests share long prefixes, each
          prefix's keys and values read once for all its requests
  scored  decode attention that also keeps, for every cached token and KV head,
          the attention weight the token has received
  window  the same weights of many query tokens at once (a prompt's last tokens,
          or a whole prompt), which give a prompt its first scores
  evict   a smaller cache from those scores: each request keeps its newest tokens
          and the heaviest of the older ones, per KV head

`own` chooses between the plain form (torch operations in fp32) and the
library's calls.
"""
import math
import random

import numpy as np
import torch

own = False

BLOCK = 16
NEG = float("-inf")
SHAPES = ((32, 8, 128), (16, 8, 128), (28, 4, 128), (4, 2, 64), (8, 8, 64), (8, 1, 128))  # Hq, Hkv, head_dim


# ------------------------------------------------------------------ cases --

def listed():
    return [
        # a few chats behind one short system prompt: the latency of the smallest call
        dict(name="prefix_short", op="prefix", B=4, Hq=16, Hkv=8, d=128, P=1, loose=0, p_lo=100, p_hi=100, lo=1, hi=40,
             lens=1),
        # a serving batch behind one system prompt, its chats of very different lengths
        dict(name="prefix_chats", op="prefix", B=64, Hq=32, Hkv=8, d=128, P=1, loose=0, p_lo=4100, p_hi=4100, lo=32,
             hi=1024, lens=2),
        # many questions about one long document, the answers just begun
        dict(name="prefix_document", op="prefix", B=128, Hq=32, Hkv=8, d=128, P=1, loose=0, p_lo=32000, p_hi=32000,
             lo=16, hi=512, lens=3),
        # several prefixes with groups of all sizes, some requests with none; seven query heads per KV head
        dict(name="prefix_groups", op="prefix", B=90, Hq=28, Hkv=4, d=128, P=6, loose=5, p_lo=500, p_hi=6000, lo=0,
             hi=900, lens=4),
        # one short chat: the latency of a scored step
        dict(name="scored_single", op="scored", B=1, Hq=32, Hkv=8, d=128, fp8=False, fresh=True, lo=1000, hi=1000,
             lens=5),
        # a serving batch, weights accumulated over its steps
        dict(name="scored_batch", op="scored", B=64, Hq=32, Hkv=8, d=128, fp8=False, fresh=False, lo=512, hi=8192,
             lens=6),
        # a few long contexts in an e4m3 cache
        dict(name="scored_fp8_long", op="scored", B=8, Hq=32, Hkv=8, d=128, fp8=True, fresh=True, lo=20000, hi=60000,
             lens=7),
        # the last tokens of a batch of prompts look back over them
        dict(name="window_batch", op="window", B=16, Hq=32, Hkv=8, d=128, fresh=True, q_lo=32, q_hi=64, lo=1000,
             hi=16000, lens=8),
        # whole prompts, every token's weight on all before it
        dict(name="window_prompts", op="window", B=2, Hq=32, Hkv=8, d=128, fresh=True, q_lo=0, q_hi=0, lo=4000, hi=7000,
             lens=9),
        # one short cache cut down
        dict(name="evict_single", op="evict", B=1, Hq=16, Hkv=8, d=128, fp8=False, lo=700, hi=700, keep=500, recent=64,
             lens=10),
        # a serving batch cut to its budget
        dict(name="evict_batch", op="evict", B=64, Hq=32, Hkv=8, d=128, fp8=False, lo=2000, hi=8192, keep=2048,
             recent=256, lens=11),
        # a few long contexts in an e4m3 cache cut to a quarter and less
        dict(name="evict_fp8_long", op="evict", B=4, Hq=28, Hkv=4, d=128, fp8=True, lo=30000, hi=120000, keep=8000,
             recent=1000, lens=12),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    most = {}
    for c in listed():
        w = work(c)
        most[c["op"]] = max(most.get(c["op"], 0), max(w["bytes"], w["flops"] / 50))
    while True:
        op = rng.choice(("prefix", "scored", "window", "evict"))
        Hq, Hkv, d = rng.choice(SHAPES)
        c = dict(op=op, B=_log(rng, 1, 128), Hq=Hq, Hkv=Hkv, d=d, lens=rng.randrange(1 << 30))
        if op == "prefix":
            a, b = _log(rng, 1, 900), _log(rng, 1, 900)
            p, q = _log(rng, 50, 32000), _log(rng, 50, 32000)
            c.update(P=_log(rng, 1, min(8, c["B"])), loose=rng.choice((0, 0, min(3, c["B"] - 1))), p_lo=min(p, q),
                     p_hi=max(p, q), lo=min(a, b), hi=max(a, b))
        elif op == "scored":
            a, b = _log(rng, 1, 60000), _log(rng, 1, 60000)
            c.update(fp8=rng.random() < 0.5, fresh=rng.random() < 0.5, lo=min(a, b), hi=max(a, b))
        elif op == "window":
            a, b = _log(rng, 20, 16000), _log(rng, 20, 16000)
            whole = rng.random() < 0.4
            m = 0 if whole else _log(rng, 1, 128)
            c.update(fresh=rng.random() < 0.5, q_lo=m, q_hi=m + m // 2, lo=min(a, b), hi=max(a, b))
            c["B"] = min(c["B"], 16)
        else:
            a, b = _log(rng, 100, 120000), _log(rng, 100, 120000)
            keep = _log(rng, 32, 9000)
            c.update(fp8=rng.random() < 0.5, lo=min(a, b), hi=max(a, b), keep=keep, recent=rng.randrange(keep + 1))
        w = work(c)
        if max(w["bytes"], w["flops"] / 50) <= most[op]:
            return c


# ---------------------------------------------------------------- lengths --

def _lengths(case):
    """Tokens each request holds (log-uniform over the case's range)."""
    r = random.Random(case["lens"])
    lo, hi = case["lo"], case["hi"]
    return [min(hi, max(lo, int(math.exp(r.uniform(math.log(lo + 1), math.log(hi + 2)))) - 1)) for _ in range(case["B"])]


def _prefixes(case):
    """(prefix lengths [P], group starts [P + 1]): the last `loose` requests have no prefix."""
    r = random.Random(case["lens"] + 1)
    P, grouped = case["P"], case["B"] - case["loose"]
    lens = [_log(r, case["p_lo"], case["p_hi"]) for _ in range(P)]
    cuts = sorted(r.sample(range(1, grouped), P - 1)) if grouped > P - 1 else list(range(1, P))
    return lens, [0] + cuts + [grouped]


def _queries(case):
    """Query tokens per request (`q_lo` 0: the whole prompt)."""
    r = random.Random(case["lens"] + 2)
    n = _lengths(case)
    return [min(x, r.randint(case["q_lo"], case["q_hi"])) if case["q_lo"] else x for x in n]


def work(case):
    Hq, Hkv, d, B = case["Hq"], case["Hkv"], case["d"], case["B"]
    n = _lengths(case)
    e = 1 if case.get("fp8") else 2
    if case["op"] == "prefix":
        lens, start = _prefixes(case)
        total = sum(n) + sum(p * (b - a) for p, a, b in zip(lens, start, start[1:]))
        return dict(bytes=2 * 2 * d * Hkv * (sum(n) + sum(lens)) + 2 * 2 * B * Hq * d, flops=4 * d * Hq * total)
    if case["op"] == "scored":
        return dict(bytes=2 * e * d * Hkv * sum(n) + (4 if case["fresh"] else 8) * Hkv * sum(n) + 2 * 2 * B * Hq * d,
                    flops=4 * d * Hq * sum(n))
    if case["op"] == "window":
        m = _queries(case)
        pairs = sum(q * (x - q) + q * (q + 1) // 2 for q, x in zip(m, n))
        return dict(bytes=2 * d * Hkv * sum(n) + 2 * d * Hq * sum(m) + (4 if case["fresh"] else 8) * Hkv * sum(n),
                    flops=2 * d * Hq * pairs)
    kept = sum(min(x, case["keep"]) for x in n)
    return dict(bytes=4 * Hkv * sum(n) + Hkv * kept * (2 * 2 * e * d + 4), flops=Hkv * sum(n))


# ----------------------------------------------------------------- inputs --

def _blocks(n):
    return [-(-x // BLOCK) for x in n]


def _tables(n, first, order, width):
    t = np.full((len(n), width), -1, np.int32)
    for row, k in zip(t, _blocks(n)):
        row[:k] = order[first:first + k]
        first += k
    return t, first


def _live(n):
    """(request, table column) of every block that holds a token."""
    k = np.asarray(_blocks(n), np.int64)
    return np.repeat(np.arange(len(n)), k), np.concatenate([np.arange(x) for x in k] or [np.zeros(0, np.int64)])


def prepare(case, seed):
    dev = "cuda"
    B, Hq, Hkv, d = case["B"], case["Hq"], case["Hkv"], case["d"]
    fp8 = bool(case.get("fp8"))
    g = torch.Generator(dev).manual_seed(seed)
    nprng = np.random.default_rng(seed)
    n = _lengths(case)
    p_lens, p_start = _prefixes(case) if case["op"] == "prefix" else ([], [])
    kept = [min(x, case["keep"]) for x in n] if case["op"] == "evict" else []
    num_blocks = sum(_blocks(n)) + sum(_blocks(p_lens)) + sum(_blocks(kept)) + 3
    order = nprng.permutation(num_blocks).astype(np.int32)

    def i32(x):
        return torch.as_tensor(np.asarray(x, np.int32)).to(dev)

    def i64(x):
        return torch.as_tensor(np.asarray(x, np.int64)).to(dev)

    width = max(_blocks(n) + [1])
    tables, used = _tables(n, 0, order, width)
    s = dict(case=case, n=i32(n), tables=i32(tables), num_blocks=num_blocks, width=width, scale=1 / math.sqrt(d))
    lean = torch.randn(Hkv, d, generator=g, device=dev)  # what a head's queries have in common

    def cache(sinks):
        x = torch.randn(num_blocks, Hkv, BLOCK, d, generator=g, device=dev, dtype=torch.bfloat16)
        if sinks is not None and len(sinks):  # the first tokens of a context draw attention
            x[sinks, :, :4] += lean[:, None].to(torch.bfloat16)
        return x

    def queries(rows):
        return (torch.randn(rows, Hkv, Hq // Hkv, d, generator=g, device=dev) + 0.5 * lean[:, None]).reshape(
            rows, Hq, d).to(torch.bfloat16)

    if case["op"] == "prefix":
        p_width = max(_blocks(p_lens) + [1])
        p_tables, used = _tables(p_lens, used, order, p_width)
        sinks = i64([row[0] for row, x in zip(p_tables, p_lens) if x])
        s.update(k=cache(sinks), v=cache(None), q=queries(B), out=torch.empty(B, Hq, d, dtype=torch.bfloat16, device=dev),
                 p_tables=i32(p_tables), p_lens=i32(p_lens), p_start=i32(p_start), P=case["P"], p_width=p_width)
        # where each request stands among the groups, padded to the largest (the last place: none)
        most = max(b - a for a, b in zip(p_start, p_start[1:]))
        place = np.full(B, case["P"] * most, np.int64)
        rows = np.zeros((case["P"], most), np.int64)
        for j, (a, b) in enumerate(zip(p_start, p_start[1:])):
            place[a:b] = j * most + np.arange(b - a)
            rows[j, :b - a] = np.arange(a, b)
        s.update(place=i64(place), rows=i64(rows))
        return s
    sinks = i64([row[0] for row, x in zip(tables, n) if x])
    k, v = cache(sinks), cache(None) if case["op"] != "window" else None
    if fp8:
        k, v = k.to(torch.float8_e4m3fn), v.to(torch.float8_e4m3fn)
    s.update(k=k, v=v)
    live = _live(n)
    s.update(live_b=i64(live[0]), live_j=i64(live[1]))
    if case["op"] == "window":
        m = _queries(case)
        start = np.concatenate([[0], np.cumsum(m)])
        rows = np.minimum(start[:-1, None] + np.arange(max(m)), max(sum(m) - 1, 0))
        s.update(q=queries(sum(m)), m=i32(m), start=i32(start), total=int(sum(m)), most=int(max(m)), rows=i64(rows))
    elif case["op"] == "scored":
        s.update(q=queries(B), out=torch.empty(B, Hq, d, dtype=torch.bfloat16, device=dev))
        if fp8:
            s.update(ks=0.5 + torch.rand(Hkv, generator=g, device=dev), vs=0.5 + torch.rand(Hkv, generator=g, device=dev))
    # weights gathered so far: most tokens little, a few much, some none at all
    before = torch.exp(2 * torch.randn(num_blocks, Hkv, BLOCK, generator=g, device=dev)) * 1e-3
    before *= torch.rand(num_blocks, Hkv, BLOCK, generator=g, device=dev) > 0.05
    s["scores"] = before
    if case["op"] in ("scored", "window") and not case["fresh"]:
        s["before"] = before.clone()
    if case["op"] == "evict":
        to, used = _tables(kept, used, order, width)
        rows = _rows(to, kept)
        s.update(to=i32(to), budget=i32([case["keep"]] * B), new=torch.empty(B, dtype=torch.int32, device=dev),
                 most=max(kept), dst_b=i64(rows[0]), dst_t=i64(rows[1]), dst_blk=i64(rows[2]))
    return s


def _rows(tables, n):
    """(request, token, block) of every token."""
    b = np.repeat(np.arange(len(n)), n)
    t = np.concatenate([np.arange(x) for x in n] or [np.zeros(0, np.int64)])
    return b, t, tables[b, t // BLOCK]


# ------------------------------------------------------------- plain forms --

def _tokens(cache, tables):
    """[B][Hkv][16 * columns][d] in fp32: the cache's tokens in the tables' order."""
    x = cache[tables.clamp(min=0).long()]  # [B][columns][Hkv][16][d]
    return x.transpose(1, 2).flatten(2, 3).float()


def _softmax_parts(q, k, v, keep, scale):
    """(max, sum, weighted values) over the kept keys; q [..][rows][d]."""
    x = (q @ k.transpose(-1, -2) * scale).masked_fill(~keep, NEG)
    top = x.amax(-1, keepdim=True).clamp(min=torch.finfo(torch.float32).min)
    w = torch.exp(x - top)
    return top, w.sum(-1, keepdim=True), w @ v


def _plain_prefix(s):
    c = s["case"]
    B, Hq, Hkv, d, P = c["B"], c["Hq"], c["Hkv"], c["d"], c["P"]
    G = Hq // Hkv
    q = s["q"].float().reshape(B, Hkv, G, d)
    at = torch.arange(s["width"] * BLOCK, device=q.device)
    m2, l2, o2 = _softmax_parts(q, _tokens(s["k"], s["tables"]), _tokens(s["v"], s["tables"]),
                                (at < s["n"][:, None])[:, None, None], s["scale"])
    qp = q[s["rows"]].permute(0, 2, 1, 3, 4).flatten(2, 3)  # [P][Hkv][group * G][d]
    at = torch.arange(s["p_width"] * BLOCK, device=q.device)
    parts = _softmax_parts(qp, _tokens(s["k"], s["p_tables"]), _tokens(s["v"], s["p_tables"]),
                           (at < s["p_lens"][:, None])[:, None, None], s["scale"])

    def by_request(x, none):
        x = x.unflatten(2, (-1, G)).transpose(1, 2).flatten(0, 1)  # [P * group][Hkv][G][.]
        return torch.cat([x, torch.full_like(x[:1], none)])[s["place"]]

    low = torch.finfo(torch.float32).min
    m1, l1, o1 = by_request(parts[0], low), by_request(parts[1], 0.0), by_request(parts[2], 0.0)
    top = torch.maximum(m1, m2)
    f1, f2 = torch.exp(m1 - top), torch.exp(m2 - top)
    total = l1 * f1 + l2 * f2
    out = torch.where(total > 0, (o1 * f1 + o2 * f2) / total, torch.zeros((), device=q.device))
    return {"out": out.reshape(B, Hq, d).to(torch.bfloat16)}


def _add_scores(s, w, new):
    """w [B][Hkv][tokens]: set where a token is new (or all are), added elsewhere."""
    c = s["case"]
    B, Hkv = w.shape[:2]
    scores = s["scores"]
    if not c["fresh"]:
        scores.copy_(s["before"])
    blk = s["tables"][s["live_b"], s["live_j"]].long()
    at = torch.arange(w.shape[2], device=w.device)
    inside = (at < s["n"][:, None])[:, None].expand_as(w)
    fresh = torch.ones_like(inside) if c["fresh"] else (at >= new[:, None])[:, None].expand_as(w)

    def cut(x):
        return x.reshape(B, Hkv, -1, BLOCK)[s["live_b"], :, s["live_j"]]

    old = scores[blk]
    scores[blk] = torch.where(cut(inside), cut(w) + torch.where(cut(fresh), torch.zeros_like(old), old), old)
    return scores


def _plain_scored(s):
    c = s["case"]
    B, Hq, Hkv, d = c["B"], c["Hq"], c["Hkv"], c["d"]
    q = s["q"].float().reshape(B, Hkv, Hq // Hkv, d)
    k, v = _tokens(s["k"], s["tables"]), _tokens(s["v"], s["tables"])
    if c["fp8"]:
        k, v = k * s["ks"][:, None, None], v * s["vs"][:, None, None]
    keep = (torch.arange(k.shape[2], device=q.device) < s["n"][:, None])[:, None, None]
    x = (q @ k.transpose(-1, -2) * s["scale"]).masked_fill(~keep, NEG)
    w = torch.exp(x - x.amax(-1, keepdim=True).clamp(min=torch.finfo(torch.float32).min))
    total = w.sum(-1, keepdim=True)
    w = torch.where(total > 0, w / total, torch.zeros((), device=q.device))
    return {"out": (w @ v).reshape(B, Hq, d).to(torch.bfloat16), "scores": _add_scores(s, w.sum(2), s["n"] - 1)}


def _plain_window(s):
    c = s["case"]
    B, Hq, Hkv, d = c["B"], c["Hq"], c["Hkv"], c["d"]
    q = s["q"].float()[s["rows"]].reshape(B, s["most"], Hkv, Hq // Hkv, d).permute(0, 2, 3, 1, 4)
    k = _tokens(s["k"], s["tables"])[:, :, None]
    i, t = torch.arange(s["most"], device=q.device), torch.arange(k.shape[3], device=q.device)
    pos = (s["n"] - s["m"])[:, None] + i
    keep = (t <= pos[..., None]) & (i < s["m"][:, None])[..., None]
    x = (q @ k.transpose(-1, -2)).mul_(s["scale"]).masked_fill_(~keep[:, None, None], NEG)
    x.sub_(x.amax(-1, keepdim=True).clamp(min=torch.finfo(torch.float32).min)).exp_()
    x.div_(x.sum(-1, keepdim=True).clamp(min=torch.finfo(torch.float32).tiny))
    return {"scores": _add_scores(s, x.sum((2, 3)), s["n"] - s["m"])}


def _plain_evict(s):
    c = s["case"]
    B, Hkv = c["B"], c["Hkv"]
    n, tables = s["n"].long(), s["tables"].clamp(min=0).long()
    x = s["scores"][tables].transpose(1, 2).flatten(2, 3)  # [B][Hkv][tokens]
    t = torch.arange(x.shape[2], device=x.device)
    new = torch.minimum(n, s["budget"].long())
    recent = new.clamp(max=c["recent"])
    old = (t < (n - recent)[:, None])[:, None].expand_as(x)
    rank = torch.sort(x.masked_fill(~old, NEG), dim=-1, descending=True, stable=True).indices
    heavy = torch.zeros_like(x, dtype=torch.bool).scatter_(-1, rank, (t < (new - recent)[:, None])[:, None].expand_as(x))
    keep = heavy | ((t < n[:, None]) & (t >= (n - recent)[:, None]))[:, None]
    src = torch.sort((~keep).to(torch.int8), dim=-1, stable=True).indices[:, :, :s["most"]]
    b, dst, blk = s["dst_b"], s["dst_t"], s["dst_blk"]
    src = src[b, :, dst]  # [rows][Hkv]
    h = torch.arange(Hkv, device=x.device)
    at = (tables[b[:, None], src // BLOCK], h, src % BLOCK)
    to = (blk[:, None], h, (dst % BLOCK)[:, None])
    for a in (s["k"], s["v"]):
        raw = a.view(torch.uint8) if c["fp8"] else a
        raw[to] = raw[at]
    s["scores"][to] = s["scores"][at]
    s["new"].copy_(new)
    return _evicted(s)


def _evicted(s):
    return {"k": s["k"], "v": s["v"], "scores": s["scores"], "new_lens": s["new"]}


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
    if "dims" not in s:
        s["dims"] = mi.dims(c["B"], c["Hq"], c["Hkv"], c["d"], s["num_blocks"], s["width"])
        s["bytes"] = {"prefix": lambda: mi.mi_paged_prefix_workspace_bytes(s["dims"], c["P"], s["p_width"]),
                      "scored": lambda: mi.mi_paged_scored_workspace_bytes(s["dims"]),
                      "window": lambda: mi.mi_paged_prefill_scores_workspace_bytes(s["dims"], s["total"], s["most"]),
                      "evict": lambda: mi.mi_paged_kv_evict_workspace_bytes(s["dims"])}[c["op"]]()
    dims, space = s["dims"], _workspace(s["bytes"])
    if c["op"] == "prefix":
        mi.check(mi.mi_paged_decode_attention_prefix(dims, c["P"], s["p_width"], s["q"], s["k"], s["v"], s["p_tables"],
                                                     s["p_lens"], s["p_start"], s["tables"], s["n"], s["scale"],
                                                     s["out"], space))
        return {"out": s["out"]}
    if c["op"] == "evict":
        evict = mi.mi_paged_kv_evict_fp8 if c["fp8"] else mi.mi_paged_kv_evict
        mi.check(evict(dims, s["k"], s["v"], s["scores"], s["tables"], s["n"], s["budget"], c["recent"], s["to"],
                       s["new"], space))
        return _evicted(s)
    if not c["fresh"]:
        s["scores"].copy_(s["before"])
    if c["op"] == "window":
        mi.check(mi.mi_paged_prefill_scores(dims, s["total"], s["most"], s["q"], s["k"], s["tables"], s["n"], s["start"],
                                            s["scale"], c["fresh"], s["scores"], space))
        return {"scores": s["scores"]}
    if c["fp8"]:
        mi.check(mi.mi_paged_decode_attention_scored_fp8(dims, s["q"], s["k"], s["v"], s["ks"], s["vs"], s["tables"],
                                                         s["n"], s["scale"], c["fresh"], s["out"], s["scores"], space))
    else:
        mi.check(mi.mi_paged_decode_attention_scored(dims, s["q"], s["k"], s["v"], s["tables"], s["n"], s["scale"],
                                                     c["fresh"], s["out"], s["scores"], space))
    return {"out": s["out"], "scores": s["scores"]}


def run(state):
    if own:
        return _own(state)
    return {"prefix": _plain_prefix, "scored": _plain_scored, "window": _plain_window, "evict": _plain_evict}[
        state["case"]["op"]](state)


# ------------------------------------------------------------------- exact --

def _one(cache, table, n, h, scale=1.0):
    """Tokens 0..n-1 of one KV head of one request, in 64 bits."""
    t = torch.arange(n, device=cache.device)
    return cache[table.long()[t // BLOCK], h, t % BLOCK].double() * scale


def exact(case, seed):
    s = prepare(case, seed)
    B, Hq, Hkv, d = case["B"], case["Hq"], case["Hkv"], case["d"]
    G, n, dev = Hq // Hkv, _lengths(case), s["k"].device
    if case["op"] == "prefix":
        p_lens, start = _prefixes(case)
        out = torch.zeros(B, Hq, d, dtype=torch.float64, device=dev)
        group = [next((j for j in range(case["P"]) if start[j] <= b < start[j + 1]), None) for b in range(B)]
        for h in range(Hkv):
            pre = [(_one(s["k"], t, x, h), _one(s["v"], t, x, h)) for t, x in zip(s["p_tables"], p_lens)]
            for b in range(B):
                k, v = _one(s["k"], s["tables"][b], n[b], h), _one(s["v"], s["tables"][b], n[b], h)
                if group[b] is not None:
                    k, v = torch.cat([pre[group[b]][0], k]), torch.cat([pre[group[b]][1], v])
                if len(k):
                    w = torch.softmax(s["q"][b, h * G:(h + 1) * G].double() @ k.T * s["scale"], -1)
                    out[b, h * G:(h + 1) * G] = w @ v
        return {"out": out}
    if case["op"] == "evict":
        scores = s["scores"].double()
        k, v, new = s["k"].double(), s["v"].double(), [min(x, case["keep"]) for x in n]
        for b in range(B):
            r = min(new[b], case["recent"])
            for h in range(Hkv):
                x = _one(s["scores"][..., None], s["tables"][b], n[b], h)[:, 0].cpu().numpy()
                first = np.lexsort((np.arange(n[b] - r), -x[:n[b] - r]))[:new[b] - r]
                src = torch.as_tensor(np.concatenate([np.sort(first), np.arange(n[b] - r, n[b])])).to(dev)
                dst = torch.arange(new[b], device=dev)
                at = (s["tables"][b].long()[src // BLOCK], h, src % BLOCK)
                to = (s["to"][b].long()[dst // BLOCK], h, dst % BLOCK)
                for x in (k, v, scores):
                    x[to] = x[at]
        return {"k": k, "v": v, "scores": scores, "new_lens": torch.tensor(new, dtype=torch.int32, device=dev)}
    scores = s["scores"].double()
    out = torch.zeros(B, Hq, d, dtype=torch.float64, device=dev)
    m = _queries(case) if case["op"] == "window" else [1] * B
    first = np.concatenate([[0], np.cumsum(m)])
    for b in range(B):
        for h in range(Hkv):
            if not n[b]:
                continue
            k = _one(s["k"], s["tables"][b], n[b], h, s["ks"][h].double() if case.get("fp8") else 1.0)
            q = s["q"][first[b]:first[b + 1], h * G:(h + 1) * G].double().transpose(0, 1)  # [G][m][d]
            x = q @ k.T * s["scale"]
            t = torch.arange(n[b], device=dev)
            x = x.masked_fill(t > (n[b] - m[b] + torch.arange(m[b], device=dev))[:, None], NEG)
            w = torch.softmax(x, -1)
            at = (s["tables"][b].long()[t // BLOCK], h, t % BLOCK)
            kept = scores[at] * (0.0 if case["fresh"] else (t < n[b] - m[b]).double())
            scores[at] = kept + w.sum((0, 1))
            if case["op"] == "scored":
                out[b, h * G:(h + 1) * G] = w[:, 0] @ _one(s["v"], s["tables"][b], n[b], h,
                                                           s["vs"][h].double() if case["fp8"] else 1.0)
    return {"scores": scores} if case["op"] == "window" else {"out": out, "scores": scores}
