"""Performance cases of the key/value cache operators.

Three operators of a model that answers one token at a time from a paged key/value cache of int8 codes (one fp32
scale per token and head) or bf16 values:

  append   rotary positions on q and k (one to three position axes), then k and v quantized into their pages
  attend   attention of one new token per sequence over its pages, optionally adding each token's attention weight
           to the cache's running score
  evict    the tokens with the largest running score (and the first and the most recent ones) moved, in order, into
           fewer pages

`own` selects between the library's calls and a plain form in elementary torch operations, in fp32.
"""
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "s8": torch.int8}
SIZE = {"f32": 4, "bf16": 2, "s8": 1}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _append(tokens, batch, heads, kv_heads, dim, page, rot, axes, type, cache, interleaved=False, mix=1):
    return {"op": "append", "tokens": tokens, "batch": batch, "heads": heads, "kv_heads": kv_heads, "dim": dim,
            "page": page, "rot": rot, "axes": axes, "type": type, "cache": cache, "interleaved": interleaved,
            "mix": mix}


def _attend(batch, length, heads, kv_heads, dim, page, type, cache, ragged=False, empty=False, window=0,
            accumulate=False, mix=1):
    return {"op": "attend", "batch": batch, "length": length, "heads": heads, "kv_heads": kv_heads, "dim": dim,
            "page": page, "type": type, "cache": cache, "ragged": ragged, "empty": empty, "window": window,
            "accumulate": accumulate, "mix": mix}


def _evict(batch, length, budget, sink, recent, kv_heads, dim, page, cache, ragged=False, mix=1):
    return {"op": "evict", "batch": batch, "length": length, "budget": budget, "sink": sink, "recent": recent,
            "kv_heads": kv_heads, "dim": dim, "page": page, "cache": cache, "ragged": ragged, "mix": mix}


def listed():
    return [
        # one user, one new token: the call is all latency
        {"name": "append 1 token", **_append(1, 1, 32, 8, 128, 16, 128, 1, "bf16", "s8")},
        # a decode step of a full batch; fp32 activations, half of each head rotated, no shared heads
        {"name": "append 96 x 1 fp32", **_append(96, 96, 12, 12, 64, 24, 32, 1, "f32", "bf16", True)},
        # the prompt of an image or video question: time, height and width positions
        {"name": "append prompt 16384", **_append(16384, 4, 32, 8, 128, 32, 128, 3, "bf16", "s8")},
        # the first answer tokens after a short prompt
        {"name": "attend 1 x 80", **_attend(1, 80, 32, 8, 128, 16, "bf16", "s8")},
        # an ordinary serving batch: ragged lengths, slots without a sequence among them
        {"name": "attend 48 ragged 4096", **_attend(48, 4096, 32, 8, 128, 16, "bf16", "s8", True, True)},
        # fp32 activations over an unquantized cache, no shared heads, pages that no tile divides, scores kept
        {"name": "attend 24 fp32 odd pages", **_attend(24, 2500, 16, 16, 64, 24, "f32", "bf16", True, False, 0, True)},
        # one key/value head for sixteen query heads of 256, sliding window
        {"name": "attend 32 shared window", **_attend(32, 9000, 16, 1, 256, 64, "bf16", "bf16", True, False, 4096)},
        # one user with a very long document: the work has to be split over the cache's length
        {"name": "attend 1 x 131072", **_attend(1, 131072, 32, 8, 128, 16, "bf16", "s8")},
        # the largest batch, with the scores that eviction reads
        {"name": "attend 64 x 8192 scores", **_attend(64, 8192, 32, 8, 128, 32, "bf16", "s8", False, False, 0, True)},
        # one conversation over its budget
        {"name": "evict 1 x 1000", **_evict(1, 1000, 512, 4, 128, 8, 128, 16, "s8")},
        # a batch halved and more, ragged lengths, some within the budget already
        {"name": "evict 32 ragged 8192", **_evict(32, 8192, 2048, 4, 256, 8, 128, 32, "s8", True)},
        # a long document cut to a quarter, unquantized
        {"name": "evict 1 x 131072", **_evict(1, 131072, 32768, 16, 4096, 8, 128, 16, "bf16")},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("append", "attend", "attend", "evict"))
    dim = rng.choice((64, 80, 96, 128, 128, 192, 256))
    page = rng.choice((8, 16, 16, 24, 32, 64, 128))
    kv_heads = rng.choice((1, 2, 4, 8, 8, 16))
    group = rng.choice((1, 2, 4, 4, 7, 8, 16))
    type, cache = rng.choice(("bf16", "bf16", "f32")), rng.choice(("s8", "s8", "bf16"))
    mix = rng.randrange(1 << 20)
    row = kv_heads * dim * SIZE[cache]
    if op == "append":
        most = max(1, min(16384, (1 << 28) // ((group + 2) * kv_heads * dim * SIZE[type])))
        tokens = _log(rng, 1, most)
        return _append(tokens, rng.randint(1, min(tokens, 64)), kv_heads * group, kv_heads, dim, page,
                       rng.choice((dim, dim, dim // 2)), rng.choice((1, 2, 3)), type, cache, rng.random() < 0.5, mix)
    if op == "attend":
        tokens = _log(rng, 64, max(64, min(400000, (1 << 29) // (2 * row * max(1, group // 4)))))
        batch = min(_log(rng, 1, 128), tokens)
        ragged = rng.random() < 0.7
        return _attend(batch, max(1, tokens // batch), kv_heads * group, kv_heads, dim, page, type, cache, ragged,
                       ragged and rng.random() < 0.5, rng.choice((0, 0, 0, rng.randint(1, 2000))),
                       rng.random() < 0.4, mix)
    tokens = _log(rng, 64, max(64, min(131072, (1 << 28) // (2 * row))))
    batch = min(_log(rng, 1, 64), tokens // 32 + 1)
    length = max(2, tokens // batch)
    budget = rng.randint(max(1, length // 8), length)
    sink = rng.choice((0, min(4, budget)))
    return _evict(batch, length, budget, sink, rng.randint(0, (budget - sink) // 2), kv_heads, dim, page, cache,
                  rng.random() < 0.7, mix)


def _lengths(c):
    """The sequences' lengths, a function of the case alone."""
    if c["op"] == "append":
        per = [c["tokens"] // c["batch"] + (b < c["tokens"] % c["batch"]) for b in range(c["batch"])]
        r = random.Random(c["mix"])
        return [r.randint(0, 500) + n for n in per], per
    r = random.Random(c["mix"])
    lens = [c["length"]] * c["batch"]
    if c["ragged"]:
        lens = [r.randint(max(1, c["length"] // 16), c["length"]) for _ in lens]
    if c.get("empty"):
        lens = [0 if r.random() < 0.1 else n for n in lens]
        lens[0] = 0
        lens[-1] = c["length"]
    return lens, None


def work(c):
    lens, per = _lengths(c)
    D, H, e = c["dim"], c["kv_heads"], SIZE[c["cache"]]
    row = H * (2 * D * e + (8 if c["cache"] == "s8" else 0))  # a token's keys and values
    if c["op"] == "append":
        T, t = c["tokens"], SIZE[c["type"]]
        rows = T if c["axes"] == 1 else min(T, _side(c) * 4)
        read = T * (c["heads"] + 2 * H) * D * t + rows * c["rot"] * 4
        back = T * H * 2 * D * 2 if c["cache"] == "s8" else 0  # the values that the codes stand for
        return {"bytes": read + T * c["heads"] * D * t + T * row + back, "flops": 3 * T * (c["heads"] + H) * c["rot"]}
    if c["op"] == "attend":
        n = sum(min(x, c["window"]) if c["window"] else x for x in lens)
        score = 8 * n * H if c["accumulate"] else 0
        return {"bytes": n * row + 2 * c["batch"] * c["heads"] * D * SIZE[c["type"]] + score,
                "flops": 4 * n * c["heads"] * D}
    n = sum(min(x, c["budget"]) for x in lens)
    back = n * H * 2 * D * 2 if c["cache"] == "s8" else 0
    return {"bytes": 4 * sum(lens) * H + n * (2 * row + H * (2 * 4 + 4)) + back, "flops": 0}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _side(c):
    return max(2, int(round(c["tokens"] ** (1.0 / 3.0))))


def _pages(gen, lens, page, more=0):
    """A page table over shuffled pages, and the number of pages; entries without a page are -1."""
    need = [-(-n // page) for n in lens]
    width = max(1, max(need))
    order = torch.randperm(sum(need) + more, generator=gen, device=DEV).to(torch.int32)
    first = torch.tensor(need).cumsum(0) - torch.tensor(need)
    at = first[:, None] + torch.arange(width)[None, :]
    have = (torch.arange(width)[None, :] < torch.tensor(need)[:, None]).to(DEV)
    table = torch.where(have, order[at.to(DEV).clamp(max=max(0, order.numel() - 1))] if order.numel() else -1, -1)
    return table.to(torch.int32).contiguous(), max(1, order.numel()), order[sum(need):]


def _cache(gen, c, pages):
    """Pages of keys and values as a model leaves them: a few head channels larger than the others."""
    shape = (pages, c["kv_heads"], c["page"], c["dim"])
    s = {}
    for name in ("k", "v"):
        x = torch.randn(shape, generator=gen, device=DEV, dtype=torch.bfloat16)
        if c["cache"] == "s8":
            s[name] = (x * 36.0).round().clamp(-127, 127).to(torch.int8)
            s[name + "_scale"] = torch.rand(shape[:3], generator=gen, device=DEV) * 0.02 + 0.01
        else:
            s[name] = x
            s[name + "_scale"] = None
        del x
    s["score"] = torch.rand(shape[:3], generator=gen, device=DEV) ** 4
    return s


def prepare(case, seed):
    c = case
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    lens, per = _lengths(c)
    s = {"case": c, "handle": None, "workspace": None}
    if c["op"] == "append":
        table, pages, _ = _pages(gen, lens, c["page"])
        s.update(_cache(gen, c, pages), table=table)
        seq = torch.repeat_interleave(torch.arange(c["batch"]), torch.tensor(per))
        start = torch.tensor([n - m for n, m in zip(lens, per)])
        first = torch.tensor(per).cumsum(0) - torch.tensor(per)
        index = torch.arange(c["tokens"]) - first[seq] + start[seq]
        s["seq"], s["index"] = seq.to(DEV, torch.int32), index.to(DEV, torch.int32)
        T, D, t = c["tokens"], c["dim"], TYPES[c["type"]]
        # q, k and v as the three parts of one projection's output
        width = (c["heads"] + 2 * c["kv_heads"]) * D
        qkv = (torch.randn((T, width), generator=gen, device=DEV)).to(t).view(T, -1, D)
        s["q"], s["k_new"], s["v_new"] = qkv.split((c["heads"], c["kv_heads"], c["kv_heads"]), 1)
        s["q_out"] = torch.empty((T, c["heads"], D), dtype=t, device=DEV)
        pairs = c["rot"] // 2
        if c["axes"] == 1:
            s["positions"], rows = s["index"].view(1, T).contiguous(), max(lens) + 1
        else:  # a grid of time, height and width, or of height and width
            side, i = _side(c), torch.arange(T, device=DEV)
            p = torch.stack((i // (side * side), i // side % side, i % side))[-c["axes"]:]
            s["positions"], rows = p.to(torch.int32).contiguous(), int(p.max()) + 1
        turn = torch.arange(rows, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(pairs) / pairs)
        s["cos"], s["sin"] = turn.cos().float().to(DEV), turn.sin().float().to(DEV)
        s["pair_axis"] = [j * c["axes"] // pairs for j in range(pairs)]
        if c["cache"] == "s8":
            s["k_back"] = torch.empty((T, c["kv_heads"], D), dtype=torch.bfloat16, device=DEV)
            s["v_back"] = torch.empty_like(s["k_back"])
        return s
    if c["op"] == "attend":
        table, pages, _ = _pages(gen, lens, c["page"])
        s.update(_cache(gen, c, pages), table=table)
        n = torch.tensor(lens, device=DEV)
        s["lengths"] = n.to(torch.int32)
        t = TYPES[c["type"]]
        s["q"] = (torch.randn((c["batch"], c["heads"], c["dim"]), generator=gen, device=DEV) * 3.0).to(t)
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty((c["batch"], c["heads"]), device=DEV)
        # what an earlier owner of the last page left behind its new owner's last token
        last = ((n - 1).clamp(min=0) // c["page"]).long()
        tail = table.gather(1, last[:, None])[:, 0][n > 0].long()
        used = ((n - 1) % c["page"] + 1)[n > 0]
        stale = torch.arange(c["page"], device=DEV)[None, None, :] >= used[:, None, None]
        for name in ("k", "v"):
            at = name + "_scale" if c["cache"] == "s8" else name
            m = stale if c["cache"] == "s8" else stale[..., None]
            s[at][tail] = torch.where(m, torch.tensor(float("nan"), device=DEV, dtype=s[at].dtype), s[at][tail])
        return s
    keep = [min(n, c["budget"]) for n in lens]
    more = sum(-(-n // c["page"]) for n in keep)
    table, pages, free = _pages(gen, lens, c["page"], more)
    s.update(_cache(gen, c, pages), table=table)
    need = torch.tensor([-(-n // c["page"]) for n in keep])
    width = max(1, int(need.max()))
    at = (need.cumsum(0) - need)[:, None] + torch.arange(width)[None, :]
    have = (torch.arange(width)[None, :] < need[:, None]).to(DEV)
    s["new_table"] = torch.where(have, free[at.clamp(max=more - 1).to(DEV)], -1).to(torch.int32).contiguous()
    s["lengths"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
    s["new_lengths"] = torch.empty_like(s["lengths"])
    s["kept"] = torch.empty((c["batch"], c["kv_heads"], c["budget"]), dtype=torch.int32, device=DEV)
    if c["cache"] == "s8":  # the kept tokens, for reading them back
        rows = torch.repeat_interleave(torch.arange(c["batch"]), torch.tensor(keep))
        first = torch.tensor(keep).cumsum(0) - torch.tensor(keep)
        s["seq"] = rows.to(DEV, torch.int32)
        s["index"] = (torch.arange(rows.numel()) - first[rows]).to(DEV, torch.int32)
        s["k_back"] = torch.empty((rows.numel(), c["kv_heads"], c["dim"]), dtype=torch.bfloat16, device=DEV)
        s["v_back"] = torch.empty_like(s["k_back"])
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _plain_rotate(x, cos, sin, interleaved):
    r = cos.shape[-1]
    y = x.float().clone()
    a, b = (slice(0, 2 * r, 2), slice(1, 2 * r, 2)) if interleaved else (slice(0, r), slice(r, 2 * r))
    x1, x2 = y[..., a].clone(), y[..., b].clone()
    y[..., a] = x1 * cos - x2 * sin
    y[..., b] = x2 * cos + x1 * sin
    return y


def _plain_quantize(y):
    scale = y.abs().amax(-1, keepdim=True)
    scale = scale / torch.full_like(scale, 127.0)  # a quotient: torch multiplies by a constant's reciprocal
    scale = torch.where(scale == 0, torch.ones_like(scale), scale)
    return (y / scale).round().clamp(-128, 127).to(torch.int8), scale[..., 0]


def _plain_read(s, page, off):
    """Keys and values of tokens (page, off), as bf16."""
    k = s["k"][page, :, off].float() * s["k_scale"][page, :, off][..., None]
    v = s["v"][page, :, off].float() * s["v_scale"][page, :, off][..., None]
    return k.to(torch.bfloat16), v.to(torch.bfloat16)


def _plain_append(s):
    c = s["case"]
    pairs = c["rot"] // 2
    axis = torch.tensor(s["pair_axis"], device=DEV)
    pos = s["positions"][axis].t().long()
    j = torch.arange(pairs, device=DEV)
    cos, sin = s["cos"][pos, j][:, None], s["sin"][pos, j][:, None]
    seq, index = s["seq"].long(), s["index"].long()
    page, off = s["table"][seq, index // c["page"]].long(), index % c["page"]
    q = _plain_rotate(s["q"], cos, sin, c["interleaved"]).to(s["q"].dtype)
    k, v = _plain_rotate(s["k_new"], cos, sin, c["interleaved"]), s["v_new"].float()
    s["score"][page, :, off] = 0.0
    if c["cache"] != "s8":
        s["k"][page, :, off], s["v"][page, :, off] = k.to(torch.bfloat16), v.to(torch.bfloat16)
        return {"q": q, "k": s["k"], "v": s["v"], "score": s["score"]}
    s["k"][page, :, off], s["k_scale"][page, :, off] = _plain_quantize(k)
    s["v"][page, :, off], s["v_scale"][page, :, off] = _plain_quantize(v)
    k, v = _plain_read(s, page, off)
    return {"q": q, "k": k, "v": v, "k_scale": s["k_scale"], "v_scale": s["v_scale"], "score": s["score"]}


def _plain_attend(s):
    c = s["case"]
    B, H, D, page = c["batch"], c["kv_heads"], c["dim"], c["page"]
    G = c["heads"] // H
    table = s["table"].long().clamp(min=0)
    n = table.shape[1] * page
    t = torch.arange(n, device=DEV)
    lens = s["lengths"].long()[:, None]
    valid = t < lens
    if c["window"]:
        valid = valid & (t >= lens - c["window"])

    def dense(name):
        x = s[name][table].float()  # [B, pages, H, page, D]
        if c["cache"] == "s8":
            x = x * s[name + "_scale"][table][..., None]
        x = x.permute(0, 2, 1, 3, 4).reshape(B, H, n, D)
        return torch.where(valid[:, None, :, None], x, torch.zeros((), device=DEV))

    q = s["q"].float().view(B, H, G, D) * (1.0 / math.sqrt(D))
    logit = torch.matmul(q, dense("k").transpose(-1, -2))
    logit = torch.where(valid[:, None, None, :], logit, torch.full((), -math.inf, device=DEV))
    top = logit.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    p = torch.exp(logit - top)
    total = p.sum(-1, keepdim=True)
    p = p / torch.where(total == 0, torch.ones_like(total), total)
    out = torch.matmul(p, dense("v")).reshape(B, c["heads"], D).to(s["q"].dtype)
    lse = (top + torch.log(total)).reshape(B, c["heads"])
    if not c["accumulate"]:
        return {"out": out, "lse": lse}
    b, i = torch.nonzero(valid, as_tuple=True)
    s["score"][table[b, i // page], :, i % page] += p.sum(2)[b, :, i]
    return {"out": out, "lse": lse, "score": s["score"]}


def _plain_evict(s):
    c = s["case"]
    B, H, page = c["batch"], c["kv_heads"], c["page"]
    table = s["table"].long().clamp(min=0)
    n = table.shape[1] * page
    score = s["score"][table].permute(0, 2, 1, 3).reshape(B, H, n)
    score = torch.where(torch.isnan(score), torch.full((), -math.inf, device=DEV), score)
    t, lens = torch.arange(n, device=DEV), s["lengths"].long()[:, None]
    sure = (t < c["sink"]) | (t >= lens - c["recent"])
    rank = torch.where(t < lens, torch.where(sure, 0, 1), 2)[:, None].expand(B, H, n)
    order = torch.sort(score, dim=-1, descending=True, stable=True).indices
    order = order.gather(-1, torch.sort(rank.gather(-1, order), dim=-1, stable=True).indices)
    keep = lens.clamp(max=c["budget"])
    j = torch.arange(c["budget"], device=DEV)
    kept = torch.full((B, H, c["budget"]), n, device=DEV)
    m = min(n, c["budget"])
    kept[..., :m] = torch.where((j < keep)[:, None, :m], order[..., :m], n)
    kept = kept.sort(-1).values
    kept = torch.where(kept == n, -1, kept)
    b, h, i = torch.nonzero(kept >= 0, as_tuple=True)
    src = kept[b, h, i]
    new = s["new_table"].long()[b, i // page], h, i % page
    old = table[b, src // page], h, src % page
    s["k"][new], s["v"][new], s["score"][new] = s["k"][old], s["v"][old], s["score"][old]
    out = {"kept": kept.to(torch.int32), "lengths": keep[:, 0].to(torch.int32), "score": s["score"]}
    if c["cache"] != "s8":
        return {**out, "k": s["k"], "v": s["v"]}
    s["k_scale"][new], s["v_scale"][new] = s["k_scale"][old], s["v_scale"][old]
    seq, index = s["seq"].long(), s["index"].long()
    k, v = _plain_read(s, s["new_table"].long()[seq, index // page], index % page)
    return {**out, "k": k, "v": v, "k_scale": s["k_scale"], "v_scale": s["v_scale"]}


# ---------------------------------------------------------------------------
# the library's calls
# ---------------------------------------------------------------------------
def _own(s):
    import int8_quantized_gb300 as lib

    c = s["case"]
    if s["handle"] is None:  # what a serving program keeps next to its cache
        s["handle"] = lib.KVCache(s["k"], s["v"], s["k_scale"], s["v_scale"], s["score"])
    cache = s["handle"]
    if c["op"] == "append":
        lib.kv_append(cache, s["table"], s["seq"], s["index"], s["k_new"], s["v_new"], q=s["q"], q_out=s["q_out"],
                      positions=s["positions"], cos=s["cos"], sin=s["sin"], pair_axis=s["pair_axis"],
                      interleaved=c["interleaved"])
        if c["cache"] != "s8":
            return {"q": s["q_out"], "k": s["k"], "v": s["v"], "score": s["score"]}
        lib.kv_gather(cache, s["table"], s["seq"], s["index"], s["k_back"], s["v_back"])
        return {"q": s["q_out"], "k": s["k_back"], "v": s["v_back"], "k_scale": s["k_scale"],
                "v_scale": s["v_scale"], "score": s["score"]}
    if c["op"] == "attend":
        if s["workspace"] is None:
            size = lib.paged_attention_workspace_size(cache, s["table"], c["heads"], c["accumulate"])
            s["workspace"] = torch.empty(size, dtype=torch.uint8, device=DEV)
        lib.paged_attention(cache, s["table"], s["lengths"], s["q"], s["out"], lse=s["lse"], window=c["window"],
                            accumulate=c["accumulate"], workspace=s["workspace"])
        out = {"out": s["out"], "lse": s["lse"]}
        return {**out, "score": s["score"]} if c["accumulate"] else out
    lib.kv_evict(cache, s["table"], s["lengths"], s["new_table"], s["kept"], s["new_lengths"], sink=c["sink"],
                 recent=c["recent"])
    out = {"kept": s["kept"], "lengths": s["new_lengths"], "score": s["score"]}
    if c["cache"] != "s8":
        return {**out, "k": s["k"], "v": s["v"]}
    lib.kv_gather(cache, s["new_table"], s["seq"], s["index"], s["k_back"], s["v_back"])
    return {**out, "k": s["k_back"], "v": s["v_back"], "k_scale": s["k_scale"], "v_scale": s["v_scale"]}


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    return _plain_append(state) if op == "append" else _plain_attend(state) if op == "attend" else _plain_evict(state)


# ---------------------------------------------------------------------------
# the definitions in 64 bits, a sequence or a token row at a time
# ---------------------------------------------------------------------------
def exact(case, seed):
    c, s = case, prepare(case, seed)
    page = c["page"]
    table = s["table"].cpu().numpy()

    def slots(row, index):
        return torch.from_numpy(row[index // page].astype(np.int64)).to(DEV), torch.from_numpy(index % page).to(DEV)

    if c["op"] == "append":
        pairs = c["rot"] // 2
        seq, index = s["seq"].cpu().numpy(), s["index"].cpu().numpy().astype(np.int64)
        pg = torch.from_numpy(table[seq, index // page].astype(np.int64)).to(DEV)
        off = torch.from_numpy(index % page).to(DEV)
        cos = torch.stack([s["cos"].double()[s["positions"][a].long(), j] for j, a in enumerate(s["pair_axis"])], -1)
        sin = torch.stack([s["sin"].double()[s["positions"][a].long(), j] for j, a in enumerate(s["pair_axis"])], -1)

        def turned(x):  # complex numbers times e^(i angle)
            x = x.double()
            head, rest = x[..., :c["rot"]], x[..., c["rot"]:]
            z = torch.complex(head[..., ::2], head[..., 1::2]) if c["interleaved"] else torch.complex(
                head[..., :pairs], head[..., pairs:])
            z = z * torch.complex(cos, sin)[:, None]
            y = torch.view_as_real(z)
            y = y.flatten(-2) if c["interleaved"] else torch.cat((y[..., 0], y[..., 1]), -1)
            return torch.cat((y, rest), -1)

        def stored(x):
            scale = x.abs().max(-1).values / 127.0
            scale[scale == 0] = 1.0
            return (x / scale[..., None]).round() * scale[..., None], scale

        k, v = turned(s["k_new"]), s["v_new"].double()
        score = s["score"].double()
        score[pg, :, off] = 0.0
        if c["cache"] != "s8":
            pk, pv = s["k"].double(), s["v"].double()
            pk[pg, :, off], pv[pg, :, off] = k, v
            return {"q": turned(s["q"]), "k": pk, "v": pv, "score": score}
        (k, ks), (v, vs) = stored(k), stored(v)
        pks, pvs = s["k_scale"].double(), s["v_scale"].double()
        pks[pg, :, off], pvs[pg, :, off] = ks, vs
        return {"q": turned(s["q"]), "k": k, "v": v, "k_scale": pks, "v_scale": pvs, "score": score}

    lens = s["lengths"].tolist()
    if c["op"] == "attend":
        G = c["heads"] // c["kv_heads"]
        out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
        lse = torch.full(s["lse"].shape, -math.inf, dtype=torch.float64, device=DEV)
        score = s["score"].double()
        for b, n in enumerate(lens):
            index = np.arange(max(0, n - c["window"]) if c["window"] else 0, n)
            if not index.size:
                continue
            pg, off = slots(table[b], index)
            k, v = s["k"][pg, :, off].double(), s["v"][pg, :, off].double()  # [n, H, D]
            if c["cache"] == "s8":
                k *= s["k_scale"][pg, :, off].double()[..., None]
                v *= s["v_scale"][pg, :, off].double()[..., None]
            q = s["q"][b].double().view(c["kv_heads"], G, c["dim"])
            x = torch.einsum("hgd,nhd->hgn", q, k) / math.sqrt(c["dim"])
            z = torch.logsumexp(x, -1)
            p = torch.exp(x - z[..., None])
            out[b] = torch.einsum("hgn,nhd->hgd", p, v).reshape(c["heads"], c["dim"])
            lse[b] = z.reshape(-1)
            score[pg, :, off] += p.sum(1).t()
        return {"out": out, "lse": lse, "score": score} if c["accumulate"] else {"out": out, "lse": lse}

    new = s["new_table"].cpu().numpy()
    score = s["score"].double()
    moved = {name: s[name].double() for name in ("k", "v")} if c["cache"] != "s8" else {}
    scales = {name: s[name].double() for name in ("k_scale", "v_scale")} if c["cache"] == "s8" else {}
    back = {name: [] for name in ("k", "v")}
    for b, n in enumerate(lens):
        pg, off = slots(table[b], np.arange(n))
        x = s["score"][pg, :, off].double().cpu().numpy()  # [n, H]
        m = min(n, c["budget"])
        mid = np.arange(c["sink"], max(c["sink"], n - c["recent"]))
        kept = []
        for h in range(c["kv_heads"]):
            if m == n:
                kept.append(np.arange(n))
                continue
            best = mid[np.lexsort((mid, -x[mid, h]))][:m - c["sink"] - c["recent"]]
            kept.append(np.sort(np.concatenate((np.arange(c["sink"]), best, np.arange(n - c["recent"], n)))))
        kept = torch.from_numpy(np.stack(kept, 1)).to(DEV)  # [m, H]
        h = torch.arange(c["kv_heads"], device=DEV)[None, :]
        npg, noff = slots(new[b], np.arange(m))
        old, to = (pg[kept], h, off[kept]), (npg[:, None], h, noff[:, None])
        score[to] = s["score"][old].double()
        for name in moved:
            moved[name][to] = s[name][old].double()
        for name in scales:
            scales[name][to] = s[name][old].double()
        if c["cache"] == "s8":
            for name in back:
                back[name].append(s[name][old].double() * s[name + "_scale"][old].double()[..., None])
    out = {"kept": None, "lengths": None, "score": score}
    if c["cache"] != "s8":
        return {**out, **moved}
    return {**out, **{name: torch.cat(x) for name, x in back.items()}, **scales}
