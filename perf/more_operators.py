"""Performance cases of the operators that complete a decode step.

  nbits   products of a few rows with 4-bit weights, a scale and a zero point per block (MatMulNBits)
  append  each head of q and k normalized by its root mean square, turned to its position, and k and v written into
          their pages, in one call
  sample  the next token from a row of logits: temperature, top-k, top-p, min-p and a given random number

`own` selects between the library's calls and a plain form in elementary torch operations: in fp32, in fp64 where a
rounding decides a whole number (the sampled token, an int8 code).
"""
import math
import random

import torch

own = False

DEV = "cuda"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "s8": torch.int8}
SIZE = {"f32": 4, "bf16": 2, "s8": 1}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _nbits(rows, n, k, block, type, scales="bf16", zero=True, bias=False):
    return {"op": "nbits", "rows": rows, "n": n, "k": k, "block": block, "type": type, "scales": scales, "zero": zero,
            "bias": bias}


def _append(tokens, batch, heads, kv_heads, dim, page, rot, axes, type, cache, interleaved=False, weights="f32", mix=1):
    return {"op": "append", "tokens": tokens, "batch": batch, "heads": heads, "kv_heads": kv_heads, "dim": dim,
            "page": page, "rot": rot, "axes": axes, "type": type, "cache": cache, "interleaved": interleaved,
            "weights": weights, "mix": mix}


def _sample(rows, vocab, type, top_k=0, top_p=1.0, min_p=0.0, temperature=1.0, spread=3.0, masked=0.0, greedy=0.0,
            empty=False):
    return {"op": "sample", "rows": rows, "vocab": vocab, "type": type, "top_k": top_k, "top_p": top_p, "min_p": min_p,
            "temperature": temperature, "spread": spread, "masked": masked, "greedy": greedy, "empty": empty}


def listed():
    return [
        # one token through a small layer: the call is all latency
        {"name": "nbits 1 x 1024 x 1024", **_nbits(1, 1024, 1024, 32, "bf16")},
        # one token through a feed-forward layer's first product
        {"name": "nbits 1 x 4096 -> 14336", **_nbits(1, 14336, 4096, 128, "bf16", zero=False)},
        # eight sequences through its second product, with the smallest common blocks and their zero points
        {"name": "nbits 8 x 14336 -> 4096", **_nbits(8, 4096, 14336, 32, "bf16")},
        # odd sizes, fp32 activations, a part full last block
        {"name": "nbits 5 x 1999 -> 1001 fp32", **_nbits(5, 1001, 1999, 16, "f32", "f32", True, True)},
        # a full decode batch
        {"name": "nbits 64 x 4096 -> 14336", **_nbits(64, 14336, 4096, 64, "bf16")},
        # one token's logits over a large vocabulary
        {"name": "nbits 1 x 4096 -> 128000", **_nbits(1, 128000, 4096, 64, "bf16")},
        # one user, one new token
        {"name": "append normed 1 token", **_append(1, 1, 32, 8, 128, 16, 128, 1, "bf16", "s8")},
        # a decode batch with fp32 activations, half of each head turned, unquantized pages
        {"name": "append normed 96 x 1 fp32", **_append(96, 96, 12, 12, 64, 24, 32, 1, "f32", "bf16", True)},
        # the prompt of an image or video question: time, height and width positions
        {"name": "append normed prompt 16384", **_append(16384, 4, 32, 8, 128, 32, 128, 3, "bf16", "bf16", False, "bf16")},
        # one answer token, the usual top-p
        {"name": "sample 1 x 32000", **_sample(1, 32000, "bf16", top_p=0.9, temperature=0.8)},
        # an ordinary batch with every filter, greedy rows and masked tokens (a grammar's) among them
        {"name": "sample 32 x 50001 fp32",
         **_sample(32, 50001, "f32", 50, 0.95, 0.02, 0.7, 3.0, 0.5, 0.1, True)},
        # the largest batch over a large vocabulary, nearly all of it kept
        {"name": "sample 128 x 128000", **_sample(128, 128000, "bf16", 0, 0.98, 0.0, 1.0, 1.5)},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("nbits", "append", "sample"))
    type = rng.choice(("bf16", "bf16", "f32"))
    if op == "nbits":
        block = rng.choice((16, 32, 32, 64, 128, 128, 256))
        k = _log(rng, 32, 16384)
        if rng.random() < 0.5:
            k = max(block, k // block * block)
        n = _log(rng, 16, max(16, min(128000, (1 << 28) // k)))
        return _nbits(_log(rng, 1, 64), n, k, block, type, rng.choice(("f32", "bf16")), rng.random() < 0.6,
                      rng.random() < 0.3)
    if op == "append":
        dim, kv_heads, group = rng.choice((64, 80, 96, 128, 128, 192, 256)), rng.choice((1, 2, 4, 8, 8, 16)), rng.choice(
            (1, 2, 4, 4, 7, 8, 16))
        cache = rng.choice(("s8", "bf16"))
        most = max(1, min(16384, (1 << 28) // ((group + 2) * kv_heads * dim * SIZE[type])))
        tokens = _log(rng, 1, most)
        return _append(tokens, rng.randint(1, min(tokens, 64)), kv_heads * group, kv_heads, dim,
                       rng.choice((8, 16, 16, 24, 32, 64, 128)), rng.choice((0, dim, dim, dim // 2)),
                       rng.choice((1, 2, 3)), type, cache, rng.random() < 0.5, rng.choice(("f32", "bf16")),
                       rng.randrange(1 << 20))
    vocab = _log(rng, 100, 200000)
    rows = _log(rng, 1, max(1, min(256, (1 << 24) // vocab)))
    return _sample(rows, vocab, type, rng.choice((0, 0, 1, 50, rng.randint(1, vocab))),
                   rng.choice((1.0, 0.9, rng.uniform(0.05, 0.999))), rng.choice((0.0, 0.0, rng.uniform(0.001, 0.5))),
                   rng.uniform(0.2, 2.0), rng.uniform(0.5, 5.0), rng.choice((0.0, 0.0, 0.9)), rng.choice((0.0, 0.1)),
                   rng.random() < 0.3)


def work(c):
    t = SIZE[c["type"]]
    if c["op"] == "nbits":
        n, k, m, blocks = c["n"], c["k"], c["rows"], -(-c["k"] // c["block"])
        weights = n * (k / 2 + blocks * (SIZE[c["scales"]] + (0.5 if c["zero"] else 0)) + (4 if c["bias"] else 0))
        return {"bytes": int(weights + m * (n + k) * t), "flops": 2 * m * n * k}
    if c["op"] == "sample":
        return {"bytes": c["rows"] * (c["vocab"] * t + 28), "flops": 40 * c["rows"] * c["vocab"]}
    T, D, H = c["tokens"], c["dim"], c["kv_heads"]
    rows = T if c["axes"] == 1 else min(T, _side(c) * 4)
    page = H * (2 * D * SIZE[c["cache"]] + (8 if c["cache"] == "s8" else 0))
    read = T * (c["heads"] + 2 * H) * D * t + rows * c["rot"] * 4
    back = T * H * 2 * D * 2 if c["cache"] == "s8" else 0  # the values that the codes stand for
    return {"bytes": read + T * (c["heads"] * D * t + page) + back, "flops": (3 * c["rot"] + 4 * D) * T * (c["heads"] + H)}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _side(c):
    return max(2, int(round(c["tokens"] ** (1.0 / 3.0))))


def _prepare_nbits(c, gen, s):
    n, k, m, block = c["n"], c["k"], c["rows"], c["block"]
    blocks = -(-k // block)
    s["B"] = torch.randint(0, 256, (n, blocks, block // 2), generator=gen, device=DEV, dtype=torch.uint8)
    x = torch.rand((n, blocks), generator=gen, device=DEV) + 0.5
    s["scales"] = (x * (0.3 / math.sqrt(k))).to(TYPES[c["scales"]])
    s["zero"] = None
    if c["zero"]:  # two to a byte; near the middle of the codes, as weights give them
        z = torch.randint(5, 11, (n, blocks + blocks % 2), generator=gen, device=DEV, dtype=torch.uint8)
        s["zero"] = (z[:, ::2] | z[:, 1::2] << 4).contiguous()
    s["bias"] = torch.randn((n,), generator=gen, device=DEV) * 0.1 if c["bias"] else None
    a = torch.randn((m, k), generator=gen, device=DEV)
    a[:, torch.randint(0, k, (max(1, k // 500),), generator=gen, device=DEV)] *= 20.0  # a few large channels
    s["A"] = a.to(TYPES[c["type"]])
    s["Y"] = torch.empty((m, n), dtype=TYPES[c["type"]], device=DEV)


def _prepare_sample(c, gen, s):
    R, V = c["rows"], c["vocab"]
    x = torch.randn((R, V), generator=gen, device=DEV) * c["spread"]
    if c["masked"]:
        x = torch.where(torch.rand((R, V), generator=gen, device=DEV) < c["masked"], -math.inf, x)
    if c["empty"]:
        x[R // 2] = -math.inf
    s["logits"] = x.to(TYPES[c["type"]])
    s["u"] = torch.rand((R,), generator=gen, device=DEV)
    one = torch.ones((R,), device=DEV)
    # every request brings its own settings
    vary = torch.rand((R,), generator=gen, device=DEV)
    s["temperature"] = c["temperature"] * (0.8 + 0.4 * vary)
    if c["greedy"]:
        s["temperature"] = torch.where(torch.rand((R,), generator=gen, device=DEV) < c["greedy"], 0.0, s["temperature"])
    s["top_k"] = s["top_p"] = s["min_p"] = None
    if c["top_k"]:
        s["top_k"] = (one * c["top_k"] * (0.5 + 0.5 * vary)).ceil().to(torch.int32)
    if c["top_p"] < 1:
        s["top_p"] = one * c["top_p"]
    if c["min_p"]:
        s["min_p"] = one * c["min_p"]
    s["tokens"] = torch.empty((R,), dtype=torch.int32, device=DEV)
    s["logprobs"] = torch.empty((R,), device=DEV)


def _prepare_append(c, gen, s):
    r = random.Random(c["mix"])
    T, B, D, H, page = c["tokens"], c["batch"], c["dim"], c["kv_heads"], c["page"]
    per = [T // B + (b < T % B) for b in range(B)]
    lens = [r.randint(0, 500) + n for n in per]
    need = [-(-n // page) for n in lens]
    order = torch.randperm(sum(need), generator=gen, device=DEV).to(torch.int32)
    first = torch.tensor(need).cumsum(0) - torch.tensor(need)
    at = first[:, None] + torch.arange(max(need))[None, :]
    have = (torch.arange(max(need))[None, :] < torch.tensor(need)[:, None]).to(DEV)
    s["table"] = torch.where(have, order[at.to(DEV).clamp(max=sum(need) - 1)], -1).to(torch.int32).contiguous()
    shape = (sum(need), H, page, D)
    for name in ("k", "v"):
        x = torch.randn(shape, generator=gen, device=DEV, dtype=torch.bfloat16)
        s[name], s[name + "_scale"] = x, None
        if c["cache"] == "s8":
            s[name] = (x * 36.0).round().clamp(-127, 127).to(torch.int8)
            s[name + "_scale"] = torch.rand(shape[:3], generator=gen, device=DEV) * 0.02 + 0.01
    seq = torch.repeat_interleave(torch.arange(B), torch.tensor(per))
    start = torch.tensor([n - m for n, m in zip(lens, per)])
    index = torch.arange(T) - (torch.tensor(per).cumsum(0) - torch.tensor(per))[seq] + start[seq]
    s["seq"], s["index"] = seq.to(DEV, torch.int32), index.to(DEV, torch.int32)
    t = TYPES[c["type"]]
    # q, k and v as the three parts of one projection's output, of a size that differs between tokens
    qkv = torch.randn((T, (c["heads"] + 2 * H) * D), generator=gen, device=DEV)
    qkv = (qkv * (torch.rand((T, 1), generator=gen, device=DEV) * 4.0 + 0.1)).to(t).view(T, -1, D)
    s["q"], s["k_new"], s["v_new"] = qkv.split((c["heads"], H, H), 1)
    s["q_out"] = torch.empty((T, c["heads"], D), dtype=t, device=DEV)
    for name in ("q_norm", "k_norm"):
        s[name] = (torch.randn((D,), generator=gen, device=DEV) * 0.2 + 1.0).to(TYPES[c["weights"]])
    s["positions"] = s["cos"] = s["sin"] = s["pair_axis"] = None
    pairs = c["rot"] // 2
    if pairs:
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
        s["k_back"] = torch.empty((T, H, D), dtype=torch.bfloat16, device=DEV)
        s["v_back"] = torch.empty_like(s["k_back"])


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    s = {"case": case, "handle": None, "eps": 1e-6}
    {"nbits": _prepare_nbits, "append": _prepare_append, "sample": _prepare_sample}[case["op"]](case, gen, s)
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _plain_nbits(s):
    c = s["case"]
    n, k, block = c["n"], c["k"], c["block"]
    codes = torch.stack((s["B"] & 15, s["B"] >> 4), -1).view(n, -1, block).float()
    zero = 8.0
    if s["zero"] is not None:
        z = torch.stack((s["zero"] & 15, s["zero"] >> 4), -1).view(n, -1)
        zero = z[:, :codes.shape[1], None].float()
    w = ((codes - zero) * s["scales"].float()[:, :, None]).view(n, -1)[:, :k]
    y = torch.matmul(s["A"].float(), w.t())
    if s["bias"] is not None:
        y = y + s["bias"]
    return {"Y": y.to(s["A"].dtype)}


def _plain_norm(x, weight, eps):
    """Each operation rounded once to fp32; the sum of squares in fp64."""
    x = x.float()
    mean = (x.double().square().sum(-1, keepdim=True) / x.shape[-1]).float()
    root = torch.sqrt(mean + eps)
    return x * (torch.ones_like(root) / root) * weight.float()


def _plain_rotate(y, s):
    c = s["case"]
    if s["cos"] is None:
        return y
    pairs = c["rot"] // 2
    pos = s["positions"][torch.tensor(s["pair_axis"], device=DEV)].t().long()
    j = torch.arange(pairs, device=DEV)
    cos, sin = s["cos"][pos, j][:, None], s["sin"][pos, j][:, None]
    a, b = (slice(0, 2 * pairs, 2), slice(1, 2 * pairs, 2)) if c["interleaved"] else (slice(0, pairs),
                                                                                      slice(pairs, 2 * pairs))
    x1, x2 = y[..., a].clone(), y[..., b].clone()
    y = y.clone()
    y[..., a] = x1 * cos - x2 * sin
    y[..., b] = x2 * cos + x1 * sin
    return y


def _plain_quantize(y):
    scale = y.abs().amax(-1, keepdim=True)
    scale = scale / torch.full_like(scale, 127.0)  # a quotient: torch multiplies by a constant's reciprocal
    scale = torch.where(scale == 0, torch.ones_like(scale), scale)
    return (y / scale).round().clamp(-128, 127).to(torch.int8), scale[..., 0]


def _plain_append(s):
    c = s["case"]
    seq, index = s["seq"].long(), s["index"].long()
    page, off = s["table"][seq, index // c["page"]].long(), index % c["page"]
    q = _plain_rotate(_plain_norm(s["q"], s["q_norm"], s["eps"]), s).to(s["q"].dtype)
    k, v = _plain_rotate(_plain_norm(s["k_new"], s["k_norm"], s["eps"]), s), s["v_new"].float()
    if c["cache"] != "s8":
        s["k"][page, :, off], s["v"][page, :, off] = k.to(torch.bfloat16), v.to(torch.bfloat16)
        return {"q": q, "k": s["k"], "v": s["v"]}
    s["k"][page, :, off], s["k_scale"][page, :, off] = _plain_quantize(k)
    s["v"][page, :, off], s["v_scale"][page, :, off] = _plain_quantize(v)
    back = [(s[x][page, :, off].float() * s[x + "_scale"][page, :, off][..., None]).to(torch.bfloat16) for x in "kv"]
    return {"q": q, "k": back[0], "v": back[1], "k_scale": s["k_scale"], "v_scale": s["v_scale"]}


def _plain_sample(s):
    x = s["logits"].double()
    R, V = x.shape
    one = torch.ones((R, 1), dtype=torch.float64, device=DEV)
    T = s["temperature"].double()[:, None]
    value, order = torch.sort(x, dim=-1, descending=True, stable=True)
    top = value[:, :1]
    w = torch.where(value == -math.inf, 0.0, torch.exp((value - top) / torch.where(T == 0, one, T)))
    rank = torch.arange(V, device=DEV)
    keep = value != -math.inf
    if s["top_k"] is not None:
        keep = keep & (rank < s["top_k"][:, None])
    sums = torch.cumsum(torch.where(keep, w, 0.0), -1)
    if s["top_p"] is not None:  # the tokens before which the sum has not been reached
        keep = keep & (sums - w < s["top_p"].double()[:, None] * sums[:, -1:])
    if s["min_p"] is not None:
        keep = keep & (w >= s["min_p"].double()[:, None])
    keep = torch.where(T == 0, (rank == 0) & (top != -math.inf), keep | ((rank == 0) & (top != -math.inf)))
    kept = torch.zeros((R, V), dtype=torch.float64, device=DEV).scatter_(1, order, torch.where(keep, w, 0.0))
    sums = torch.cumsum(kept, -1)
    total = sums[:, -1:]
    token = (sums <= s["u"].double()[:, None] * total).sum(-1).clamp(max=V - 1)
    token = torch.where(total[:, 0] == 0, 0, token)
    weight = kept.gather(1, token[:, None])
    return {"tokens": torch.where(total[:, 0] == 0, -1, token).to(torch.int32),
            "logprobs": torch.where(total == 0, -math.inf, torch.log(weight / total))[:, 0].float()}


# ---------------------------------------------------------------------------
# the library's calls
# ---------------------------------------------------------------------------
def _own(s):
    import int8_quantized_gb300 as lib

    c = s["case"]
    if c["op"] == "nbits":
        if s["handle"] is None:  # a layer's weights, laid out once
            s["handle"] = lib.MatMulNBits(s["B"], s["scales"], c["k"], c["block"], zero_points=s["zero"], bias=s["bias"])
        return {"Y": s["handle"].forward(s["A"], s["Y"])}
    if c["op"] == "append":
        if s["handle"] is None:
            s["handle"] = lib.KVCache(s["k"], s["v"], s["k_scale"], s["v_scale"])
        lib.kv_append(s["handle"], s["table"], s["seq"], s["index"], s["k_new"], s["v_new"], q=s["q"], q_out=s["q_out"],
                      positions=s["positions"], cos=s["cos"], sin=s["sin"], pair_axis=s["pair_axis"],
                      interleaved=c["interleaved"], q_norm=s["q_norm"], k_norm=s["k_norm"], norm_eps=s["eps"])
        if c["cache"] != "s8":
            return {"q": s["q_out"], "k": s["k"], "v": s["v"]}
        lib.kv_gather(s["handle"], s["table"], s["seq"], s["index"], s["k_back"], s["v_back"])
        return {"q": s["q_out"], "k": s["k_back"], "v": s["v_back"], "k_scale": s["k_scale"], "v_scale": s["v_scale"]}
    lib.sample(s["logits"], s["u"], s["tokens"], logprobs=s["logprobs"], temperature=s["temperature"],
               top_k=s["top_k"], top_p=s["top_p"], min_p=s["min_p"])
    return {"tokens": s["tokens"], "logprobs": s["logprobs"]}


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    return _plain_nbits(state) if op == "nbits" else _plain_append(state) if op == "append" else _plain_sample(state)


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def _exact_nbits(c, s):
    n, k, block = c["n"], c["k"], c["block"]
    y = torch.zeros((c["rows"], n), dtype=torch.float64, device=DEV)
    A = s["A"].double()
    for b in range(-(-k // block)):  # block by block: the codes' products first, then the block's scale
        a = A[:, b * block:(b + 1) * block]
        q = torch.empty((n, block), dtype=torch.float64, device=DEV)
        q[:, 0::2], q[:, 1::2] = s["B"][:, b] % 16, s["B"][:, b] // 16
        z = 8.0 if s["zero"] is None else (s["zero"][:, b // 2] // (16 if b % 2 else 1) % 16).double()[:, None]
        y += (a @ (q - z)[:, :a.shape[1]].t()) * s["scales"][:, b].double()
    return {"Y": y if s["bias"] is None else y + s["bias"].double()}


def _exact_append(c, s):
    page, pairs = c["page"], c["rot"] // 2
    at = s["table"].cpu()[s["seq"].cpu().long(), s["index"].cpu().long() // page].to(DEV).long()
    off = s["index"].long() % page
    turn = None
    if pairs:
        cos = torch.stack([s["cos"].double()[s["positions"][a].long(), j] for j, a in enumerate(s["pair_axis"])], -1)
        sin = torch.stack([s["sin"].double()[s["positions"][a].long(), j] for j, a in enumerate(s["pair_axis"])], -1)
        turn = torch.complex(cos, sin)[:, None]

    def placed(x, weight):  # complex numbers times e^(i angle)
        x = x.double()
        x = x / ((x * x).mean(-1, keepdim=True) + s["eps"]).sqrt() * weight.double()
        if turn is None:
            return x
        head, rest = x[..., :c["rot"]], x[..., c["rot"]:]
        z = torch.complex(head[..., ::2], head[..., 1::2]) if c["interleaved"] else torch.complex(
            head[..., :pairs], head[..., pairs:])
        y = torch.view_as_real(z * turn)
        y = y.flatten(-2) if c["interleaved"] else torch.cat((y[..., 0], y[..., 1]), -1)
        return torch.cat((y, rest), -1)

    def stored(x):
        scale = x.abs().max(-1).values / 127.0
        scale[scale == 0] = 1.0
        return (x / scale[..., None]).round() * scale[..., None], scale

    q, k, v = placed(s["q"], s["q_norm"]), placed(s["k_new"], s["k_norm"]), s["v_new"].double()
    if c["cache"] != "s8":
        pk, pv = s["k"].double(), s["v"].double()
        pk[at, :, off], pv[at, :, off] = k, v
        return {"q": q, "k": pk, "v": pv}
    (k, ks), (v, vs) = stored(k), stored(v)
    pks, pvs = s["k_scale"].double(), s["v_scale"].double()
    pks[at, :, off], pvs[at, :, off] = ks, vs
    return {"q": q, "k": k, "v": v, "k_scale": pks, "v_scale": pvs}


def _exact_sample(c, s):
    tokens, logprobs = [], []
    pick = lambda name, r, off: off if s[name] is None else s[name][r].item()
    for r in range(c["rows"]):  # a row at a time, its tokens in groups of equal logits
        x, T = s["logits"][r].double(), s["temperature"][r].item()
        top = x.max().item()
        if top == -math.inf:
            tokens.append(-1), logprobs.append(-math.inf)
            continue
        if T == 0:
            tokens.append(int((x == top).nonzero()[0, 0])), logprobs.append(0.0)
            continue
        value, inverse, count = torch.unique(-x, return_inverse=True, return_counts=True)  # from the largest on
        weight = torch.exp((-value - top) / T) * (value != math.inf)
        count = count * (value != math.inf)
        k = pick("top_k", r, c["vocab"])
        before = count.cumsum(0) - count
        taken = (k - before).clamp(min=0).minimum(count)  # of each group, those among the first k
        mass = taken * weight
        want = pick("top_p", r, 1.0) * mass.sum()
        if s["top_p"] is not None:
            missing = want - (mass.cumsum(0) - mass)  # before each group
            taken = torch.where(weight > 0, (missing / weight).ceil().clamp(min=0).minimum(taken.double()), 0.0).long()
        taken = torch.where(weight >= pick("min_p", r, 0.0), taken, 0)
        taken[0] = max(1, int(taken[0]))
        # of a group, its first by index
        by = torch.sort(inverse, stable=True).indices
        place = torch.empty_like(by)
        place[by] = torch.arange(x.numel(), device=DEV) - before_all(inverse, by)
        w = torch.where(place < taken[inverse], weight[inverse], 0.0)
        sums = w.cumsum(0)
        token = int(torch.searchsorted(sums, s["u"][r].double() * sums[-1], right=True))
        tokens.append(token), logprobs.append(math.log(w[token].item() / sums[-1].item()))
    return {"tokens": torch.tensor(tokens, dtype=torch.int32, device=DEV),
            "logprobs": torch.tensor(logprobs, dtype=torch.float64, device=DEV)}


def before_all(inverse, by):
    """For each place of the sorted tokens, where its group begins."""
    g = inverse[by]
    start = torch.ones_like(g, dtype=torch.bool)
    start[1:] = g[1:] != g[:-1]
    at = torch.arange(g.numel(), device=DEV)
    return torch.where(start, at, 0).cummax(0).values


def exact(case, seed):
    s = prepare(case, seed)
    return {"nbits": _exact_nbits, "append": _exact_append, "sample": _exact_sample}[case["op"]](case, s)
