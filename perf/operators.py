"""Timed cases of the operators that stand between the quantized products of
a decode step: the residual addition with its RMS norm, the GEMV over
activations that the norm left in 8 bits, the store into a paged key-value
cache, the attention of one new token over that cache, and the routing of
tokens to experts.

`run` computes a case in plain torch operations (`own` false) or through the
public calls of dequant_quantized_gemv_amd.qk (`own` true); `exact` computes
it in 64 bits.
"""
import math

import torch

own = False

BLOCK_BYTES = {"q4_0": 18, "q4_1": 20, "q8_0": 34, "q5_0": 22, "q5_1": 24}
X8_BYTES = 36      # an 8-bit activation block: fp32 scale, 32 int8 codes
EPS = 1e-5


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------

def _norm(name, n, k, x, out):
    return {"name": name, "op": "norm", "n": n, "k": k, "x": x, "out": out}


def _gemv(name, fmt, m, k, n):
    return {"name": name, "op": "gemv", "fmt": fmt, "m": m, "k": k, "n": n}


def _store(name, kind, tokens, heads, dim, page, pages):
    return {"name": name, "op": "store", "kind": kind, "tokens": tokens, "heads": heads, "dim": dim,
            "page": page, "pages": pages}


def _attn(name, kind, seqs, most, ragged, q_heads, heads, dim, page, window=0, sinks=0, out="f32"):
    return {"name": name, "op": "attn", "kind": kind, "seqs": seqs, "most": most, "ragged": ragged,
            "q_heads": q_heads, "heads": heads, "dim": dim, "page": page, "window": window, "sinks": sinks,
            "out": out}


def _route(name, tokens, experts, used, score, bias, groups, kept, best):
    return {"name": name, "op": "route", "tokens": tokens, "experts": experts, "used": used, "score": score,
            "bias": bias, "groups": groups, "kept": kept, "best": best}


def listed():
    return [
        # one token's residual stream before a projection: the smallest call, all latency
        _norm("norm 1x4096", 1, 4096, "f32", "f32"),
        # a prompt's rows quantized for 8-bit products
        _norm("norm 2048x4096 x8", 2048, 4096, "f32", "x8"),
        # one token through an attention projection
        _gemv("gemv q4_0 4096x4096 n1", "q4_0", 4096, 4096, 1),
        # eight tokens through a feed-forward matrix
        _gemv("gemv q4_1 11008x4096 n8", "q4_1", 11008, 4096, 8),
        # one new token of each of 64 sequences
        _store("store f16 64", "f16", 64, 8, 128, 16, 4),
        # a prompt of 4000 tokens into 8-bit pages that it fills but for the last
        _store("store i8 4000", "i8", 4000, 8, 128, 16, 250),
        # one short conversation: latency
        _attn("attn f16 1x1000", "f16", 1, 1000, False, 32, 8, 128, 16),
        # a batch of 64 conversations of all lengths over an 8-bit cache
        _attn("attn i8 64x4096", "i8", 64, 4096, True, 32, 8, 128, 16),
        # one long document: few rows, a long axis
        _attn("attn f16 1x131072", "f16", 1, 131072, False, 32, 8, 128, 64),
        # every head with keys of its own, a window of 1024 and 4 first tokens, pages that end inside a tile
        _attn("attn f16 16x8000 w1024", "f16", 16, 8000, True, 32, 32, 64, 24, 1024, 4, "f16"),
        # one token, 8 of 128 experts
        _route("route 1x128", 1, 128, 8, "softmax", False, 1, 1, 1),
        # a prompt: biased sigmoid scores, the best 4 of 8 groups
        _route("route 4096x256 groups", 4096, 256, 8, "sigmoid", True, 8, 4, 2),
    ]


def _spread(rng, lo, hi):
    """A whole number of lo..hi, spread over its logarithm."""
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49))))))


def draw(rng):
    op = rng.choice(["norm", "gemv", "store", "attn", "attn", "route"])
    if op == "norm":
        out = rng.choice(["f32", "f16", "x8"])
        k = _spread(rng, 33, 16384)
        k = max(32, k // 32 * 32) if out == "x8" else k
        n = _spread(rng, 1, max(1, min(4096, 2048 * 4096 // k)))
        c = _norm("", n, k, rng.choice(["f32", "f16"]), out)
    elif op == "gemv":
        k = 32 * _spread(rng, 4, 344)
        c = _gemv("", rng.choice(sorted(BLOCK_BYTES)), _spread(rng, 17, 11008 * 4096 // max(k, 4096)), k,
                  rng.randint(1, 8))
    elif op == "store":
        page = rng.choice([1, 8, 16, 24, 32, 64, 100])
        tokens = _spread(rng, 1, 4000)
        heads, dim = rng.choice([1, 2, 3, 4, 8]), 32 * rng.randint(1, 8)
        tokens = max(1, min(tokens, 4000 * 8 * 128 // (heads * dim)))
        kind = rng.choice(["f16", "i8"])
        c = _store("", kind, tokens, heads, dim, page, -(-tokens // page) if kind == "i8" else 2)
    elif op == "attn":
        heads = rng.choice([1, 2, 4, 5, 8])
        group = rng.choice([1, 2, 3, 4, 6, 7, 8, 12, 16])
        dim = 32 * rng.choice([1, 2, 2, 3, 4, 4, 4, 5, 6, 8])
        seqs = _spread(rng, 1, 64)
        most = _spread(rng, 1, max(1, min(131072, 64 * 4096 * 8 * 128 // (2 * seqs * heads * dim))))
        window = rng.choice([0, 0, _spread(rng, 1, 4096)])
        c = _attn("", rng.choice(["f16", "i8"]), seqs, most, bool(seqs > 1 and rng.random() < 0.7), heads * group,
                  heads, dim, rng.choice([8, 16, 24, 32, 64, 128]), window,
                  rng.choice([0, 1, 4, 50]) if window else 0, rng.choice(["f32", "f16"]))
    else:
        groups = rng.choice([1, 1, 2, 4, 8])
        experts = groups * _spread(rng, max(2, 8 // groups), 512 // groups)
        kept = rng.randint(1, groups)
        used = rng.randint(1, min(16, kept * (experts // groups)))
        c = _route("", _spread(rng, 1, max(1, 4096 * 256 // experts)), experts, used,
                   rng.choice(["softmax", "sigmoid"]), rng.random() < 0.5, groups, kept, rng.choice([1, 2]))
    del c["name"]
    return c


def _lens(c):
    """Tokens in the cache of each sequence, before they are shuffled."""
    n, most = c["seqs"], c["most"]
    return [max(1, math.ceil(most * (i + 1) / n)) for i in range(n)] if c["ragged"] else [most] * n


def work(c):
    op = c["op"]
    if op == "norm":
        n, k, xb = c["n"], c["k"], {"f32": 4, "f16": 2}[c["x"]]
        yb = {"f32": 4.0, "f16": 2.0, "x8": X8_BYTES / 32}[c["out"]]
        return {"bytes": n * k * (3 * xb + yb) + 4 * k, "flops": 6 * n * k}
    if op == "gemv":
        m, k, n = c["m"], c["k"], c["n"]
        return {"bytes": m * (k // 32) * BLOCK_BYTES[c["fmt"]] + n * (k // 32) * X8_BYTES + 4 * n * m,
                "flops": 2 * m * k * n}
    if op == "store":
        one = c["heads"] * c["dim"] * (4 + (2 if c["kind"] == "f16" else 1)) + (4 * c["heads"] if c["kind"] == "i8" else 0)
        return {"bytes": 2 * c["tokens"] * one + 8 * c["tokens"], "flops": 4 * c["tokens"] * c["heads"] * c["dim"]}
    if op == "attn":
        w, s = c["window"], c["sinks"]
        seen = sum(n if not w else min(n, w) + min(s, max(0, n - w)) for n in _lens(c))
        row = c["dim"] * 2 if c["kind"] == "f16" else c["dim"] + 4
        io = c["seqs"] * c["q_heads"] * c["dim"] * (4 + (4 if c["out"] == "f32" else 2))
        return {"bytes": 2 * seen * c["heads"] * row + io + 4 * -(-seen // c["page"]),
                "flops": 4 * seen * c["q_heads"] * c["dim"]}
    t = c["tokens"]
    return {"bytes": t * (4 * c["experts"] + 8 * c["used"]) + (4 * c["experts"] if c["bias"] else 0),
            "flops": 8 * t * c["experts"]}


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------

def _gen(seed, device="cuda"):
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, device="cuda", generator=g)


def _pow2(e):
    """2^e as fp32 for whole e in -126..127."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _x8_codes(y):
    """Codes and scales of the 8-bit activation format (n, blocks, 32): the
    scale is the least power of two with 127 scales >= the block's largest
    magnitude, the codes round half to even."""
    b = y.view(y.shape[0], -1, 32)
    top = b.abs().amax(-1, keepdim=True)
    mant, ex = torch.frexp(top)
    e = (ex - 7 + (mant > 127.0 / 128.0)).clamp(min=-126)
    d = _pow2(e)
    q = torch.round(b / d.to(b.dtype))
    return q, torch.where(top == 0, torch.zeros_like(d), d)


def _weights(g, fmt, m, k):
    """m rows of k/32 random blocks, as ggml lays them out."""
    nb, size = m * (k // 32), BLOCK_BYTES[fmt]
    w = torch.randint(0, 256, (nb, size), device="cuda", dtype=torch.uint8, generator=g)
    d = (0.001 + 0.009 * torch.rand(nb, 1, device="cuda", generator=g)).half()
    w[:, 0:2] = d.view(torch.uint8)
    if fmt in ("q4_1", "q5_1"):
        w[:, 2:4] = (-0.1 * torch.rand(nb, 1, device="cuda", generator=g)).half().view(torch.uint8)
    return w.view(-1)


def prepare(c, seed):
    g = _gen(seed)
    s = {"c": dict(c)}
    op = c["op"]
    if op == "norm":
        dt = {"f32": torch.float32, "f16": torch.float16}[c["x"]]
        # a few channels carry larger values, as residual streams do
        loud = 1 + 7 * (torch.rand(c["k"], device="cuda", generator=g) < 0.01).float()
        s["x"] = (_randn(g, c["n"], c["k"]) * 0.5).to(dt)
        s["r"] = (_randn(g, c["n"], c["k"]) * 2 * loud).to(dt)
        s["w"] = 1 + 0.2 * _randn(g, c["k"])
    elif op == "gemv":
        s["w"] = _weights(g, c["fmt"], c["m"], c["k"])
        q, d = _x8_codes(_randn(g, c["n"], c["k"]))
        xq = torch.empty(c["n"], c["k"] // 32, X8_BYTES, dtype=torch.uint8, device="cuda")
        xq[..., :4] = d.contiguous().view(torch.uint8)
        xq[..., 4:] = q.to(torch.int8).view(torch.uint8)
        s["x"] = xq.view(c["n"], -1)
    elif op in ("store", "attn"):
        page, heads, dim = c["page"], c["heads"], c["dim"]
        if op == "store" and c["kind"] == "i8":
            # one prompt
            seqs, per = 1, c["pages"]
            s["seq"] = torch.zeros(c["tokens"], dtype=torch.int32, device="cuda")
            s["pos"] = torch.arange(c["tokens"], dtype=torch.int32, device="cuda")
        elif op == "store":
            # one token of each sequence, each somewhere in its pages
            seqs, per = c["tokens"], c["pages"]
            s["seq"] = torch.arange(seqs, dtype=torch.int32, device="cuda")
            s["pos"] = torch.randint(0, per * page, (seqs,), device="cuda", dtype=torch.int32, generator=g)
        else:
            seqs, per = c["seqs"], -(-c["most"] // page)
            at = torch.randperm(seqs, device="cuda", generator=g)
            s["lens"] = torch.tensor(_lens(c), dtype=torch.int32, device="cuda")[at]
        pages = seqs * per
        # the pages of a sequence lie anywhere in the cache
        s["table"] = torch.randperm(pages, device="cuda", generator=g).to(torch.int32).view(seqs, per)
        shape = (pages, heads, page, dim)
        if op == "store":
            s["k"], s["v"] = _randn(g, c["tokens"], heads, dim), _randn(g, c["tokens"], heads, dim)
            for p in ("k", "v"):
                s[p + "c"] = torch.zeros(shape, dtype=torch.float16 if c["kind"] == "f16" else torch.int8, device="cuda")
        else:
            s["q"] = _randn(g, seqs, c["q_heads"], dim) * 1.5
            s["scale"] = dim ** -0.5
            for p in ("k", "v"):
                x = torch.randn(shape, device="cuda", dtype=torch.float16, generator=g)
                s[p + "c"] = x if c["kind"] == "f16" else (x * 40).clamp_(-127, 127).round_().to(torch.int8)
        for p in ("k", "v"):
            s[p + "s"] = None
            if c["kind"] == "i8":
                s[p + "s"] = torch.zeros(shape[:3], device="cuda") if op == "store" else \
                    0.02 + 0.01 * torch.rand(shape[:3], device="cuda", generator=g)
        if own:
            from dequant_quantized_gemv_amd import qk
            s["cache"] = qk.KVCache(s["kc"], s["vc"], s["ks"], s["vs"])
            if op == "attn":
                # scratch that a serving loop keeps
                s["scratch"] = qk.attn_decode_workspace(s["cache"], seqs, c["q_heads"], c["most"],
                                                        window=c["window"], sinks=c["sinks"])
    else:
        s["x"] = _randn(g, c["tokens"], c["experts"]) * 1.5
        s["b"] = 0.1 * _randn(g, c["experts"]) if c["bias"] else None
    return s


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------

def _plain_norm(s):
    c = s["c"]
    t = s["x"].float() + s["r"].float()
    y = t * torch.rsqrt((t * t).mean(-1, keepdim=True) + EPS) * s["w"]
    if c["out"] == "x8":
        q, d = _x8_codes(y)
        y = (q * d).to(torch.bfloat16).view(y.shape)  # 7-bit codes by powers of two: exact
    elif c["out"] == "f16":
        y = y.half()
    return y, t.to(s["x"].dtype)


def _own_norm(s):
    from dequant_quantized_gemv_amd import qk
    c = s["c"]
    y, t = qk.rms_norm(s["x"], s["w"], EPS, residual=s["r"], out_dtype=c["out"])
    if c["out"] == "x8":
        # the values that the blocks stand for
        b = y.view(c["n"], -1, X8_BYTES)
        v = torch.empty(c["n"], c["k"] // 32, 32, dtype=torch.bfloat16, device=y.device)
        y = torch.mul(b[..., 4:].view(torch.int8), y.view(torch.float32).view(c["n"], -1, 9)[..., :1], out=v)
        y = y.view(c["n"], c["k"])
    return y, t


def _plain_weights(fmt, w, m, k, dtype=torch.float32):
    b = w.view(m, k // 32, BLOCK_BYTES[fmt])

    def half(at):
        return b[..., at:at + 2].contiguous().view(torch.float16).to(dtype)

    def nibbles(at):
        qs = b[..., at:at + 16]
        return torch.cat([qs & 15, qs >> 4], -1)

    def fifth(at):
        qh = b[..., at:at + 4]
        bits = (qh.unsqueeze(-1) >> torch.arange(8, device=w.device, dtype=torch.uint8)) & 1
        return bits.reshape(*qh.shape[:-1], 32) << 4

    if fmt == "q8_0":
        v = b[..., 2:].contiguous().view(torch.int8).to(dtype) * half(0)
    elif fmt == "q4_0":
        v = (nibbles(2).to(dtype) - 8) * half(0)
    elif fmt == "q4_1":
        v = nibbles(4).to(dtype) * half(0) + half(2)
    elif fmt == "q5_0":
        v = ((nibbles(6) | fifth(2)).to(dtype) - 16) * half(0)
    else:
        v = (nibbles(8) | fifth(4)).to(dtype) * half(0) + half(2)
    return v.view(m, k)


def _x8_values(x, dtype=torch.float32):
    b = x.view(x.shape[0], -1, X8_BYTES)
    d = b[..., :4].contiguous().view(torch.float32).to(dtype)
    return (b[..., 4:].contiguous().view(torch.int8).to(dtype) * d).view(x.shape[0], -1)


def _plain_store(s):
    c = s["c"]
    pos = s["pos"].long()
    at = s["table"][s["seq"].long(), pos // c["page"]].long()
    slot = pos % c["page"]
    out = []
    for p in ("k", "v"):
        x, pool = s[p], s[p + "c"]
        if c["kind"] == "f16":
            pool[at, :, slot] = x.half()
            out.append(pool)
        else:
            # (divided by a tensor: a plain 127 would be a product with its rounded reciprocal)
            top = x.abs().amax(-1, keepdim=True)
            d = top / torch.full_like(top, 127)
            q = torch.where(d > 0, torch.round(x / d), torch.zeros_like(x))
            pool[at, :, slot] = q.to(torch.int8)
            s[p + "s"][at, :, slot] = d[..., 0]
            out.append(torch.mul(pool, s[p + "s"][..., None]))
    return out


def _own_store(s):
    from dequant_quantized_gemv_amd import qk
    c = s["c"]
    qk.kv_store(s["cache"], s["k"], s["v"], s["table"], s["pos"], seq=s["seq"])
    if c["kind"] == "f16":
        return [s["kc"], s["vc"]]
    return [torch.mul(s[p + "c"], s[p + "s"][..., None]) for p in ("k", "v")]


def _plain_attn(s):
    c = s["c"]
    n, heads, dim, page = c["seqs"], c["heads"], c["dim"], c["page"]
    per = s["table"].shape[1]
    table = s["table"].long().view(-1)

    def rows(p):
        x = s[p + "c"][table].float()
        if c["kind"] == "i8":
            x = x * s[p + "s"][table][..., None]
        return x.view(n, per, heads, page, dim).permute(0, 2, 1, 3, 4).reshape(n, heads, per * page, dim)

    t = torch.arange(per * page, device="cuda")
    lens = s["lens"].long()[:, None]
    seen = t < lens
    if c["window"]:
        seen = seen & ((t >= lens - c["window"]) | (t < c["sinks"]))
    q = s["q"].view(n, heads, -1, dim) * s["scale"]
    z = torch.matmul(q, rows("k").transpose(-1, -2).contiguous())
    z = z.masked_fill(~seen[:, None, None], float("-inf"))
    z = torch.exp(z - z.amax(-1, keepdim=True))
    y = torch.matmul(z, rows("v")) / z.sum(-1, keepdim=True)
    y = y.reshape(n, c["q_heads"], dim)
    return y.half() if c["out"] == "f16" else y


def _own_attn(s):
    from dequant_quantized_gemv_amd import qk
    c = s["c"]
    return qk.attn_decode(s["cache"], s["q"], s["table"], s["lens"], s["scale"], window=c["window"],
                          sinks=c["sinks"], max_len=c["most"], out_dtype=c["out"], workspace=s["scratch"])


def _scores(x, score):
    if score == "sigmoid":
        return 1 / (1 + torch.exp(-x))
    e = torch.exp(x - x.amax(-1, keepdim=True))
    # (the sum in 64 bits and rounded once, so that its order does not decide a choice)
    return e / e.sum(-1, keepdim=True, dtype=torch.float64).to(x.dtype)


def _choose(c, x, b):
    """Chosen experts and their weights, from fp32 or fp64 logits."""
    p = _scores(x, c["score"])
    by_logit = b is None and c["best"] == 1  # both scores rise with the logit
    v = x if by_logit else p if b is None else p + b.to(x.dtype)
    if c["kept"] < c["groups"]:
        per = v.view(v.shape[0], c["groups"], -1)
        best = per.sort(-1, descending=True)[0][..., :c["best"]].sum(-1)
        keep = best.sort(dim=-1, descending=True, stable=True)[1][:, :c["kept"]]
        in_kept = torch.zeros_like(best, dtype=torch.bool).scatter_(1, keep, True)
        v = per.masked_fill(~in_kept[..., None], float("-inf")).view(v.shape)
    ids = v.sort(dim=-1, descending=True, stable=True)[1][:, :c["used"]]
    w = p.gather(1, ids)
    return ids.to(torch.int32), w / w.sum(-1, keepdim=True)


def _own_route(s):
    from dequant_quantized_gemv_amd import qk
    c = s["c"]
    return qk.moe_route(s["x"], c["used"], score=c["score"], bias=s["b"], n_groups=c["groups"],
                        topk_groups=c["kept"], group_top=c["best"])


def run(s):
    c = s["c"]
    op = c["op"]
    if op == "norm":
        return _own_norm(s) if own else _plain_norm(s)
    if op == "gemv":
        if own:
            from dequant_quantized_gemv_amd import qk
            return qk.mul_mat_vec_x8q(c["fmt"], s["w"], c["m"], c["k"], s["x"])
        return torch.matmul(_x8_values(s["x"]), _plain_weights(c["fmt"], s["w"], c["m"], c["k"]).t())
    if op == "store":
        return _own_store(s) if own else _plain_store(s)
    if op == "attn":
        return _own_attn(s) if own else _plain_attn(s)
    return _own_route(s) if own else _choose(c, s["x"], s["b"])


# --------------------------------------------------------------------------
# 64 bits
# --------------------------------------------------------------------------

def _weight_by_index(fmt, blocks):
    """Weights in 64 bits (rows, blocks, 32), element t of a block from its own bytes."""
    f64 = torch.float64
    t = torch.arange(32, device=blocks.device)
    b = blocks.long()

    def half(at):
        return blocks[..., at:at + 2].clone().view(torch.float16).to(f64)

    if fmt == "q8_0":
        q = b[..., 2 + t]
        return half(0) * (q - 256 * (q > 127)).to(f64)
    low, high = {"q4_0": (2, None), "q4_1": (4, None), "q5_0": (6, 2), "q5_1": (8, 4)}[fmt]
    q = (b[..., low + t % 16] >> (4 * (t // 16))) & 15
    if high is not None:
        q = q + 16 * ((b[..., high + t // 8] >> (t % 8)) & 1)
    if fmt in ("q4_1", "q5_1"):
        return half(0) * q.to(f64) + half(2)
    return half(0) * (q - {"q4_0": 8, "q5_0": 16}[fmt]).to(f64)


def exact(c, seed):
    s = prepare(c, seed)
    op, f64 = c["op"], torch.float64
    if op == "norm":
        t = s["x"].to(f64) + s["r"].to(f64)
        ms = torch.square(t).sum(-1, keepdim=True) / c["k"]
        # (8-bit outputs are held against the values that they were rounded from)
        return t / torch.sqrt(ms + EPS) * s["w"].to(f64), t
    if op == "gemv":
        m, k, n = c["m"], c["k"], c["n"]
        xb = s["x"].view(n, k // 32, X8_BYTES)
        code = xb[..., 4:].to(f64)
        x = torch.where(code > 127, code - 256, code) * xb[..., :4].clone().view(torch.float32).to(f64)
        blocks = s["w"].view(m, k // 32, -1)
        out = []
        for i in range(0, m, 2048):  # a part of the rows at a time
            w = _weight_by_index(c["fmt"], blocks[i:i + 2048])
            out.append((w[None] * x[:, None]).sum((-1, -2)))
        return torch.cat(out, 1)
    if op == "store":
        out = []
        for p in ("k", "v"):
            x = s[p].to(f64)
            if c["kind"] == "i8":
                d = x.abs().amax(-1, keepdim=True) / 127
                x = torch.round(x / d) * d
            pool, table = s[p + "c"].to(f64), s["table"].tolist()
            for i, (q, t) in enumerate(zip(s["seq"].tolist(), s["pos"].tolist())):
                pool[table[q][t // c["page"]], :, t % c["page"]] = x[i]
            out.append(pool)
        return out
    if op == "attn":
        out = []
        group, page = c["q_heads"] // c["heads"], c["page"]
        for i, n in enumerate(s["lens"].tolist()):
            t = torch.arange(n, device="cuda")
            if c["window"]:
                t = t[(t < c["sinks"]) | (t >= n - c["window"])]
            at, slot = s["table"][i].long()[t // page], t % page
            kv = []
            for p in ("k", "v"):
                x = s[p + "c"][at, :, slot].to(f64)
                kv.append(x * s[p + "s"][at, :, slot].to(f64)[..., None] if c["kind"] == "i8" else x)
            rows = []
            for h in range(c["q_heads"]):
                z = (kv[0][:, h // group] * s["q"][i, h].to(f64)).sum(-1) * s["scale"]
                z = torch.softmax(z, 0)
                rows.append((z[:, None] * kv[1][:, h // group]).sum(0))
            out.append(torch.stack(rows))
        return torch.stack(out)
    # experts taken one after another
    x = s["x"].to(f64)
    p = torch.sigmoid(x) if c["score"] == "sigmoid" else torch.softmax(x, -1)
    v = p.clone() if s["b"] is None else p + s["b"].to(f64)
    size, rows = c["experts"] // c["groups"], torch.arange(c["tokens"], device="cuda")
    if c["kept"] < c["groups"]:
        best = sum(v.view(-1, c["groups"], size).topk(min(c["best"], size), -1)[0].unbind(-1))
        dropped = best.topk(c["groups"] - c["kept"], -1, largest=False)[1]
        v.view(-1, c["groups"], size)[rows[:, None], dropped] = -math.inf
    taken = []
    for _ in range(c["used"]):
        i = v.argmax(-1)
        taken.append(p[rows, i])
        v[rows, i] = -math.inf
    w = torch.stack(taken, -1)
    return [None, w / w.sum(-1, keepdim=True)]
