"""Timed cases of the operators with which one prompt is given many answers:
the pages of a cache as sequences fork, grow, are dropped and packed together,
the attention of a batch whose sequences share prefixes, and the log
probabilities, entropy and best alternatives of a vocabulary's logits.

`run` computes a case in plain torch operations (`own` false) or through the
public calls of dequant_quantized_gemv_amd.qk (`own` true); `exact` computes
it in 64 bits (pages: one after another).
"""
import math

import torch

own = False


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------

def _copy(name, kind, pairs, heads, dim, page):
    return {"name": name, "op": "copy", "kind": kind, "pairs": pairs, "heads": heads, "dim": dim, "page": page}


def _fork(name, rows, most, page, spare, how):
    return {"name": name, "op": "fork", "rows": rows, "most": most, "page": page, "spare": spare, "how": how}


def _compact(name, rows, most, page, n_pages):
    return {"name": name, "op": "compact", "rows": rows, "most": most, "page": page, "pages": n_pages}


def _attn(name, kind, groups, seqs, ragged, shared, tail, q_heads, heads, dim, page, out="f32"):
    return {"name": name, "op": "attn", "kind": kind, "groups": groups, "seqs": seqs, "ragged": ragged,
            "shared": shared, "tail": tail, "q_heads": q_heads, "heads": heads, "dim": dim, "page": page, "out": out}


def _logp(name, x, n, vocab, ids, top, scale=1.0, masked=False):
    return {"name": name, "op": "logp", "x": x, "n": n, "vocab": vocab, "ids": ids, "top": top, "scale": scale,
            "masked": masked}


def listed():
    return [
        # eight branches of an answer begin to differ inside a page of their 8-bit cache
        _copy("copy i8 8", "i8", 8, 8, 128, 16),
        # half of a pool packed into its other half
        _copy("copy f16 2000", "f16", 2000, 8, 128, 16),
        # four beams, each step
        _fork("fork 4 beams", 4, 1000, 16, 64, "beams"),
        # a prompt forked for 64 answers, each of which has begun to grow
        _fork("fork 64 of 4096", 64, 4096, 16, 512, "fork"),
        # a small pool after some of its sequences have ended
        _compact("compact 8 rows", 8, 1000, 16, 1024),
        # a large pool half of which is free
        _compact("compact 64 rows", 64, 8192, 16, 65536),
        # four answers to one short prompt: latency
        _attn("attn f16 1x4 of 1000", "f16", 1, 4, False, 1000, 64, 32, 8, 128, 16),
        # sixteen prompts with four to twelve answers each, every head with keys of its own in pages that end inside a tile
        _attn("attn f16 16x8 of 2000", "f16", 16, 128, True, 2000, 200, 16, 16, 64, 24, "f16"),
        # a system prompt in front of 64 conversations, in 8 bits
        _attn("attn i8 1x64 of 8192", "i8", 1, 64, False, 8192, 1024, 32, 8, 128, 16),
        # 64 questions about one long document
        _attn("attn f16 1x64 of 32768", "f16", 1, 64, False, 32768, 256, 32, 8, 128, 64),
        # one sampled token: its probability and the 20 likeliest
        _logp("logp f32 1x32000 top20", "f32", 1, 32000, 1, 20),
        # a prompt's tokens scored
        _logp("logp f32 2048x32000 top5", "f32", 2048, 32000, 1, 5),
    ]


def _spread(rng, lo, hi):
    """A whole number of lo..hi, spread over its logarithm."""
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49))))))


def draw(rng):
    op = rng.choice(["copy", "fork", "compact", "attn", "attn", "logp", "logp"])
    page = rng.choice([1, 8, 16, 16, 24, 32, 64, 100])
    if op == "copy":
        heads, dim = rng.choice([1, 2, 3, 4, 8]), 32 * rng.randint(1, 8)
        c = _copy("", rng.choice(["f16", "i8"]), _spread(rng, 1, max(1, min(4000, 2000 * 16 * 8 * 128 // (page * heads * dim)))),
                  heads, dim, page)
    elif op == "fork":
        rows = _spread(rng, 1, 256)
        c = _fork("", rows, _spread(rng, 1, 64 * 256 // rows * page), page, _spread(rng, 1, 1024),
                  rng.choice(["fork", "beams", "grow"]))
    elif op == "compact":
        rows = _spread(rng, 1, 256)
        most = _spread(rng, 1, 64 * 512 // rows * page)
        least = rows * -(-most // page)
        c = _compact("", rows, most, page, _spread(rng, max(2, least), max(least + 2, min(65536, 4 * least))))
    elif op == "attn":
        heads = rng.choice([1, 2, 4, 5, 8])
        q_heads = heads * rng.choice([1, 2, 3, 4, 6, 7, 8, 16])
        dim = 32 * rng.choice([1, 2, 2, 3, 4, 4, 4, 5, 6, 8])
        seqs = _spread(rng, 1, 128)
        groups = min(seqs, _spread(rng, 1, 16))
        page = max(page, 8)
        cost = 64 * 32 * 32768 * 128 // (seqs * q_heads * dim)
        shared = _spread(rng, 1, max(1, min(65536, cost // 2, 32768 * 8 * 128 // (groups * heads * dim))))
        tail = _spread(rng, 1, max(1, min(1024, 64 * 1024 * 8 * 128 // (seqs * heads * dim))))
        c = _attn("", rng.choice(["f16", "i8"]), groups, seqs, rng.random() < 0.6, shared, tail, q_heads, heads, dim,
                  page, rng.choice(["f32", "f16"]))
    else:
        vocab = _spread(rng, 2, 262144)
        n = _spread(rng, 1, max(1, min(4096, 2048 * 32000 // vocab)))
        c = _logp("", rng.choice(["f32", "f16"]), n, vocab, rng.choice([0, 1, 1, 2, 7]),
                  min(vocab, rng.choice([0, 0, 1, 5, 8, 20, 64])), rng.choice([1.0, 0.5, 1.25, 2.0]), rng.random() < 0.3)
    del c["name"]
    return c


def _group_sizes(c):
    """Sequences of each group."""
    n, g = c["seqs"], c["groups"]
    if not c["ragged"]:
        return [n * (i + 1) // g - n * i // g for i in range(g)]
    # from half to one and a half of an even share
    ends = [0] + [min(n, round(n * (0.5 * x + 0.5 * x * x))) for x in ((i + 1) / g for i in range(g))]
    return [b - a for a, b in zip(ends, ends[1:])]


def _group_shared(c):
    """Tokens that each group shares."""
    n, g = c["shared"], c["groups"]
    return [max(1, n * (2 * i + 1) // (2 * g)) if c["ragged"] and g > 1 else n for i in range(g)]


def _tails(c):
    """Tokens of its own of each sequence, before they are shuffled."""
    n = c["seqs"]
    return [max(1, math.ceil(c["tail"] * (i + 1) / n)) for i in range(n)]


def work(c):
    op = c["op"]
    if op == "copy":
        row = c["dim"] * 2 if c["kind"] == "f16" else c["dim"] + 4
        return {"bytes": 4 * c["pairs"] * c["heads"] * c["page"] * row + 8 * c["pairs"], "flops": 0}
    if op in ("fork", "compact"):
        entries = c["rows"] * -(-c["most"] // c["page"])
        pages = entries + c["spare"] if op == "fork" else c["pages"]
        return {"bytes": 8 * entries + pages // 8 + (20 * c["rows"] if op == "fork" else 4 * c["rows"] + 4 * pages), "flops": 0}
    if op == "attn":
        sizes, shared, tails = _group_sizes(c), _group_shared(c), _tails(c)
        row = c["dim"] * 2 if c["kind"] == "f16" else c["dim"] + 4
        tokens = sum(s for s, z in zip(shared, sizes) if z) + sum(tails)
        seen = sum(s * z for s, z in zip(shared, sizes)) + sum(tails)
        io = c["seqs"] * c["q_heads"] * c["dim"] * (4 + (4 if c["out"] == "f32" else 2))
        return {"bytes": 2 * tokens * c["heads"] * row + io + 4 * -(-tokens // c["page"]),
                "flops": 4 * seen * c["q_heads"] * c["dim"]}
    size = 4 if c["x"] == "f32" else 2
    return {"bytes": c["n"] * (c["vocab"] * size + 8 * c["ids"] + 8 * c["top"] + 4), "flops": 6 * c["n"] * c["vocab"]}


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _int(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _perm(g, n):
    return torch.randperm(n, device="cuda", generator=g).to(torch.int32)


def _pools(s, c, g, pages):
    shape = (pages, c["heads"], c["page"], c["dim"])
    for p in ("k", "v"):
        x = torch.randn(shape, device="cuda", dtype=torch.float16, generator=g)
        s[p + "c"], s[p + "s"] = x, None
        if c["kind"] == "i8":
            s[p + "c"] = (x * 40).clamp_(-127, 127).round_().to(torch.int8)
            s[p + "s"] = 0.02 + 0.01 * torch.rand(shape[:3], device="cuda", generator=g)


def _prepare_attn(s, c, g):
    page, sizes, shared = c["page"], _group_sizes(c), _group_shared(c)
    n, most = c["seqs"], c["shared"] + c["tail"]
    per = -(-most // page)
    own_pages = [-(-(sh + c["tail"]) // page) - sh // page for sh in shared]
    total = sum(sh // page + z * o for sh, z, o in zip(shared, sizes, own_pages))
    _pools(s, c, g, total)
    ids, at, row = _perm(g, total), 0, 0
    table = torch.zeros(n, per, dtype=torch.int32, device="cuda")
    for sh, z, o in zip(shared, sizes, own_pages):
        whole = sh // page
        table[row:row + z, :whole] = ids[at:at + whole]
        at += whole
        table[row:row + z, whole:whole + o] = ids[at:at + z * o].view(z, o)
        at += z * o
        if sh % page and z > 1:
            # the shared tokens of a page that each sequence has a copy of
            first, rest = table[row, whole].long(), table[row + 1:row + z, whole].long()
            for p in ("kc", "vc", "ks", "vs"):
                if s[p] is not None:
                    s[p][rest, :, :sh % page] = s[p][first, :, :sh % page]
        row += z
    s["table"] = table
    order = torch.randperm(n, device="cuda", generator=g)
    each = torch.tensor([sh for sh, z in zip(shared, sizes) for _ in range(z)], device="cuda")
    s["lens"] = (each + torch.tensor(_tails(c), device="cuda")[order]).to(torch.int32)
    ends = [sum(sizes[:i]) for i in range(len(sizes) + 1)]
    s["starts"], s["shared"] = _int(ends), _int(shared)
    s["q"] = torch.randn(n, c["q_heads"], c["dim"], device="cuda", generator=g) * 1.5
    s["scale"] = c["dim"] ** -0.5


def prepare(c, seed):
    g = _gen(seed)
    s = {"c": dict(c)}
    op = c["op"]
    if op == "copy":
        n = c["pairs"]
        _pools(s, c, g, 2 * n + 1)
        ids = _perm(g, 2 * n + 1)
        s["src"], s["dst"] = ids[:n].clone(), ids[n:2 * n].clone()
        if n >= 4:
            # rows that have nothing to copy
            none = torch.rand(n, device="cuda", generator=g) < 0.1
            s["src"][none] = -1
            s["dst"][none] = -1
    elif op == "fork":
        rows, most, page = c["rows"], c["most"], c["page"]
        per = -(-most // page)
        s["pages"] = rows * per + c["spare"]
        s["table"] = _perm(g, s["pages"])[:rows * per].view(rows, per)
        s["lens"] = torch.randint(1, most + 1, (rows,), device="cuda", generator=g).to(torch.int32)
        s["parent"] = None
        if c["how"] == "fork":
            s["parent"] = torch.zeros(rows, dtype=torch.int32, device="cuda")
            s["lens"][0] = max(1, most - most // 8)
        elif c["how"] == "beams":
            s["parent"] = torch.randint(0, rows, (rows,), device="cuda", generator=g).to(torch.int32)
        old = s["lens"] if s["parent"] is None else s["lens"][s["parent"].long()]
        s["new"] = (old + torch.randint(1, 5, (rows,), device="cuda", generator=g)).clamp(max=most).to(torch.int32)
    elif op == "compact":
        rows, most, page = c["rows"], c["most"], c["page"]
        per = -(-most // page)
        s["table"] = _perm(g, c["pages"])[:rows * per].view(rows, per)
        s["lens"] = torch.randint(0, most + 1, (rows,), device="cuda", generator=g).to(torch.int32)
    elif op == "attn":
        _prepare_attn(s, c, g)
    else:
        n, vocab = c["n"], c["vocab"]
        # logits of a language model: a few tokens stand out
        x = torch.randn(n, vocab, device="cuda", generator=g) * 2
        x += 8 * (torch.rand(n, vocab, device="cuda", generator=g) < 4 / vocab)
        if c["masked"]:
            x[torch.rand(n, vocab, device="cuda", generator=g) < 0.3] = -math.inf
            x[:, vocab // 2] = 0.0
        s["x"] = x if c["x"] == "f32" else x.half()
        s["ids"] = torch.randint(0, vocab, (n, c["ids"]), device="cuda", generator=g).to(torch.int32) if c["ids"] else None
    if own:
        from dequant_quantized_gemv_amd import qk
        # scratch that a serving loop keeps
        if op in ("copy", "attn"):
            s["cache"] = qk.KVCache(s["kc"], s["vc"], s["ks"], s["vs"])
        if op == "attn":
            s["scratch"] = qk.attn_decode_shared_workspace(s["cache"], c["seqs"], c["q_heads"],
                                                           c["shared"] + c["tail"], c["shared"], c["tail"])
        elif op == "fork":
            s["scratch"] = qk.kv_pages_workspace(c["rows"], s["pages"])
        elif op == "compact":
            s["scratch"] = qk.kv_pages_workspace(c["rows"], c["pages"])
        elif op == "logp":
            s["scratch"] = qk.token_logprobs_workspace(c["n"], c["vocab"], c["top"])
    return s


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------

def _pool_values(s):
    if s["ks"] is None:
        return [s["kc"], s["vc"]]
    return [torch.mul(s[p + "c"], s[p + "s"][..., None]) for p in ("k", "v")]


def _plain_copy(s):
    src, dst = s["src"].long(), s["dst"].long()
    # a pair of -1 writes a page over itself that is nobody's source or destination
    used = torch.zeros(s["kc"].shape[0], dtype=torch.uint8, device="cuda")
    used[src.clamp(min=0)] = 1
    used[dst.clamp(min=0)] = 1
    idle, ok = torch.argmin(used), src >= 0
    src, dst = torch.where(ok, src, idle), torch.where(ok, dst, idle)
    for p in ("kc", "vc", "ks", "vs"):
        if s[p] is not None:
            s[p][dst] = s[p][src]


def _lists(held, n):
    """Numbers of the pages that are true in `held`, ascending, in a tensor of n (-1 behind them), and their count."""
    at = torch.cumsum(held, 0) - 1
    out = torch.full((n + 1,), -1, dtype=torch.int64, device="cuda")
    out.scatter_(0, torch.where(held & (at < n), at, n), torch.arange(held.shape[0], device="cuda"))
    return out[:n], held.sum()


def _plain_fork(s):
    c = s["c"]
    page, pages, table = c["page"], s["pages"], s["table"].long()
    rows, per = table.shape
    old = s["lens"].long()
    if s["parent"] is not None:
        par = s["parent"].long()
        table, old = table[par], old[par]
    new = s["new"].long()
    kept = (torch.minimum(old, new) + page - 1) // page
    want = (new + page - 1) // page
    j = torch.arange(per, device="cuda")
    table = torch.where(j < kept[:, None], table, -1)
    count = torch.zeros(pages + 1, dtype=torch.int64, device="cuda")
    count.scatter_add_(0, table.view(-1) % (pages + 1), torch.ones(rows * per, dtype=torch.int64, device="cuda"))
    count = count[:pages]  # (-1 counts behind the last page)
    at = (old // page).clamp(max=per - 1)
    last = table.gather(1, at[:, None])[:, 0]
    copied = (new > old) & (old % page != 0) & (count[last.clamp(min=0)] > 1)
    wanted = ((j >= kept[:, None]) & (j < want[:, None])) | (copied[:, None] & (j == at[:, None]))
    free, n = _lists(count == 0, pages)
    rank = torch.cumsum(wanted.view(-1), 0).view(rows, per) - 1
    got = torch.where(rank < n, free[rank.clamp(0, pages - 1)], -1)
    out = torch.where(wanted, got, table)
    dst = torch.where(copied, out.gather(1, at[:, None])[:, 0], -1)
    src = torch.where(dst >= 0, last, -1)
    missing = (wanted.sum() - n).clamp(min=0).view(1)
    return [x.to(torch.int32) for x in (out, src, dst, missing)]


def _plain_compact(s):
    c = s["c"]
    page, pages, table = c["page"], c["pages"], s["table"].long()
    rows, per = table.shape
    kept = (s["lens"].long() + page - 1) // page
    table = torch.where(torch.arange(per, device="cuda") < kept[:, None], table, -1)
    held = torch.zeros(pages + 1, dtype=torch.bool, device="cuda")
    held[table.view(-1) % (pages + 1)] = True
    held = held[:pages]
    p = torch.arange(pages, device="cuda")
    n = held.sum()
    src, moved = _lists(held & (p >= n), pages // 2)
    dst, _ = _lists(~held & (p < n), pages // 2)
    name = torch.cat([p, p[:1] - 1])
    back = torch.where(src >= 0, src, pages)
    name.scatter_(0, back, torch.where(src >= 0, dst, -1))
    return [x.to(torch.int32) for x in (name[table % (pages + 1)], src, dst, n.view(1))]


def _plain_attn(s):
    c = s["c"]
    heads, dim, page, per = c["heads"], c["dim"], c["page"], s["table"].shape[1]
    n, group = c["seqs"], c["q_heads"] // c["heads"]

    def rows(p, table):
        """Values (sequences, heads, tokens, dim) of whole pages."""
        x = s[p + "c"][table].float()
        if c["kind"] == "i8":
            x = x * s[p + "s"][table][..., None]
        return x.permute(0, 2, 1, 3, 4).reshape(table.shape[0], heads, -1, dim)

    q = (s["q"] * s["scale"]).view(n, heads, group, dim)
    out, row = [], 0
    for size, shared in zip(_group_sizes(c), _group_shared(c)):
        if size == 0:
            continue
        table, lens = s["table"][row:row + size].long(), s["lens"][row:row + size].long()
        first, last = shared // page, min(per, -(-(shared + c["tail"]) // page))
        qg = q[row:row + size]
        # the prefix once for all, then each sequence's own tokens
        pages = table[:1, :-(-shared // page)]
        pk, pv = rows("k", pages)[0, :, :shared], rows("v", pages)[0, :, :shared]
        qp = qg.transpose(0, 1).reshape(heads, size * group, dim)
        z0 = torch.matmul(qp, pk.transpose(-1, -2).contiguous())
        z0 = z0.view(heads, size, group, shared).transpose(0, 1)
        z1 = torch.matmul(qg, rows("k", table[:, first:last]).transpose(-1, -2).contiguous())
        t = torch.arange(first * page, last * page, device="cuda")
        seen = (t >= shared) & (t < lens[:, None])
        z1 = z1.masked_fill(~seen[:, None, None], float("-inf"))
        m = torch.maximum(z0.amax(-1, keepdim=True), z1.amax(-1, keepdim=True))
        z0, z1 = torch.exp(z0 - m), torch.exp(z1 - m)
        y0 = torch.matmul(z0.transpose(0, 1).reshape(heads, size * group, shared), pv)
        y = y0.view(heads, size, group, dim).transpose(0, 1) + torch.matmul(z1, rows("v", table[:, first:last]))
        out.append((y / (z0.sum(-1, keepdim=True) + z1.sum(-1, keepdim=True))).reshape(size, c["q_heads"], dim))
        row += size
    y = torch.cat(out)
    return y.half() if c["out"] == "f16" else y


def _plain_logp(s):
    c = s["c"]
    x = s["x"].float()
    n, vocab = x.shape
    top = x.amax(-1, keepdim=True)
    z = (x - top) * c["scale"]
    e = torch.exp(z)
    # (sums in 64 bits: the logarithm of one near 1 is an answer)
    total = e.sum(-1, keepdim=True, dtype=torch.float64)
    ln = torch.log(total)
    ez = torch.where(e > 0, e * z, 0).sum(-1, dtype=torch.float64)
    entropy = (ln[:, 0] - ez / total[:, 0]).float()
    lp = ids = best = None
    if s["ids"] is not None:
        lp = (z.gather(1, s["ids"].long()) - ln).float()
    if c["top"]:
        # of equal logits the first: the order of the floats, then the index from behind
        bits = (x + 0.0).view(torch.int32).long()
        key = torch.where(bits < 0, -(bits & 0x7FFFFFFF), bits)
        key = key * vocab + torch.arange(vocab - 1, -1, -1, device="cuda")
        at = key.topk(c["top"], -1)[1]
        ids, best = at.to(torch.int32), (z.gather(1, at) - ln).float()
    return lp, entropy, ids, best


def _own(s):
    from dequant_quantized_gemv_amd import qk
    c = s["c"]
    op = c["op"]
    if op == "copy":
        qk.kv_copy(s["cache"], s["src"], s["dst"])
        return _pool_values(s)
    if op == "fork":
        return qk.kv_fork(s["table"], s["lens"], s["new"], c["page"], s["pages"], parent=s["parent"], workspace=s["scratch"])
    if op == "compact":
        return qk.kv_compact(s["table"], s["lens"], c["page"], c["pages"], workspace=s["scratch"])
    if op == "attn":
        return qk.attn_decode_shared(s["cache"], s["q"], s["table"], s["lens"], s["starts"], s["shared"], s["scale"],
                                     max_len=c["shared"] + c["tail"], max_shared=c["shared"], max_own=c["tail"],
                                     out_dtype=c["out"], workspace=s["scratch"])
    return qk.token_logprobs(s["x"], s["ids"], top=c["top"], scale=c["scale"], workspace=s["scratch"])


def run(s):
    if own:
        return _own(s)
    op = s["c"]["op"]
    if op == "copy":
        _plain_copy(s)
        return _pool_values(s)
    return {"fork": _plain_fork, "compact": _plain_compact, "attn": _plain_attn, "logp": _plain_logp}[op](s)


# --------------------------------------------------------------------------
# from the definitions, in 64 bits
# --------------------------------------------------------------------------

def _exact_fork(s, c):
    page, pages = c["page"], s["pages"]
    table, lens, new = s["table"].tolist(), s["lens"].tolist(), s["new"].tolist()
    parent = list(range(c["rows"])) if s["parent"] is None else s["parent"].tolist()
    per, out, holders = len(table[0]), [], {}
    for p, n in zip(parent, new):
        row = table[p][:-(-min(lens[p], n) // page)]
        for i in row:
            holders[i] = holders.get(i, 0) + 1
        out.append(row)
    free = [i for i in range(pages) if i not in holders][::-1]
    src, dst, missing = [], [], 0

    def take():
        nonlocal missing
        if free:
            return free.pop()
        missing += 1
        return -1

    for row, p, n in zip(out, parent, new):
        a = b = -1
        if n > lens[p] and lens[p] % page and holders[row[-1]] > 1:
            b = take()
            a = row[-1] if b >= 0 else -1
            row[-1] = b
        while len(row) * page < n:
            row.append(take())
        src.append(a)
        dst.append(b)
        row += [-1] * (per - len(row))
    return [_int(out), _int(src), _int(dst), _int([missing])]


def _exact_compact(s, c):
    lens, per = s["lens"].tolist(), s["table"].shape[1]
    rows = [r[:-(-n // c["page"])] for r, n in zip(s["table"].tolist(), lens)]
    live = sorted({i for r in rows for i in r})
    n, have = len(live), set(live)
    src = [i for i in live if i >= n]
    dst = [i for i in range(n) if i not in have]
    to = dict(zip(src, dst))
    out = [[to.get(i, i) for i in r] + [-1] * (per - len(r)) for r in rows]
    pad = [-1] * (c["pages"] // 2 - len(src))
    return [_int(out), _int(src + pad), _int(dst + pad), _int([n])]


def exact(c, seed):
    s = prepare(c, seed)
    op, f64 = c["op"], torch.float64
    if op == "copy":
        out = []
        for p in ("k", "v"):
            x = s[p + "c"].to(f64)
            if s[p + "s"] is not None:
                x = x * s[p + "s"].to(f64)[..., None]
            for a, b in zip(s["src"].tolist(), s["dst"].tolist()):
                if a >= 0:
                    x[b] = x[a]
            out.append(x)
        return out
    if op == "fork":
        return _exact_fork(s, c)
    if op == "compact":
        return _exact_compact(s, c)
    if op == "attn":
        # every sequence over all of its tokens
        out, group = [], c["q_heads"] // c["heads"]
        if c["seqs"] * c["heads"] > 4096:
            return None
        for i, n in enumerate(s["lens"].tolist()):
            t = torch.arange(n, device="cuda")
            at, slot = s["table"][i].long()[t // c["page"]], t % c["page"]
            kv = []
            for p in ("k", "v"):
                x = s[p + "c"][at, :, slot].to(f64)
                kv.append(x if s[p + "s"] is None else x * s[p + "s"][at, :, slot].to(f64)[..., None])
            q = s["q"][i].to(f64).view(c["heads"], group, c["dim"]) * s["scale"]
            heads = []
            for h in range(c["heads"]):
                p = torch.softmax(q[h] @ kv[0][:, h].T, -1)
                heads.append(p @ kv[1][:, h])
            out.append(torch.cat(heads))
        return torch.stack(out)
    x = s["x"].to(f64) * c["scale"]
    lp, entropy = [], []
    ids, best = ([], []) if c["top"] else (None, None)
    for i in range(0, c["n"], 256):  # a part of the rows at a time
        part = x[i:i + 256]
        p = torch.log_softmax(part, -1)
        entropy.append(torch.special.entr(torch.exp(p)).sum(-1))
        if c["ids"]:
            lp.append(p.gather(1, s["ids"][i:i + 256].long()))
        if c["top"]:
            at = s["x"][i:i + 256].to(f64).sort(dim=-1, descending=True, stable=True)[1][:, :c["top"]]
            ids.append(at.to(torch.int32))
            best.append(p.gather(1, at))
    return (torch.cat(lp) if c["ids"] else None, torch.cat(entropy),
            torch.cat(ids) if c["top"] else None, torch.cat(best) if c["top"] else None)
