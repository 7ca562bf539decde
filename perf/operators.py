"""Measured cases of the attention block of a decode step: queries and keys normalised per head and rotated
(``qk_norm_rope``), keys and values appended to a paged cache of E4M3 codes with one power-of-two scale for each page
and head (``kv_append``), and attention over that cache (``kv_attention``).

``run`` computes an operator in elementary 32-bit torch operations, or with ``own`` set through the library's calls;
``exact`` computes it in 64 bits, one sequence at a time, from the definition.
"""
import math
import random

import torch

own = False  # set by whoever measures: run() makes the library's calls

EPS = 1e-6
THETA = 10000.0
E_MIN, E_MAX = -64, 64  # exponents of the page scales


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one request's decode step: 28 query heads of 128 feed the 3584-wide projection
        dict(name="append 1 token", op="append", batch=1, new=1, max_len=700, spread=1, heads=28, kv_heads=4, dim=128,
             page=64, rot=128, interleaved=False, norm=True),
        # decode step of a batch in which the page scales grow on the way; small heads and pages
        dict(name="append 48 decode rows", op="append", batch=48, new=1, max_len=8000, spread=2, heads=32, kv_heads=8,
             dim=64, page=16, rot=64, interleaved=False, norm=False),
        # prompts of one scheduling step, ragged
        dict(name="append prompts", op="append", batch=5, new=1638, max_len=5000, spread=3, heads=64, kv_heads=8,
             dim=128, page=32, rot=128, interleaved=True, norm=True),
        # a decode batch's queries and keys, out of the packed projection output
        dict(name="norm+rope 16 rows", op="rope", tokens=16, heads=28, kv_heads=4, dim=128, rot=128,
             interleaved=False, norm=True),
        # a long prompt, half of each head rotated
        dict(name="norm+rope prompt", op="rope", tokens=12345, heads=64, kv_heads=8, dim=128, rot=64,
             interleaved=False, norm=True),
        # one short request: latency
        dict(name="attend 1 short", op="attend", batch=1, new=1, max_len=333, spread=4, heads=28, kv_heads=4, dim=128,
             page=64, window=0),
        # an ordinary decode batch
        dict(name="attend 32 rows", op="attend", batch=32, new=1, max_len=4096, spread=5, heads=28, kv_heads=4,
             dim=128, page=64, window=0),
        # one request with a very long context: the work of few rows is split over the GPU
        dict(name="attend 1 long", op="attend", batch=1, new=1, max_len=200003, spread=6, heads=64, kv_heads=8,
             dim=128, page=128, window=0),
        # a large serving batch, ragged: the largest cache read
        dict(name="attend 96 long rows", op="attend", batch=96, new=1, max_len=16384, spread=7, heads=64, kv_heads=8,
             dim=128, page=64, window=0),
        # five drafted tokens a request are verified at once; small heads and pages, a sliding window
        dict(name="attend verify window", op="attend", batch=12, new=5, max_len=10000, spread=8, heads=32, kv_heads=8,
             dim=64, page=16, window=4095),
        # a chunk of two prompts against their context: bound by arithmetic, not by the cache
        dict(name="attend prompt chunk", op="attend", batch=2, new=700, max_len=6007, spread=9, heads=28, kv_heads=4,
             dim=128, page=32, window=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("append", "rope", "attend", "attend", "attend"))
    dim = rng.choice((64, 128, 128))
    group = rng.choice((1, 2, 4, 5, 7, 8, 16))
    kv_heads = rng.choice((1, 2, 4, 8))
    c = dict(op=op, heads=group * kv_heads, kv_heads=kv_heads, dim=dim)
    if op == "rope":
        c.update(tokens=_log(rng, 1, 12000), rot=rng.choice((dim, dim // 2)), interleaved=rng.random() < 0.5,
                 norm=rng.random() < 0.7)
        return c
    c.update(page=rng.choice((16, 32, 64, 128)), spread=rng.randrange(1 << 20))
    if op == "append":
        batch, new = (_log(rng, 1, 256), 1) if rng.random() < 0.5 else (_log(rng, 1, 8), _log(rng, 2, 1500))
        c.update(batch=batch, new=new, max_len=max(new, _log(rng, 32, 4000)), rot=rng.choice((dim, dim // 2)),
                 interleaved=rng.random() < 0.5, norm=rng.random() < 0.7)
        return c
    kind = rng.random()
    if kind < 0.6:
        batch, new = _log(rng, 1, 128), 1
    elif kind < 0.85:
        batch, new = _log(rng, 1, 32), rng.randint(2, 8)
    else:
        batch, new = rng.randint(1, 3), _log(rng, 20, 700)
    most = 12_000_000 // (batch * kv_heads) if new <= 8 else 8000
    max_len = max(new, min(_log(rng, 16, 150_000), most))
    c.update(batch=batch, new=new, max_len=max_len, window=rng.choice((0, 0, 1023)) if max_len > 1500 else 0)
    return c


def _lengths(c):
    """New tokens and length (with them) of every sequence: the case's own, whatever the seed of the values."""
    r = random.Random(c["spread"])
    new = [c["new"] if c["new"] <= 8 else r.randint(max(1, c["new"] // 2), c["new"]) for _ in range(c["batch"])]
    lens = [max(n, c["max_len"] if i == 0 else r.randint(1, c["max_len"])) for i, n in enumerate(new)]
    return new, lens


def _keys(c, n, length, i):
    """Positions [lo, hi) that the i-th of n new tokens attends to."""
    hi = length - n + i + 1
    return (max(0, hi - c["window"]) if c["window"] else 0), hi


def work(c):
    d, h, hk = c["dim"], c["heads"], c["kv_heads"]
    if c["op"] == "rope":
        t = c["tokens"]
        return {"bytes": 2 * 2 * t * (h + hk) * d + 4 * t * (c["rot"] + 1), "flops": 10 * t * (h + hk) * d}
    new, lens = _lengths(c)
    t = sum(new)
    if c["op"] == "append":
        pages = sum((l - 1) // c["page"] - (l - n) // c["page"] + 1 for n, l in zip(new, lens))
        return {"bytes": t * (2 * 2 * h * d + 2 * hk * (2 * d + d) + 4 * c["rot"]) + pages * (4 + 16 * hk),
                "flops": 10 * t * (h + 2 * hk) * d}
    # keys and values that some new token attends to, once each; their pages' scales and table entries
    seen = sum(l - _keys(c, n, l, 0)[0] for n, l in zip(new, lens))
    pairs = sum(hi - lo for n, l in zip(new, lens) for lo, hi in (_keys(c, n, l, i) for i in range(n)))
    return {"bytes": 2 * seen * hk * d + seen // c["page"] * (8 * hk + 4) + 2 * 2 * t * h * d,
            "flops": 4 * pairs * h * d}


# ----------------------------------------------------------------- inputs
def _randn(g, *shape):
    return torch.randn(*shape, device="cuda", generator=g)


def _pow2(e):
    """2^e as FP32, exactly, for whole e (2^-126 below that)."""
    return ((e.clamp(-126, 127).int() + 127) << 23).view(torch.float32)


def _table(rows, rot):
    """Row p: cos, then sin, of p theta^(-2i/rot)."""
    inv = THETA ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)
    a = torch.arange(rows, device="cuda", dtype=torch.float64)[:, None] * inv
    return torch.cat([a.cos(), a.sin()], 1).float()


def _fill(g, pages, hk, page, dim):
    """Codes and scales of a cache in use: every page and head has values of its own size."""
    codes = torch.empty(pages, hk, page, dim, dtype=torch.float8_e4m3fn, device="cuda")
    scale = torch.empty(pages, hk, device="cuda")
    step = max(1, (1 << 26) // (hk * page * dim))
    for p in range(0, pages, step):
        n = min(step, pages - p)
        x = _randn(g, n, hk, page, dim) * torch.exp2(_randn(g, n, hk))[:, :, None, None]
        m, e = torch.frexp(x.abs().amax((2, 3)))
        e = e - 9 + (m > 0.875)
        codes[p:p + n] = (x * _pow2(-e)[:, :, None, None]).to(torch.float8_e4m3fn)
        scale[p:p + n] = _pow2(e)
    return codes, scale


def prepare(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    d, h, hk = c["dim"], c["heads"], c["kv_heads"]
    s = {"case": c}
    if c["op"] != "attend":
        s["weights"] = [(1 + 0.2 * _randn(g, d)).bfloat16() if c["norm"] else None for _ in range(2)]
    if c["op"] == "rope":
        t = c["tokens"]
        qkv = _randn(g, t, h + 2 * hk, d).bfloat16()  # the projection's packed output
        s["q_in"], s["k_in"] = qkv[:, :h], qkv[:, h:h + hk]
        s["positions"] = torch.randint(0, 32768, (t,), device="cuda", generator=g, dtype=torch.int32)
        s["table"] = _table(32768, c["rot"])
        s["q_out"] = torch.empty(t, h, d, device="cuda", dtype=torch.bfloat16)
        s["k_out"] = torch.empty(t, hk, d, device="cuda", dtype=torch.bfloat16)
    else:
        new, lens = _lengths(c)
        need = [-(-l // c["page"]) for l in lens]
        pages = sum(need) + 3
        order = torch.randperm(pages, device="cuda", generator=g).int()
        table = torch.zeros(c["batch"], max(need), dtype=torch.int32, device="cuda")
        at = 0
        for i, n in enumerate(need):
            table[i, :n] = order[at:at + n]
            at += n
        s["block_table"] = table
        s["seq_len"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        s["q_start"] = torch.tensor([sum(new[:i]) for i in range(len(new) + 1)], dtype=torch.int32, device="cuda")
        s["tokens"], s["max_new"] = sum(new), max(new)
        s["k"], s["k_scale"] = _fill(g, pages, hk, c["page"], d)
        s["v"], s["v_scale"] = _fill(g, pages, hk, c["page"], d)
        if c["op"] == "append":
            s["table"] = _table(max(lens), c["rot"])
            qkv = _randn(g, s["tokens"], h + 2 * hk, d).mul_(torch.exp2(_randn(g, s["tokens"], 1, 1))).bfloat16()
            s["q_in"], s["k_in"], s["v_in"] = qkv.split((h, hk, hk), 1)
            s["q_out"] = torch.empty(s["tokens"], h, d, device="cuda", dtype=torch.bfloat16)
        else:
            s["q"] = _randn(g, s["tokens"], h, d).bfloat16()
            s["out"] = torch.empty_like(s["q"])
    if own:  # the handles that a program keeps for its cache, its batch and its rotation
        import skinny_bf16_gemm_residual_gb300 as sgr

        if c["op"] != "attend":
            s["rope"] = sgr.RopeNorm(s["table"], q_weight=s["weights"][0], k_weight=s["weights"][1], eps=EPS,
                                     interleaved=c["interleaved"])
        if c["op"] != "rope":
            s["cache"] = sgr.KvCache(s["k"], s["v"], s["k_scale"], s["v_scale"])
            s["batch"] = sgr.KvBatch(s["block_table"], s["seq_len"], s["q_start"], tokens=s["tokens"],
                                     max_new=s["max_new"])
        if c["op"] == "attend":
            s["workspace"] = sgr.kv_attention_workspace(s["cache"], s["batch"], h)
    return s


# -------------------------------------------------------------------- run
def run(s):
    c = s["case"]
    if own:
        import skinny_bf16_gemm_residual_gb300 as sgr

        if c["op"] == "rope":
            sgr.sgr_qk_norm_rope(s["q_in"], s["k_in"], s["positions"], s["rope"], q_out=s["q_out"], k_out=s["k_out"])
            return {"q": s["q_out"], "k": s["k_out"]}
        if c["op"] == "append":
            sgr.sgr_kv_append(s["cache"], s["batch"], s["k_in"], s["v_in"], s["rope"], q=s["q_in"], q_out=s["q_out"])
            return {"q": s["q_out"], "k": s["k"], "v": s["v"], "k_scale": s["k_scale"], "v_scale": s["v_scale"]}
        return sgr.sgr_kv_attention(s["cache"], s["batch"], s["q"], out=s["out"], window=c["window"],
                                    workspace=s["workspace"])
    return {"rope": _plain_rope, "append": _plain_append, "attend": _plain_attend}[c["op"]](s, c)


def _norm_rope(x, weight, pos, s, c):
    """[tokens, heads, dim] BF16 -> FP32: RMS norm of each head, then the rotation of its first `rot` elements."""
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * weight.float()
    rot = c["rot"]
    row = s["table"][pos.long()][:, None]
    cos, sin = row[..., :rot // 2], row[..., rot // 2:]
    if c["interleaved"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turned, x[..., rot:]], -1)


def _plain_rope(s, c):
    return {"q": _norm_rope(s["q_in"], s["weights"][0], s["positions"], s, c).bfloat16(),
            "k": _norm_rope(s["k_in"], s["weights"][1], s["positions"], s, c).bfloat16()}


def _plain_append(s, c):
    page = c["page"]
    start, length = s["q_start"].long(), s["seq_len"].long()
    row = torch.arange(s["tokens"], device="cuda")
    seq = torch.searchsorted(start[1:], row, right=True)
    first = length - (start[1:] - start[:-1])  # position of each sequence's first new token
    pos = first[seq] + row - start[seq]
    slot, off = s["block_table"][seq, pos // page].long(), pos % page
    kept = s["block_table"].long().gather(1, (first // page)[:, None])[:, 0]  # pages that may hold older tokens
    older = torch.arange(page, device="cuda") < (first % page)[:, None]
    out = {"q": _norm_rope(s["q_in"], s["weights"][0], pos, s, c).bfloat16()}
    k = _norm_rope(s["k_in"], s["weights"][1], pos, s, c)
    for name, x in (("k", k), ("v", s["v_in"].float())):
        codes, scale = s[name], s[name + "_scale"]
        top = torch.zeros_like(scale).index_reduce_(0, slot, x.abs().amax(-1), "amax")
        m, e = torch.frexp(top)
        e = torch.where(top > 0, (e - 9 + (m > 0.875)).clamp(E_MIN, E_MAX), E_MIN)
        was = torch.frexp(scale[kept])[1] - 1
        e_kept = torch.where((first % page > 0)[:, None], torch.maximum(e[kept], was), e[kept])
        e.index_copy_(0, kept, e_kept.to(e.dtype))
        old = codes.view(torch.uint8)[kept]
        again = old.view(torch.float8_e4m3fn).float() * _pow2(was - e_kept)[:, :, None, None]
        again = again.to(torch.float8_e4m3fn).view(torch.uint8)
        codes.view(torch.uint8).index_copy_(0, kept, torch.where(older[:, None, :, None], again, old))
        q = (x * _pow2(-e[slot])[:, :, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
        codes.view(torch.uint8)[slot, :, off] = q.view(torch.uint8)
        scale.index_copy_(0, slot, _pow2(e)[slot])
        out[name], out[name + "_scale"] = codes, scale
    return out


def _plain_attend(s, c):
    h, hk, d, page = c["heads"], c["kv_heads"], c["dim"], c["page"]
    b, group = c["batch"], h // hk
    start, length = s["q_start"].long(), s["seq_len"].long()
    n = start[1:] - start[:-1]
    i = torch.arange(s["max_new"], device="cuda")
    at = (start[:-1, None] + i).clamp(max=s["tokens"] - 1)
    q = s["q"][at].float().view(b, -1, hk, group, d).permute(0, 2, 3, 1, 4).reshape(b, hk, -1, d)
    table = s["block_table"].long()

    def cached(name):
        x = s[name].view(torch.uint8)[table].view(torch.float8_e4m3fn).float()
        x.mul_(s[name + "_scale"][table][..., None, None])
        return x.transpose(1, 2).reshape(b, hk, -1, d)

    p = q @ cached("k").transpose(-1, -2) * (1 / math.sqrt(d))
    key = torch.arange(table.shape[1] * page, device="cuda")
    last = length[:, None] - n[:, None] + i  # position of each new token
    seen = key <= last[..., None]
    if c["window"]:
        seen = seen & (key > last[..., None] - c["window"])
    seen = seen[:, None].expand(b, group, -1, -1).reshape(b, 1, -1, key.shape[0])
    p = p.masked_fill_(~seen, -math.inf)
    p = torch.exp(p.sub_(p.amax(-1, keepdim=True)))
    o = p @ cached("v") / p.sum(-1, keepdim=True)
    o = o.view(b, hk, group, -1, d).permute(0, 3, 1, 2, 4).reshape(b, -1, h, d).bfloat16()
    row = torch.arange(s["tokens"], device="cuda")
    seq = torch.searchsorted(start[1:], row, right=True)
    return o[seq, row - start[seq]]


# ------------------------------------------------------------------ exact
def _e4m3(x):
    """Nearest E4M3 value, ties to even, in 64 bits (|x| <= 448)."""
    quantum = torch.exp2((torch.frexp(x.abs())[1].double() - 4).clamp_min(-9))
    return torch.round(x / quantum) * quantum


def _turn64(x, weight, pos, s, c):
    x = x.double()
    if weight is not None:
        x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / c["dim"] + EPS) * weight.double()
    half = c["rot"] // 2
    i = torch.arange(half, device="cuda")
    a, b = (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + half)
    cos, sin = s["table"].double()[pos.long(), None, :half], s["table"].double()[pos.long(), None, half:]
    y = x.clone()
    y[..., a] = x[..., a] * cos - x[..., b] * sin
    y[..., b] = x[..., a] * sin + x[..., b] * cos
    return y


def exact(c, seed):
    s = prepare(c, seed)
    h, hk = c["heads"], c["kv_heads"]
    if c["op"] == "rope":
        return {"q": _turn64(s["q_in"], s["weights"][0], s["positions"], s, c),
                "k": _turn64(s["k_in"], s["weights"][1], s["positions"], s, c)}
    page, (new, lens) = c["page"], _lengths(c)
    table, row = s["block_table"].tolist(), 0
    if c["op"] == "append":
        pos = torch.cat([torch.arange(l - n, l, device="cuda") for n, l in zip(new, lens)])
        out = {"q": _turn64(s["q_in"], s["weights"][0], pos, s, c)}
        k = _turn64(s["k_in"], s["weights"][1], pos, s, c)
        for name, x in (("k", k), ("v", s["v_in"].double())):
            codes, scale = s[name].double(), s[name + "_scale"].double()
            row = 0
            for b, (n, l) in enumerate(zip(new, lens)):
                for p in range((l - n) // page, (l - 1) // page + 1):
                    lo, hi = max(p * page, l - n), min((p + 1) * page, l)
                    at, part = table[b][p], x[row + lo - (l - n):row + hi - (l - n)].transpose(0, 1)
                    top = part.abs().amax((1, 2))
                    m, e = torch.frexp((top / 448).clamp_min(2.0 ** E_MIN))
                    e = (e - (m == 0.5).int()).clamp(E_MIN, E_MAX).double()
                    if lo > p * page:
                        was = torch.frexp(scale[at])[1].double() - 1
                        e = torch.maximum(e, was)
                        before = codes[at, :, :lo - p * page]
                        codes[at, :, :lo - p * page] = _e4m3(before * torch.exp2(was - e)[:, None, None])
                    scale[at] = torch.exp2(e)
                    codes[at, :, lo - p * page:hi - p * page] = _e4m3(part / scale[at][:, None, None])
                row += n
            out[name], out[name + "_scale"] = codes, scale
        return out
    out = torch.empty(s["tokens"], h, c["dim"], dtype=torch.float64, device="cuda")
    for b, (n, l) in enumerate(zip(new, lens)):
        used = torch.tensor(table[b][:-(-l // page)], device="cuda")
        k, v = ((s[m].view(torch.uint8)[used].view(torch.float8_e4m3fn).double()
                 * s[m + "_scale"][used].double()[:, :, None, None]).transpose(0, 1).flatten(1, 2)[:, :l]
                for m in ("k", "v"))
        q = s["q"][row:row + n].double().view(n, hk, h // hk, -1)
        score = torch.einsum("nkgd,ktd->kgnt", q, k) / math.sqrt(c["dim"])
        t = torch.arange(l, device="cuda")
        at = torch.arange(l - n, l, device="cuda")[:, None]
        hidden = (t > at) | (t <= at - c["window"]) if c["window"] else t > at
        weights = torch.softmax(score.masked_fill(hidden, -math.inf), -1)
        out[row:row + n] = torch.einsum("kgnt,ktd->nkgd", weights, v).reshape(n, h, -1)
        row += n
    return out
