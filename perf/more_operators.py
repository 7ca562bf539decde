"""Measured cases of what long and drafted decoding needs beside plain attention over the paged E4M3 cache: attention
for trees of drafted tokens (``tree``), attention with a sliding window and first positions that stay visible
(``sinks``), the attention weight that every cached position gets, accumulated (``mass``), and the eviction of the
positions with the least of it (``evict``).

``run`` computes an operator in elementary 32-bit torch operations, or with ``own`` set through the library's calls;
``exact`` computes it in 64 bits, one sequence at a time, from the definition.
"""
import math
import random

import torch

own = False  # set by whoever measures: run() makes the library's calls

E_MIN, E_MAX = -64, 64  # exponents of the page scales


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one request verifies a small tree of drafted tokens: latency
        dict(name="tree 1 x 7", op="tree", batch=1, new=7, max_len=700, spread=1, heads=28, kv_heads=4, dim=128,
             page=64, window=0, sinks=0),
        # an ordinary batch of trees; small heads and pages
        dict(name="tree 16 x 25", op="tree", batch=16, new=25, max_len=5000, spread=2, heads=32, kv_heads=8, dim=64,
             page=16, window=0, sinks=0),
        # wide trees over long contexts, under a sliding window with sinks: bound by arithmetic
        dict(name="tree 6 x 129 window", op="tree", batch=6, new=129, max_len=40000, spread=3, heads=64, kv_heads=8,
             dim=128, page=128, window=16384, sinks=4),
        # one request that has streamed far past its window: latency
        dict(name="sinks 1 row", op="sinks", batch=1, new=1, max_len=9001, spread=4, heads=28, kv_heads=4, dim=128,
             page=64, window=1020, sinks=4),
        # a large streaming batch, ragged
        dict(name="sinks 96 rows", op="sinks", batch=96, new=1, max_len=20000, spread=5, heads=64, kv_heads=8, dim=128,
             page=64, window=8188, sinks=4),
        # chunks of two prompts; a system prompt of odd length stays visible
        dict(name="sinks prompt chunk", op="sinks", batch=2, new=700, max_len=9007, spread=6, heads=28, kv_heads=4,
             dim=128, page=32, window=2047, sinks=333),
        # one short request's weights: latency
        dict(name="mass 1 short", op="mass", batch=1, new=1, max_len=333, spread=7, heads=28, kv_heads=4, dim=128,
             page=64, window=0, sinks=0),
        # the weights of a large decode batch, ragged
        dict(name="mass 64 rows", op="mass", batch=64, new=1, max_len=16384, spread=8, heads=64, kv_heads=8, dim=128,
             page=64, window=0, sinks=0),
        # those of a chunk of two prompts: bound by exponentials
        dict(name="mass prompt chunk", op="mass", batch=2, new=500, max_len=4001, spread=9, heads=32, kv_heads=8, dim=64,
             page=16, window=0, sinks=0),
        # one request falls back to its budget
        dict(name="evict 1 short", op="evict", batch=1, max_len=1100, keep=1000, first=4, recent=256, spread=10,
             kv_heads=4, dim=128, page=64),
        # a prompt of a long document is cut to an eighth
        dict(name="evict 1 long", op="evict", batch=1, max_len=130001, keep=16250, first=4, recent=1000, spread=11,
             kv_heads=8, dim=128, page=128),
        # a serving batch falls back to its budget, ragged; small heads and pages
        dict(name="evict 48", op="evict", batch=48, max_len=8000, keep=4000, first=16, recent=500, spread=12,
             kv_heads=8, dim=64, page=16),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("tree", "sinks", "mass", "evict"))
    kv_heads = rng.choice((1, 2, 4, 8))
    c = dict(op=op, kv_heads=kv_heads, dim=rng.choice((64, 128, 128)), page=rng.choice((16, 32, 64, 128)),
             spread=rng.randrange(1 << 20))
    if op == "evict":
        batch = _log(rng, 1, 64)
        max_len = min(_log(rng, 16, 130_000), 4_000_000 // (batch * kv_heads))
        keep = max(1, int(max_len * rng.uniform(0.05, 0.9)))
        c.update(batch=batch, max_len=max_len, keep=keep, first=rng.choice((0, 4, 33)), recent=int(keep * rng.uniform(0, 0.5)))
        return c
    group = rng.choice((1, 2, 4, 5, 7, 8, 16))
    kind = rng.random()
    if op == "tree":
        batch, new = _log(rng, 1, 24), _log(rng, 2, 150)
    elif kind < 0.6:
        batch, new = _log(rng, 1, 96), 1
    elif kind < 0.8:
        batch, new = _log(rng, 1, 32), rng.randint(2, 9)
    else:
        batch, new = rng.randint(1, 3), _log(rng, 20, 600)
    most = 10_000_000 // (batch * kv_heads) if new <= 9 else 500_000_000 // (batch * new * group * kv_heads)
    max_len = max(new, min(_log(rng, 16, 120_000), most))
    windowed = op == "sinks" or rng.random() < 0.3
    c.update(batch=batch, new=new, max_len=max_len, heads=group * kv_heads,
             window=_log(rng, 16, 9000) if windowed else 0, sinks=rng.choice((1, 4, 4, 29, 260)) if windowed else 0)
    return c


def _lengths(c):
    """New tokens and length (with them) of every sequence: the case's own, whatever the seed of the values."""
    r = random.Random(c["spread"])
    if c["op"] == "evict":
        return None, [c["max_len"] if i == 0 else r.randint(max(1, c["max_len"] // 2), c["max_len"]) for i in range(c["batch"])]
    few = c["new"] <= 9
    new = [c["new"] if few or i == 0 else r.randint(max(1, c["new"] // 2), c["new"]) for i in range(c["batch"])]
    lens = [max(n, c["max_len"] if i == 0 else r.randint(1, c["max_len"])) for i, n in enumerate(new)]
    return new, lens


def _parents(c):
    """Each sequence's tree: the parent of every drafted token but the first (tokens come behind their parents)."""
    r = random.Random(c["spread"] + 1)
    return [[r.randrange(max(0, i - 12), i) for i in range(1, n)] for n in _lengths(c)[0]]


def _paths(parents):
    """For each drafted token the tokens from the root to it."""
    paths = [[0]]
    for i, p in enumerate(parents, 1):
        paths.append(paths[p] + [i])
    return paths


def _prefix(c, first, at):
    """Number of positions below `first` that a token at position `at` sees."""
    if not c["window"]:
        return first
    lo = max(0, at - c["window"] + 1)
    return max(0, first - lo) + min(lo, c["sinks"], first)


def work(c):
    d, hk, page = c["dim"], c["kv_heads"], c["page"]
    new, lens = _lengths(c)
    if c["op"] == "evict":
        kept = sum(min(c["keep"], l) for l in lens)
        pages = sum(-(-l // page) + -(-min(c["keep"], l) // page) for l in lens)
        return {"bytes": hk * (4 * sum(lens) + kept * (2 * 2 * d + 4 + 4)) + pages * (4 + 8 * hk), "flops": 2 * d * hk * kept}
    h, seen, pairs = c["heads"], 0, 0
    paths = [_paths(p) for p in _parents(c)] if c["op"] == "tree" else None
    for b, (n, l) in enumerate(zip(new, lens)):
        first = l - n
        # positions that some new token sees, once each: those of the first one, and the new ones
        seen += _prefix(c, first, first) + n
        for i in range(n):
            at, mine = (first + len(paths[b][i]) - 1, len(paths[b][i])) if paths else (first + i, None)
            if mine is None:
                lo = max(0, at - c["window"] + 1) if c["window"] else 0
                mine = at + 1 - max(first, lo) + (min(lo, c["sinks"]) - first if min(lo, c["sinks"]) > first else 0)
            pairs += _prefix(c, first, at) + mine
    t = sum(new)
    if c["op"] == "mass":
        return {"bytes": seen * hk * d + seen // page * (4 * hk + 4) + 8 * hk * seen - 4 * hk * t + t * h * (2 * d + 4),
                "flops": 2 * pairs * h * d}
    words = -(-c["new"] // 64) if c["op"] == "tree" else 0
    return {"bytes": 2 * seen * hk * d + seen // page * (8 * hk + 4) + 2 * 2 * t * h * d + 8 * words * t,
            "flops": 4 * pairs * h * d}


# ----------------------------------------------------------------- inputs
def _randn(g, *shape):
    return torch.randn(*shape, device="cuda", generator=g)


def _pow2(e):
    """2^e as FP32, exactly, for whole e (2^-126 below that)."""
    return ((e.clamp(-126, 127).int() + 127) << 23).view(torch.float32)


def _fill(g, pages, hk, page, dim):
    """Codes and scales of a cache in use: every page and head has values of its own size."""
    codes = torch.empty(pages, hk, page, dim, dtype=torch.float8_e4m3fn, device="cuda")
    scale = torch.empty(pages, hk, device="cuda")
    step = max(1, (1 << 26) // (hk * page * dim))
    for p in range(0, pages, step):
        n = min(step, pages - p)
        x = _randn(g, n, hk, page, dim) * torch.exp2(0.5 * _randn(g, n, hk))[:, :, None, None]
        m, e = torch.frexp(x.abs().amax((2, 3)))
        e = e - 9 + (m > 0.875)
        codes[p:p + n] = (x * _pow2(-e)[:, :, None, None]).to(torch.float8_e4m3fn)
        scale[p:p + n] = _pow2(e)
    return codes, scale


def _tables(g, *needs):
    """Block tables of sequences that need so many pages each, out of one shuffled cache, and its size."""
    pages = sum(sum(n) for n in needs) + 3
    order, at, out = torch.randperm(pages, device="cuda", generator=g).int().tolist(), 0, []
    for need in needs:
        table = torch.zeros(len(need), max(need), dtype=torch.int32)
        for i, n in enumerate(need):
            table[i, :n] = torch.tensor(order[at:at + n], dtype=torch.int32)
            at += n
        out.append(table.cuda())
    return out, pages


def prepare(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    d, hk, page = c["dim"], c["kv_heads"], c["page"]
    new, lens = _lengths(c)
    s = {"case": c}
    need = [-(-l // page) for l in lens]
    if c["op"] == "evict":
        (s["block_table"], s["new_table"]), pages = _tables(g, need, [-(-min(c["keep"], l) // page) for l in lens])
        # what positions have gathered: few have much, many next to nothing, some the same
        s["mass"] = torch.exp(3 * _randn(g, pages, hk, page))
        s["mass"] = torch.where(_randn(g, pages, hk, page) > 1, torch.floor(s["mass"]), s["mass"])
        s["keep"] = torch.full((c["batch"],), c["keep"], dtype=torch.int32, device="cuda")
        s["new_len"] = torch.zeros(c["batch"], dtype=torch.int32, device="cuda")
        s["kept"] = torch.full((c["batch"], hk, s["new_table"].shape[1] * page), -1, dtype=torch.int32, device="cuda")
        new = [1] * len(lens)
    else:
        (s["block_table"],), pages = _tables(g, need)
    s["seq_len"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    s["q_start"] = torch.tensor([sum(new[:i]) for i in range(len(new) + 1)], dtype=torch.int32, device="cuda")
    s["tokens"], s["max_new"] = sum(new), max(new)
    s["k"], s["k_scale"] = _fill(g, pages, hk, page, d)
    s["v"], s["v_scale"] = _fill(g, pages, hk, page, d) if c["op"] != "mass" else (s["k"].clone(), s["k_scale"].clone())
    if c["op"] != "evict":
        s["q"] = _randn(g, s["tokens"], c["heads"], d).bfloat16()
        s["tree"] = None
    if c["op"] == "tree":
        words = -(-s["max_new"] // 64)
        rows = [[sum(1 << (j - 64 * w) for j in path if j // 64 == w) for w in range(words)]
                for parents in _parents(c) for path in _paths(parents)]
        s["tree"] = torch.tensor([[x - (1 << 64) if x >> 63 else x for x in r] for r in rows], device="cuda")
    if c["op"] == "mass":
        s["lse"] = torch.logsumexp(_scores(s, c).double(), -1).float()
        b, _, n = s["lse"].shape
        s["lse"] = s["lse"].view(b, hk, -1, s["max_new"]).permute(0, 3, 1, 2).reshape(b, s["max_new"], -1)[_rows(s)]
        # what a few calls like this one have left
        s["mass"] = torch.rand(pages, hk, page, device="cuda", generator=g) * (3 * c["new"] * c["heads"] / (hk * c["max_len"]))
    elif c["op"] != "evict":
        s["out"] = torch.empty_like(s["q"])
    if own:  # the handles that a program keeps for its cache and its batch
        import skinny_bf16_gemm_residual_gb300 as sgr

        s["cache"] = sgr.KvCache(s["k"], s["v"], s["k_scale"], s["v_scale"])
        s["batch"] = sgr.KvBatch(s["block_table"], s["seq_len"], s["q_start"], tokens=s["tokens"], max_new=s["max_new"])
        if c["op"] in ("tree", "sinks"):
            s["workspace"] = sgr.kv_attention_workspace(s["cache"], s["batch"], c["heads"])
        if c["op"] == "mass":
            s["workspace"] = sgr.kv_mass_workspace(s["cache"], s["batch"], c["heads"])
    return s


# -------------------------------------------------------------------- run
def run(s):
    c = s["case"]
    if own:
        import skinny_bf16_gemm_residual_gb300 as sgr

        if c["op"] == "mass":
            sgr.sgr_kv_mass(s["cache"], s["batch"], s["q"], s["lse"], s["mass"], window=c["window"], sinks=c["sinks"],
                            workspace=s["workspace"])
            return s["mass"]
        if c["op"] == "evict":
            sgr.sgr_kv_evict(s["cache"], s["batch"], s["mass"], s["keep"], s["new_table"], first=c["first"],
                             recent=c["recent"], new_len=s["new_len"], kept=s["kept"])
            return _evicted(s)
        return sgr.sgr_kv_attention(s["cache"], s["batch"], s["q"], out=s["out"], window=c["window"], sinks=c["sinks"],
                                    tree=s["tree"], workspace=s["workspace"])
    return {"tree": _plain_attend, "sinks": _plain_attend, "mass": _plain_mass, "evict": _plain_evict}[c["op"]](s, c)


def _evicted(s):
    return {n: s[n] for n in ("k", "v", "k_scale", "v_scale", "mass", "kept", "new_len")}


def _rows(s):
    """(sequence, place in it) of every row."""
    row = torch.arange(s["tokens"], device="cuda")
    seq = torch.searchsorted(s["q_start"][1:].long(), row, right=True)
    return seq, row - s["q_start"].long()[seq]


def _cached(s, c, name):
    """[batch, kv_heads, positions, dim] in FP32."""
    table = s["block_table"].long()
    x = s[name].view(torch.uint8)[table].view(torch.float8_e4m3fn).float()
    x.mul_(s[name + "_scale"][table][..., None, None])
    return x.transpose(1, 2).reshape(c["batch"], c["kv_heads"], -1, c["dim"])


def _scores(s, c):
    """Scaled scores [batch, kv_heads, group * new, positions], -inf where masked."""
    h, hk, d, b = c["heads"], c["kv_heads"], c["dim"], c["batch"]
    start, length = s["q_start"].long(), s["seq_len"].long()
    n = start[1:] - start[:-1]
    i = torch.arange(s["max_new"], device="cuda")
    at = (start[:-1, None] + i).clamp(max=s["tokens"] - 1)
    q = s["q"][at].float().view(b, -1, hk, h // hk, d).permute(0, 2, 3, 1, 4).reshape(b, hk, -1, d)
    key = torch.arange(s["block_table"].shape[1] * c["page"], device="cuda")
    first = (length - n)[:, None, None]
    if s["tree"] is not None:
        bits = s["tree"][at][..., None] >> torch.arange(64, device="cuda") & 1  # [batch, new, words, 64]
        bits = bits.flatten(2).bool()
        pos = first + bits.sum(-1, keepdim=True) - 1
        j = (key - first).expand(b, s["max_new"], -1)
        drafted = bits.gather(2, j.clamp(0, bits.shape[2] - 1)) & (j >= 0) & (j < n[:, None, None])
    else:
        pos = first + i[:, None]
        drafted = None
    seen = key <= pos
    if c["window"]:
        seen = seen & ((key > pos - c["window"]) | (key < c["sinks"]))
    if drafted is not None:
        seen = torch.where(key < first, seen, drafted)
    seen = seen & (i < n[:, None])[..., None]  # rows that fill up a shorter sequence
    seen = seen[:, None].expand(b, h // hk, -1, -1).reshape(b, 1, -1, key.shape[0])
    return (q @ _cached(s, c, "k").transpose(-1, -2)).mul_(1 / math.sqrt(d)).masked_fill_(~seen, -math.inf)


def _plain_attend(s, c):
    h, hk, d, b = c["heads"], c["kv_heads"], c["dim"], c["batch"]
    p = _scores(s, c)
    p = torch.exp(p.sub_(p.amax(-1, keepdim=True)))
    o = p @ _cached(s, c, "v") / p.sum(-1, keepdim=True)
    o = o.view(b, hk, h // hk, -1, d).permute(0, 3, 1, 2, 4).reshape(b, -1, h, d).bfloat16()
    return o[_rows(s)]


def _plain_mass(s, c):
    hk, b, n = c["kv_heads"], c["batch"], s["max_new"]
    start, length = s["q_start"].long(), s["seq_len"].long()
    at = (start[:-1, None] + torch.arange(n, device="cuda")).clamp(max=s["tokens"] - 1)
    lse = s["lse"][at].view(b, n, hk, -1).permute(0, 2, 3, 1).reshape(b, hk, -1, 1)
    w = torch.exp(_scores(s, c).sub_(lse)).sum(2)  # [batch, kv_heads, positions]
    t = torch.arange(w.shape[2], device="cuda")
    seq, t = (t < length[:, None]).nonzero(as_tuple=True)
    page, off = s["block_table"].long()[seq, t // c["page"]], t % c["page"]
    older = (t < (length - start[1:] + start[:-1])[seq])[:, None]
    s["mass"][page, :, off] = torch.where(older, s["mass"][page, :, off], 0) + w[seq, :, t]
    return s["mass"]


def _plain_evict(s, c):
    b, hk, page, d = c["batch"], c["kv_heads"], c["page"], c["dim"]
    table, to, length = s["block_table"].long(), s["new_table"].long(), s["seq_len"].long()[:, None, None]
    mass = s["mass"][table].transpose(1, 2).reshape(b, hk, -1)
    t = torch.arange(mass.shape[2], device="cuda")
    n = torch.minimum(s["keep"].long()[:, None, None], length)
    f = n.clamp(max=c["first"])
    r = (n - f).clamp(max=c["recent"])
    worth = mass.masked_fill((t < f) | (t >= length - r), math.inf).masked_fill_((t >= length), -math.inf)
    order = torch.sort(worth, dim=-1, descending=True, stable=True).indices  # of the same worth, the first
    room = to.shape[1] * page
    kept = torch.where(torch.arange(order.shape[2], device="cuda") < n, order, order.shape[2])
    kept = torch.nn.functional.pad(kept, (0, max(0, room - kept.shape[2])), value=order.shape[2])
    kept = torch.sort(kept, dim=-1).values[..., :room]
    there = torch.arange(room, device="cuda") < n  # [batch, 1, room]
    at = kept.clamp(max=t.shape[0] - 1)
    head = torch.arange(hk, device="cuda")[:, None]
    src, off = table[torch.arange(b, device="cuda")[:, None, None], at // page], at % page
    seq, hh, slot = there.expand(b, hk, -1).nonzero(as_tuple=True)
    dst = to[seq, slot // page]
    for name in ("k", "v"):
        codes, scale = s[name].view(torch.uint8), s[name + "_scale"]
        x = codes[src, head, off].view(torch.float8_e4m3fn).float() * scale[src, head][..., None]
        x = x.masked_fill_(~there[..., None], 0)
        top = x.view(b, hk, -1, page * d).abs().amax(-1)
        m, e = torch.frexp(top)
        e = torch.where(top > 0, (e - 9 + (m > 0.875)).clamp(E_MIN, E_MAX), E_MIN)
        x = (x.view(b, hk, -1, page * d) * _pow2(-e)[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
        codes[dst, hh, slot % page] = x.view(b, hk, -1, d)[seq, hh, slot]
        scale[dst, hh] = _pow2(e)[seq, hh, slot // page]
    s["mass"][dst, hh, slot % page] = mass.gather(2, at)[seq, hh, slot]
    s["kept"].copy_(torch.where(there, kept, s["kept"].long()))
    s["new_len"].copy_(n.flatten())
    return _evicted(s)


# ------------------------------------------------------------------ exact
def _e4m3(x):
    """Nearest E4M3 value, ties to even, in 64 bits (|x| <= 448)."""
    quantum = torch.exp2((torch.frexp(x.abs())[1].double() - 4).clamp_min(-9))
    return torch.round(x / quantum) * quantum


def _values(s, name, pages):
    """[kv_heads, positions, dim] of a sequence's pages, in 64 bits."""
    x = s[name].view(torch.uint8)[pages].view(torch.float8_e4m3fn).double()
    return (x * s[name + "_scale"][pages].double()[:, :, None, None]).transpose(0, 1).flatten(1, 2)


def _hidden(c, n, l, paths):
    """Which of l positions each of n new tokens does not see."""
    t, first = torch.arange(l, device="cuda"), l - n
    at = torch.tensor([first + len(p) - 1 for p in paths] if paths else list(range(first, l)), device="cuda")[:, None]
    hidden = t > at
    if c["window"]:
        hidden = hidden | ((t <= at - c["window"]) & (t >= c["sinks"]))
    if paths:
        hidden[:, first:] = True
        at = [(i, first + j) for i, p in enumerate(paths) for j in p]
        hidden[[i for i, _ in at], [j for _, j in at]] = False
    return hidden


def exact(c, seed):
    s = prepare(c, seed)
    hk, page, (new, lens) = c["kv_heads"], c["page"], _lengths(c)
    table = s["block_table"].tolist()
    if c["op"] == "evict":
        out = {n: s[n].double() for n in ("k", "v", "k_scale", "v_scale", "mass")}
        to = s["new_table"].tolist()
        for b, l in enumerate(lens):
            pages = torch.tensor(table[b][:-(-l // page)], device="cuda")
            mass = s["mass"][pages].transpose(0, 1).flatten(1)[:, :l].double()
            values = {name: _values(s, name, pages)[:, :l] for name in ("k", "v")}
            n = min(c["keep"], l)
            f = min(c["first"], n)
            r = min(c["recent"], n - f)
            middle = mass[:, f:l - r]
            # rank by value, then by position: sorted from the last position on, so that of equals the first comes last
            last = torch.sort(middle.flip(1), dim=1, stable=True).indices[:, middle.shape[1] - (n - f - r):]
            mark = torch.zeros(hk, l, dtype=torch.bool, device="cuda")
            mark[:, :f] = True
            mark[:, l - r:] = True
            mark.scatter_(1, f + middle.shape[1] - 1 - last, True)
            at = mark.nonzero()[:, 1].view(hk, n)
            for lo in range(0, n, page):
                part, p = at[:, lo:lo + page], to[b][lo // page]
                out["mass"][p, :, :part.shape[1]] = mass.gather(1, part)
                for name in ("k", "v"):
                    x = values[name].gather(1, part[..., None].expand(-1, -1, c["dim"]))
                    m, e = torch.frexp((x.abs().amax((1, 2)) / 448).clamp_min(2.0 ** E_MIN))
                    e = (e - (m == 0.5).int()).clamp(E_MIN, E_MAX).double()
                    out[name + "_scale"][p] = torch.exp2(e)
                    out[name][p, :, :part.shape[1]] = _e4m3(x / torch.exp2(e)[:, None, None])
        return {**out, "kept": None, "new_len": None}
    paths = [_paths(p) for p in _parents(c)] if c["op"] == "tree" else [None] * len(new)
    out = s["mass"].double() if c["op"] == "mass" else torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    row = 0
    for b, (n, l) in enumerate(zip(new, lens)):
        used = torch.tensor(table[b][:-(-l // page)], device="cuda")
        q = s["q"][row:row + n].double().view(n, hk, c["heads"] // hk, -1)
        hidden = _hidden(c, n, l, paths[b])
        for h in range(hk):
            score = torch.einsum("ngd,td->gnt", q[:, h], _values(s, "k", used)[h, :l]) / math.sqrt(c["dim"])
            score = score.masked_fill_(hidden, -math.inf)
            if c["op"] == "mass":
                lse = s["lse"][row:row + n].double().view(n, hk, -1)[:, h]
                w = torch.exp(score - lse.t()[..., None]).sum((0, 1))
                pos = torch.arange(l, device="cuda")
                slots = out[:, h]
                at = used[pos // page], pos % page
                slots[at] = torch.where(pos < l - n, slots[at], 0) + w
            else:
                weights = torch.softmax(score, -1)
                out[row:row + n, h * (c["heads"] // hk):(h + 1) * (c["heads"] // hk)] = torch.einsum(
                    "gnt,td->ngd", weights, _values(s, "v", used)[h, :l])
        row += n
    return out
