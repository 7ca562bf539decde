"""The attention operators' definitions in 64 bits (torch float64 on the CPU,
one sequence and one page at a time), seeded inputs for their tests, and the
error bounds that the tests hold the kernels to."""
from __future__ import annotations

import math

import torch

E_MIN, E_MAX = -64, 64
NAN_CODE = 0x7F


def e4m3_values():
    """Value of each of the 256 codes."""
    return torch.arange(256, dtype=torch.int32).to(torch.uint8).view(torch.float8_e4m3fn).double()


def quantum(x):
    """Spacing of the E4M3 values around |x| (|x| < 464)."""
    e = torch.frexp(x.abs().clamp_min(2.0 ** -30))[1].double() - 1
    return torch.exp2((e - 3).clamp_min(-9))


def norm_rope(x, weight, pos, table, interleaved, eps):
    """x [tokens, heads, dim] (float64 values of BF16), pos [tokens]."""
    x = x.double()
    if weight is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * weight.double()
    if table is None:
        return x
    rot = table.shape[1]
    half = rot // 2
    i = torch.arange(half)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    row = table.double()[pos.long().clamp(0, table.shape[0] - 1)][:, None]
    cos, sin = row[..., :half], row[..., half:]
    y = x.clone()
    y[..., a] = x[..., a] * cos - x[..., b] * sin
    y[..., b] = x[..., b] * cos + x[..., a] * sin
    return y


def rope_table(rows, rot):
    inv = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    a = torch.arange(rows, dtype=torch.float64)[:, None] * inv
    return torch.cat([a.cos(), a.sin()], 1).float()


def rows_of(q_start, b):
    return (b, b + 1) if q_start is None else (int(q_start[b]), int(q_start[b + 1]))


def scale_exp(top):
    """Smallest e in [-64, 64] with top <= 448 2^e."""
    if top == 0:
        return E_MIN
    m, e = math.frexp(top / 448.0)
    return min(max(e - (1 if m == 0.5 else 0), E_MIN), E_MAX)


def append(codes, scale, x, block_table, seq_len, q_start, page_size):
    """One of k, v: codes [pages, heads, page_size, dim] uint8, scale [pages,
    heads], x [tokens, heads, dim] float64.  Returns the cache's values before
    rounding where the call writes (NaN elsewhere) and the scales after it."""
    table = e4m3_values()
    want = torch.full(codes.shape, math.nan, dtype=torch.float64)
    scale = scale.double().clone()
    for b in range(len(seq_len)):
        r0, r1 = rows_of(q_start, b)
        n, length = r1 - r0, int(seq_len[b])
        for block in range(max(length - n, 0) // page_size, (length - 1) // page_size + 1 if length and n else 0):
            t0, t1 = max(block * page_size, length - n, 0), min((block + 1) * page_size, length)
            if t1 <= t0:
                continue
            page, off = int(block_table[b, block]), t0 - block * page_size
            for h in range(codes.shape[1]):
                part = x[r0 + t0 - (length - n):r0 + t1 - (length - n), h]
                finite = part[torch.isfinite(part)].abs()
                e = scale_exp(float(finite.max()) if finite.numel() else 0.0)
                if off:
                    was = int(math.log2(float(scale[page, h])))
                    e = max(e, was)
                    want[page, h, :off] = table[codes[page, h, :off].long()] * 2.0 ** was
                scale[page, h] = 2.0 ** e
                want[page, h, off:off + t1 - t0] = part
    return want, scale


def attention(q, k, v, block_table, seq_len, q_start, page_size, scale, window):
    """q [tokens, heads, dim]; k, v [pages, kv_heads, page_size, dim] float64
    values (whatever lies behind a sequence's end is not looked at).  Returns
    the outputs and, for the error bound, sum p |v| / sum p."""
    out = torch.zeros(q.shape, dtype=torch.float64)
    mag = torch.zeros(q.shape, dtype=torch.float64)
    hk = k.shape[1]
    for b in range(len(seq_len)):
        r0, r1 = rows_of(q_start, b)
        length = int(seq_len[b])
        for r in range(r0, r1):
            pos = length - (r1 - r0) + r - r0
            lo = max(0, pos - window + 1) if window else 0
            if pos < lo:
                continue
            t = torch.arange(lo, pos + 1)
            pages = block_table[b].long()[t // page_size]
            kk, vv = k[pages, :, t % page_size], v[pages, :, t % page_size]  # [t, hk, dim]
            qq = q[r].double().view(hk, -1, q.shape[-1])
            p = torch.softmax(torch.einsum("kgd,tkd->kgt", qq, kk) * scale, -1)
            out[r] = torch.einsum("kgt,tkd->kgd", p, vv).reshape(q.shape[1:])
            mag[r] = torch.einsum("kgt,tkd->kgd", p, vv.abs()).reshape(q.shape[1:])
    return out, mag


# ------------------------------------------------------------------ error bounds
def check_bf16(got, want, what=""):
    """Rounded once: half a BF16 ulp (2^-9 of the value), twice that allowed,
    and the 32-bit arithmetic's error of some 2^-21 of the row's largest value."""
    got = got.double().cpu()
    tol = 2.0 ** -8 * want.abs() + 2.0 ** -20 * want.abs().amax(-1, keepdim=True)
    bad = ~((got - want).abs() <= tol)
    bad &= ~(got.isnan() & want.isnan())
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, first {tuple(bad.nonzero()[0].tolist())}"


def check_attention(got, want, mag, what=""):
    """BF16 rounding (2^-8 of the value, twice half an ulp) and, on the sum
    p |v|: the weights p held to 8 bits (2^-8 at most) and the scores to about
    2^-10 (q in 8 bits and 32-bit sums), together below 2^-7."""
    got = got.double().cpu()
    tol = 2.0 ** -8 * want.abs() + 2.0 ** -7 * mag
    bad = ~((got - want).abs() <= tol)
    bad &= ~(got.isnan() & want.isnan())
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} off, first {tuple(bad.nonzero()[0].tolist())}: "
                           f"got {got[bad][0]} want {want[bad][0]}")


def check_append(got_codes, got_scale, before, want, want_scale, what=""):
    """Scales equal; each code the nearest of its neighbours (half a spacing,
    with 2^-10 of it for values whose 32-bit form lies across a tie); what the
    call does not write is unchanged."""
    assert torch.equal(got_scale.double().cpu(), want_scale), f"{what}: scales"
    codes = got_codes.cpu()
    still = want.isnan()
    values = e4m3_values()[codes.long()] * want_scale[:, :, None, None]
    x = (want / want_scale[:, :, None, None]).nan_to_num(0.0).clamp(-448, 448)
    step = quantum(x) * want_scale[:, :, None, None]
    bad = ~still & ~((values - x * want_scale[:, :, None, None]).abs() <= step * (0.5 + 2.0 ** -10))
    assert not bad.any(), f"{what}: {int(bad.sum())} codes, first {tuple(bad.nonzero()[0].tolist())}"
    assert torch.equal(codes[still], before[still]), f"{what}: codes that the call does not write"


# ------------------------------------------------------------------------ inputs
class Problem:
    """A cache in use and the sequences of a call.  Whatever no sequence may
    see -- pages of nobody, positions behind a sequence's end, their scales --
    holds NaN."""

    def __init__(self, dim, page, hk, lens, new, seed=0, heads_inside=False, extra_pages=2):
        g = torch.Generator().manual_seed(seed)
        self.dim, self.page, self.hk, self.lens, self.new = dim, page, hk, lens, new
        need = [-(-l // page) for l in lens]
        self.pages = sum(need) + extra_pages
        order = torch.randperm(self.pages, generator=g).int()
        self.max_pages = max(need + [1])
        self.block_table = torch.full((len(lens), self.max_pages), -1, dtype=torch.int32)
        self.codes, self.scale = [], []
        live = torch.zeros(self.pages, page, dtype=torch.bool)
        at = 0
        for b, n in enumerate(need):
            self.block_table[b, :n] = order[at:at + n]
            for i in range(n):
                live[order[at + i], :min(page, lens[b] - i * page)] = True
            at += n
        for _ in range(2):
            x = torch.randn(self.pages, hk, page, dim, generator=g) * torch.exp2(torch.randn(self.pages, hk, 1, 1, generator=g))
            top = x.abs().amax((2, 3))
            e = torch.tensor([[scale_exp(float(t)) for t in row] for row in top])
            codes = (x * torch.exp2(-e[:, :, None, None].float())).to(torch.float8_e4m3fn).view(torch.uint8)
            codes[~live[:, None, :, None].expand_as(codes)] = NAN_CODE
            scale = torch.exp2(e.float())
            scale[~live.any(1)] = math.nan
            if heads_inside:  # [pages, page, heads, dim] in memory
                codes = codes.transpose(1, 2).contiguous().transpose(1, 2)
            self.codes.append(codes)
            self.scale.append(scale)
        self.seq_len = torch.tensor(lens, dtype=torch.int32)
        self.q_start = torch.tensor([sum(new[:i]) for i in range(len(new) + 1)], dtype=torch.int32)
        self.tokens, self.max_new = sum(new), max(new + [1])
        self.g = g

    def randn(self, *shape):
        return torch.randn(*shape, generator=self.g)

    def values(self, i):
        return e4m3_values()[self.codes[i].long()] * self.scale[i].double()[:, :, None, None]

    def cache(self, sgr):
        dev = [(t.cuda() if t.is_contiguous() else t.transpose(1, 2).cuda().transpose(1, 2)).view(torch.float8_e4m3fn)
               for t in self.codes]
        return sgr.KvCache(dev[0], dev[1], self.scale[0].cuda(), self.scale[1].cuda())

    def batch(self, sgr, with_rows=True):
        return sgr.KvBatch(self.block_table.cuda(), self.seq_len.cuda(), self.q_start.cuda() if with_rows else None,
                           tokens=self.tokens, max_new=self.max_new)
