"""Definitions in 64 bits (torch float64 on the CPU, one sequence and head at a
time) of attention under masks -- windows, sinks, trees of drafted tokens --
with its log-sum-exp, and the trees of the tests."""
from __future__ import annotations

import math
import random

import torch

import kv_ref as ref


def random_tree(n, r: random.Random):
    """For each of n drafted tokens those that it sees: the path from the root to it."""
    paths = [[0]]
    for i in range(1, n):
        paths.append(paths[r.randrange(max(0, i - 5), i)] + [i])
    return paths[:n]


def tree_words(paths, words):
    """int64 [tokens, words] of lists of seen tokens."""
    out = torch.zeros(len(paths), words, dtype=torch.int64)
    for i, path in enumerate(paths):
        for w in range(words):
            x = sum(1 << (j - 64 * w) for j in path if j // 64 == w)
            out[i, w] = x - (1 << 64) if x >> 63 else x
    return out


def seen(n, length, window, sinks, paths):
    """[n, length] whether each of a sequence's n rows sees a position."""
    t, first = torch.arange(length), length - n
    rows = []
    for i in range(n):
        if first + i < 0:  # a padding row
            rows.append(torch.zeros(length, dtype=torch.bool))
            continue
        if paths is None:
            p = first + i
        else:
            there = [j for j in paths[i] if first + j >= 0 and j < n]
            p = max(first, 0) + max(len(there) - 1, 0)
        s = t <= p
        if window:
            s &= (t > p - window) | (t < sinks)
        if paths is not None:
            s &= t < first
            for j in there:
                s[first + j] = True
        rows.append(s)
    return torch.stack(rows) if rows else torch.zeros(0, length, dtype=torch.bool)


def sequences(block_table, seq_len, q_start, page):
    """(first row, rows, length, (pages, places) of its positions) of each sequence."""
    for b in range(len(seq_len)):
        r0, r1 = ref.rows_of(q_start, b)
        length = int(seq_len[b])
        t = torch.arange(length)
        yield b, r0, r1 - r0, length, block_table[b].long()[t // page], t % page


def attention(q, k, v, block_table, seq_len, q_start, page, scale, window=0, sinks=0, trees=None):
    """Outputs, sum p |v| / sum p, log-sum-exp, and the largest |q| |k| scale of a
    row's scores.  k, v [pages, kv_heads, page, dim] float64 values; trees: each
    sequence's lists of seen tokens."""
    hk, heads = k.shape[1], q.shape[1]
    group = heads // hk
    out, mag = torch.zeros(q.shape, dtype=torch.float64), torch.zeros(q.shape, dtype=torch.float64)
    lse, reach = torch.full(q.shape[:2], -math.inf, dtype=torch.float64), torch.zeros(q.shape[:2], dtype=torch.float64)
    for b, r0, n, length, pages, place in sequences(block_table, seq_len, q_start, page):
        see = seen(n, length, window, sinks, trees[b] if trees else None)
        for i in range(n):
            t = see[i].nonzero()[:, 0]
            if not t.numel():
                continue
            for h in range(hk):
                kk, vv = k[pages[t], h, place[t]], v[pages[t], h, place[t]]
                qq = q[r0 + i, h * group:(h + 1) * group].double()
                s = qq @ kk.T * scale
                p = torch.softmax(s, -1)
                rows = slice(h * group, (h + 1) * group)
                out[r0 + i, rows] = p @ vv
                mag[r0 + i, rows] = p @ vv.abs()
                lse[r0 + i, rows] = torch.logsumexp(s, -1)
                reach[r0 + i, rows] = qq.norm(dim=-1) * kk.norm(dim=-1).max() * abs(scale)
    return out, mag, lse, reach


def check_lse(got, want, reach, what=""):
    """Scores to 2^-16 of |q| |k| scale; exponentials to 2^-22 and their sum of 32
    bits below 2^-17 together; the logarithm's rounding, 2^-23 of it."""
    got = got.double().cpu()
    assert torch.equal(got.isinf(), want.isinf()) and torch.equal(got.isnan(), want.isnan()), f"{what}: rows without positions"
    tol = 2.0 ** -16 * reach + 2.0 ** -17 + 2.0 ** -22 * want.abs()
    bad = ~((got - want).abs() <= tol) & want.isfinite()
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, first {tuple(bad.nonzero()[0].tolist())}"


# ------------------------------------------------------------------ mass, eviction
def mass(before, q, k, lse, block_table, seq_len, q_start, page, scale, window=0, sinks=0, trees=None):
    """before [pages, kv_heads, page] float64 -> the same with the call's weights,
    and the error allowed for them.  lse [tokens, heads]: as the call gets it.

    A weight's: the scores', 2^-17 of |q| |k| scale (a query's elements to 2^-22 of
    its largest, over 128 of them, and 32-bit products and sums), 2^-20 of 1 + |lse|
    (its rounding and the exponential's); a sum's: 2^-18 of it (up to some 2^12
    terms, half of 2^-24 each on the average); the mass's rounding, 2^-23.  Weights
    below 2^-126, FP32's least normal number, count as zeros: up to 2^12 of them,
    2^-114 together."""
    out, tol = before.clone(), torch.zeros_like(before)
    hk = k.shape[1]
    group = q.shape[1] // hk
    for b, r0, n, length, pages, place in sequences(block_table, seq_len, q_start, page):
        see = seen(n, length, window, sinks, trees[b] if trees else None)
        new = torch.arange(length) >= length - n
        any_row = see.any(0)
        touched = (any_row | new).nonzero()[:, 0]
        for h in range(hk):
            total = torch.zeros(length, dtype=torch.float64)
            err = torch.zeros(length, dtype=torch.float64)
            t = any_row.nonzero()[:, 0]
            if t.numel():
                kk = k[pages[t], h, place[t]]
                qq = q[r0:r0 + n, h * group:(h + 1) * group].double()
                s = torch.einsum("ngd,td->ngt", qq, kk) * scale
                at = lse[r0:r0 + n, h * group:(h + 1) * group].double()[..., None]
                w = torch.where(see[:, None, t], torch.exp(s - at), 0.0)
                reach = qq.norm(dim=-1)[..., None] * kk.norm(dim=-1) * abs(scale)
                total[t] = w.sum((0, 1))
                rel = torch.where(see[:, None, t], 2.0 ** -17 * reach + 2.0 ** -20 * (1 + at.abs()), 0.0)
                err[t] = (w * rel).sum((0, 1)) + 2.0 ** -18 * total[t] + 2.0 ** -114
            old = out[pages[touched], h, place[touched]]
            old[new[touched]] = 0.0
            out[pages[touched], h, place[touched]] = old + total[touched]
            tol[pages[touched], h, place[touched]] = err[touched] + 2.0 ** -23 * (old + total[touched])
    return out, tol


def check_mass(got, want, tol, what=""):
    got = got.double().cpu()
    bad = ~((got - want).abs() <= tol) & ~(got.isnan() & want.isnan())
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} off, first {tuple(bad.nonzero()[0].tolist())}: "
                           f"got {got[bad][0]} want {want[bad][0]} tol {tol[bad][0]}")


def chosen(m, keep, first, recent):
    """Positions that stay of masses m [length] (a list of floats)."""
    length = len(m)
    n = min(keep, length)
    f = min(first, n)
    r = min(recent, n - f)
    middle = range(f, length - r)
    order = sorted(middle, key=lambda t: (0 if math.isnan(m[t]) else 1, -m[t] if not math.isnan(m[t]) else 0.0, t))
    return sorted(list(range(f)) + order[:n - f - r] + list(range(length - r, length)))


def evict(codes, scale, masses, block_table, seq_len, new_table, page, keep, first, recent):
    """codes: K and V uint8 [pages, heads, page, dim], scale float [pages, heads].
    Returns the same after the call (codes as their values under the new scales
    before rounding, NaN where not written), the masses, and the kept positions."""
    values = ref.e4m3_values()
    want = [torch.full(c.shape, math.nan, dtype=torch.float64) for c in codes]
    scales, masses, kept = [s.double().clone() for s in scale], masses.clone(), []
    source = masses.clone()
    heads = codes[0].shape[1]
    for b in range(len(seq_len)):
        length = int(seq_len[b])
        t = torch.arange(length)
        pages, place = block_table[b].long()[t // page], t % page
        kept.append([])
        for h in range(heads):
            stay = torch.tensor(chosen(source[pages, h, place].tolist(), int(keep[b]), first, recent), dtype=torch.long)
            kept[b].append(stay)
            for lo in range(0, len(stay), page):
                part, to = stay[lo:lo + page], int(new_table[b, lo // page])
                masses[to, h, :len(part)] = source[pages[part], h, place[part]]
                for i in range(2):
                    x = values[codes[i][pages[part], h, place[part]].long()] * scale[i].double()[pages[part], h, None]
                    finite = x[torch.isfinite(x)].abs()
                    scales[i][to, h] = 2.0 ** ref.scale_exp(float(finite.max()) if finite.numel() else 0.0)
                    want[i][to, h, :len(part)] = x
    return want, scales, masses, kept
