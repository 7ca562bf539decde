"""What the header says of the attention operators' arguments where no other test
looks, on the GPU against the header's own formulas."""
import random

import pytest
import torch

import kv_mask_ref as mref
import kv_ref as ref
import skinny_bf16_gemm_residual_gb300 as sgr

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    torch.cuda.set_device(0)
    sgr.sgr_init(0)
    sgr.sgr_device_error(0)
    yield


@pytest.fixture(autouse=True)
def _no_device_error():
    yield
    assert sgr.sgr_device_error(0) == 0


def test_positions_without_a_rotation_table_are_not_looked_at():
    pr = ref.Problem(64, 16, 2, [40, 20], [3, 1], seed=1)
    rope = sgr.RopeNorm(None, k_weight=(1 + 0.3 * pr.randn(64)).bfloat16().cuda())
    q, k, v = pr.randn(4, 8, 64).bfloat16().cuda().split((4, 2, 2), 1)
    with_them, without = pr.cache(sgr), pr.cache(sgr)
    a = sgr.sgr_kv_append(with_them, pr.batch(sgr), k, v, rope, q=q, positions=torch.tensor([-1, 5, 1 << 30, -7], dtype=torch.int32).cuda())
    b = sgr.sgr_kv_append(without, pr.batch(sgr), k, v, rope, q=q)
    assert torch.equal(a, b) and torch.equal(with_them.k.view(torch.uint8), without.k.view(torch.uint8))


def sees(n, length, window, sinks, bits):
    """[n, length] what each row of a tree sees, by the header's words; bits [n, n]."""
    first, t = length - n, torch.arange(length)
    out = torch.zeros(n, length, dtype=torch.bool)
    for i in range(n):
        if first + i < 0:  # a padding row
            continue
        there = bits[i].clone()
        there[:max(-first, 0)] = False  # (padding rows' bits)
        at = max(first, 0) + max(int(there.sum()), 1) - 1
        before = (t < first) & (t <= at)
        if window:
            before &= (t > at - window) | (t < sinks)
        out[i] = before
        out[i, max(first, 0):] |= there[max(-first, 0):]
    return out


@pytest.mark.parametrize("flags", [sgr.SGR_FLAG_KV_FEW_ROWS, sgr.SGR_FLAG_KV_MANY_ROWS])
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (2, 0), (1, 3), (20, 0), (20, 4), (150, 0)])
def test_tree_rows_without_bits_under_windows(window, sinks, flags):
    """Rows without any bit, with one, and with many, under windows that leave the
    former little or nothing: outputs, log-sum-exps and accumulated weights."""
    lens, new = [100, 200, 7, 5], [9, 30, 7, 8]  # (the last: three padding rows)
    pr = ref.Problem(64, 16, 2, lens, new, seed=window)
    g = torch.Generator().manual_seed(3)
    bits = [torch.rand(n, n, generator=g) < 0.3 for n in new]
    for b in bits:
        b[0] = False
        b[-2] = False
        b[2] = False
        b[2, 1] = True
    words = torch.zeros(pr.tokens, 1, dtype=torch.int64)
    for i, row in enumerate(row for b in bits for row in b):
        words[i, 0] = sum(1 << int(j) for j in row.nonzero()[:, 0])
    cache, batch = pr.cache(sgr), pr.batch(sgr)
    q = (1.5 * pr.randn(pr.tokens, 4, 64)).bfloat16()
    lse = torch.empty(pr.tokens, 4, device="cuda")
    out = sgr.sgr_kv_attention(cache, batch, q.cuda(), window=window, sinks=sinks, tree=words.cuda(), lse=lse, flags=flags)
    mass = sgr.sgr_kv_mass(cache, batch, q.cuda(), lse, cache.zero_mass(), window=window, sinks=sinks, tree=words.cuda())
    k, v = pr.values(0), pr.values(1)
    row, want, mag = 0, torch.zeros(q.shape, dtype=torch.float64), torch.zeros(q.shape, dtype=torch.float64)
    for b, (n, length) in enumerate(zip(new, lens)):
        see = sees(n, length, window, sinks, bits[b])
        t = torch.arange(length)
        pages = pr.block_table[b].long()[t // 16]
        for h in range(4):
            s = torch.where(see, q[row:row + n, h].double() @ k[pages, h // 2, t % 16].T / 8, -torch.inf)
            p = torch.softmax(s, -1).nan_to_num(nan=0.0)  # (rows that see nothing)
            want[row:row + n, h] = p @ v[pages, h // 2, t % 16]
            mag[row:row + n, h] = p @ v[pages, h // 2, t % 16].abs()
            assert torch.equal(lse[row:row + n, h].cpu().isinf(), ~see.any(1))
        got = mass[pages, :, t % 16].cpu()
        assert torch.equal(got[:, 0] != 0, see.any(0)) and torch.equal(got[:, 1] != 0, see.any(0))
        row += n
    ref.check_attention(out, want, mag)


def test_masses_where_only_some_steps_are_weighed():
    """Pages that hold NaN masses of their last user; a prompt in two chunks of which
    the second is weighed, a weighed tree, its accepted branch and a decode step that
    are not, a weighed decode step, and an eviction: with the new positions of the
    steps that are not weighed set to zero, all masses are the definition's."""
    heads, hk, dim, page, lens = 8, 2, 64, 16, [150, 70]
    g = torch.Generator().manual_seed(2)
    cache = sgr.KvCache.empty(60, hk, page, dim)
    mass = cache.zero_mass()
    mass.fill_(float("nan"))
    rope = sgr.RopeNorm(ref.rope_table(400, dim).cuda())
    order = torch.randperm(60, generator=g).int()
    table, host = order[:24].view(2, 12).cuda(), order[:24].view(2, 12).long()
    want = torch.zeros(mass.shape, dtype=torch.float64)
    tol = torch.zeros_like(want)

    def step(length, new, weighed, trees=None, positions=None, rows=None):
        """Appends `new` tokens up to `length` positions; weighs them or clears their masses."""
        nonlocal want, tol
        n = sum(new)
        start = torch.tensor([0, new[0], n], dtype=torch.int32)
        batch = sgr.KvBatch(table, torch.tensor(length, dtype=torch.int32).cuda(), start.cuda(), tokens=n, max_new=max(new))
        q, k, v = torch.randn(n, heads + 2 * hk, dim, generator=g).bfloat16().cuda().split((heads, hk, hk), 1)
        if rows is not None:
            k, v = rows[0][rows[2]], rows[1][rows[2]]
        q = sgr.sgr_kv_append(cache, batch, k, v, rope, q=q, positions=positions)
        lse = torch.empty(n, heads, device="cuda")
        words = torch.cat([mref.tree_words(t, 1) for t in trees]).cuda() if trees else None
        sgr.sgr_kv_attention(cache, batch, q, tree=words, lse=lse)
        places = [(host[b, t // page], t % page) for b in range(2) for t in range(length[b] - new[b], length[b])]
        if weighed:
            sgr.sgr_kv_mass(cache, batch, q, lse, mass, tree=words)
            kk = (cache.k.float() * cache.k_scale[:, :, None, None]).double().cpu()
            want, more = mref.mass(want, q.cpu(), kk, lse.cpu(), host, length, start, page, dim ** -0.5, trees=trees)
            for p, at in places:
                tol[p, :, at] = 0.0
            tol += more
        else:
            for p, at in places:
                mass[p, :, at] = 0.0
                want[p, :, at] = tol[p, :, at] = 0.0
        return k, v

    step([90, 30], [90, 30], False)
    step(lens, [60, 40], True)
    r = random.Random(5)
    trees = [mref.random_tree(7, r) for _ in range(2)]
    depth = torch.tensor([lens[b] + len(path) - 1 for b in range(2) for path in trees[b]], dtype=torch.int32).cuda()
    k, v = step([lens[0] + 7, lens[1] + 7], [7, 7], True, trees, depth)
    paths = [max(t, key=len) for t in trees]
    count = [len(p) for p in paths]
    rows = torch.tensor([7 * b + j for b in range(2) for j in paths[b]]).cuda()
    lens = [lens[b] + count[b] for b in range(2)]
    step(lens, count, False, positions=depth[rows], rows=(k, v, rows))
    lens = [n + 1 for n in lens]
    step(lens, [1, 1], False)
    lens = [n + 1 for n in lens]
    step(lens, [1, 1], True)
    masses = mass.double().cpu()
    for b in range(2):
        t = torch.arange(lens[b])
        pages = host[b][t // page]
        got, w, e = masses[pages, :, t % page], want[pages, :, t % page], tol[pages, :, t % page]
        assert ((got - w).abs() <= e).all() and (w > 0).any()
    keep = torch.tensor([64, 40], dtype=torch.int32).cuda()
    batch = sgr.KvBatch(table, torch.tensor(lens, dtype=torch.int32).cuda())
    new_len, kept = sgr.sgr_kv_evict(cache, batch, mass, keep, order[30:38].view(2, 4).cuda(), first=2, recent=4)
    for b in range(2):
        t = torch.arange(lens[b])
        for h in range(hk):
            stay = mref.chosen(masses[host[b][t // page], h, t % page].tolist(), int(keep[b]), 2, 4)
            assert kept[b, h, :int(new_len[b])].tolist() == stay


def test_numbers_past_32_bits_are_refused():
    pr = ref.Problem(64, 16, 1, [20], [1])
    cache, batch, q = pr.cache(sgr), pr.batch(sgr), pr.randn(1, 2, 64).bfloat16().cuda()
    lse, mass = torch.zeros(1, 2, device="cuda"), pr.cache(sgr).zero_mass()
    keep, to = torch.ones(1, dtype=torch.int32, device="cuda"), torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    for big in (1 << 31, (1 << 32) + 5):
        for call in (lambda: sgr.sgr_kv_attention(cache, batch, q, window=big),
                     lambda: sgr.sgr_kv_attention(cache, batch, q, window=big, lse=lse),
                     lambda: sgr.sgr_kv_attention(cache, batch, q, window=4, sinks=big),
                     lambda: sgr.sgr_kv_mass(cache, batch, q, lse, mass, window=big),
                     lambda: sgr.sgr_kv_evict(cache, batch, mass, keep, to, first=big),
                     lambda: sgr.sgr_kv_evict(cache, batch, mass, keep, to, recent=big)):
            with pytest.raises(ValueError, match="32 bits"):
                call()


def test_plain_calls_of_medium_row_counts_keep_small_elements():
    """A query's elements far below its largest keep their 8 bits (multiples of
    2^-20 from 2^-14 to 2^-12, beside a 1 that meets zeros), where all scores come
    from them, in a plain call with 160 rows a head; with or without a log-sum-exp.
    Scores are then good to the 32-bit sums' 2^-20 of them, far below the allowed
    2^-7 of sum p |v|; steps of 2^-18 would move scores of some 4 by a tenth."""
    pr = ref.Problem(64, 64, 8, [1500] * 4, [40] * 4, seed=2)
    for b in pr.block_table:
        pr.codes[0][b.long(), :, :, 0] = 0
    small = torch.randint(64, 256, (160, 32, 64), generator=pr.g) * (2 * torch.randint(0, 2, (160, 32, 64), generator=pr.g) - 1)
    q = (small * 2.0 ** -20).bfloat16()
    q[:, :, 0] = 1.0
    assert (q[:, :, 1:].float() == small[:, :, 1:] * 2.0 ** -20).all()
    cache, batch = pr.cache(sgr), pr.batch(sgr)
    scale = 2.0 ** 11
    out = sgr.sgr_kv_attention(cache, batch, q.cuda(), scale=scale)
    lse = torch.empty(160, 32, device="cuda")
    assert torch.equal(sgr.sgr_kv_attention(cache, batch, q.cuda(), scale=scale, lse=lse), out)
    k, v = pr.values(0), pr.values(1)
    want, mag = torch.zeros(q.shape, dtype=torch.float64), torch.zeros(q.shape, dtype=torch.float64)
    t = torch.arange(1500)
    for b in range(4):
        pages, rows = pr.block_table[b].long()[t // 64], slice(40 * b, 40 * b + 40)
        hidden = t > torch.arange(1460, 1500)[:, None]
        for h in range(32):
            s = (q[rows, h].double() @ k[pages, h // 4, t % 64].T * scale).masked_fill(hidden, -torch.inf)
            assert 1 < float(s[:, :1460].std()) < 64
            p = torch.softmax(s, -1)
            want[rows, h] = p @ v[pages, h // 4, t % 64]
            mag[rows, h] = p @ v[pages, h // 4, t % 64].abs()
    ref.check_attention(out, want, mag)
    with pytest.raises(AssertionError):  # (the call's choice is what this is about)
        ref.check_attention(sgr.sgr_kv_attention(cache, batch, q.cuda(), scale=scale, flags=sgr.SGR_FLAG_KV_MANY_ROWS), want, mag)


@pytest.mark.parametrize("window,many", [(0, True), (4000, True), (512, True), (64, False)])
def test_choice_of_plain_calls_under_windows(window, many):
    """A window takes no call that has many rows away from the kernel for them,
    unless it is so short that there is next to nothing to do."""
    pr = ref.Problem(64, 64, 4, [3000] * 3 + [700] * 13, [18] * 16, seed=1)
    q = pr.randn(pr.tokens, 28, 64).bfloat16().cuda()
    cache, batch = pr.cache(sgr), pr.batch(sgr)
    out, forced = (sgr.sgr_kv_attention(cache, batch, q, window=window, flags=f)
                   for f in (0, sgr.SGR_FLAG_KV_MANY_ROWS if many else sgr.SGR_FLAG_KV_FEW_ROWS))
    assert torch.equal(out, forced)
    other = sgr.sgr_kv_attention(cache, batch, q, window=window, flags=sgr.SGR_FLAG_KV_FEW_ROWS if many else sgr.SGR_FLAG_KV_MANY_ROWS)
    assert not torch.equal(out, other)


@pytest.mark.parametrize("dim,page,heads,hk,lens,new", [
    (128, 32, 4, 2, [13, 319], [2, 107]), (64, 16, 24, 2, [2000] * 5, [30] * 5), (128, 64, 28, 4, [9000], [7]),
    (64, 64, 32, 8, [1500] * 4, [40] * 4), (64, 64, 8, 8, [4000] * 40, [5] * 40)])
def test_workspace_is_enough_for_trees_and_windows(dim, page, heads, hk, lens, new):
    """One workspace for calls with and without trees, windows, sinks and a
    log-sum-exp, which may take different kernels and row tiles."""
    pr = ref.Problem(dim, page, hk, [1] * len(lens), [1] * len(lens), extra_pages=4)  # (no position is looked at)
    cache = pr.cache(sgr)
    table = torch.zeros(len(lens), -(-max(lens) // page), dtype=torch.int32, device="cuda")
    start = torch.zeros(len(lens) + 1, dtype=torch.int32, device="cuda")  # no rows
    batch = sgr.KvBatch(table, torch.zeros(len(lens), dtype=torch.int32, device="cuda"), start, tokens=sum(new), max_new=max(new))
    q = torch.zeros(sum(new), heads, dim, dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros(sum(new), heads, device="cuda")
    words = torch.zeros(sum(new), -(-max(new) // 64), dtype=torch.int64, device="cuda")
    for flags in (0, sgr.SGR_FLAG_KV_FEW_ROWS, sgr.SGR_FLAG_KV_MANY_ROWS):
        work = sgr.kv_attention_workspace(cache, batch, heads, flags)
        for window in (0, 1, 30, 300, 1000, 4000, 100000):
            for sinks in (0, 4, 600):
                for tree in (None, words):
                    for stat in (None, lse):
                        sgr.sgr_kv_attention(cache, batch, q, window=window, sinks=sinks, tree=tree, lse=stat, workspace=work,
                                             flags=flags)
