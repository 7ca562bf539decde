"""Accumulated attention weight and eviction by it on the GPU against their
definitions in 64 bits (tests/kv_mask_ref.py), alone and as a server uses them."""
import math
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


def inputs(pr, heads, window=0, sinks=0, trees=None, factor=1.5):
    """Queries, their log-sum-exp as FP32, the tree's words, and a mass in use."""
    q = (factor * pr.randn(pr.tokens, heads, pr.dim)).bfloat16()
    _, _, lse, _ = mref.attention(q, pr.values(0), pr.values(1), pr.block_table, pr.seq_len, pr.q_start, pr.page,
                                  pr.dim ** -0.5, window, sinks, trees)
    tree = None if trees is None else torch.cat([mref.tree_words(t, -(-pr.max_new // 64)) for t in trees]).cuda()
    mass = torch.rand(pr.pages, pr.hk, pr.page, generator=pr.g)
    return q, lse.float(), tree, mass


def weigh(pr, heads, window=0, sinks=0, trees=None, factor=1.5):
    q, lse, tree, mass = inputs(pr, heads, window, sinks, trees, factor)
    want, tol = mref.mass(mass.double(), q, pr.values(0), lse, pr.block_table, pr.seq_len, pr.q_start, pr.page,
                          pr.dim ** -0.5, window, sinks, trees)
    cache, batch = pr.cache(sgr), pr.batch(sgr)
    got = mass.cuda()
    back = sgr.sgr_kv_mass(cache, batch, q.cuda(), lse.cuda(), got, window=window, sinks=sinks, tree=tree)
    assert back is got
    mref.check_mass(got, want, tol)
    # the same bits again, in a wider buffer and with heads inside pages
    wide = torch.full((pr.pages, pr.page, pr.hk + 1), 5.0, device="cuda").transpose(1, 2).contiguous().view(pr.pages, pr.hk + 1, pr.page)
    wide[:, :pr.hk] = mass.cuda()
    sgr.sgr_kv_mass(cache, batch, q.cuda(), lse.cuda(), wide[:, :pr.hk], window=window, sinks=sinks, tree=tree)
    assert torch.equal(wide[:, :pr.hk], got) and (wide[:, pr.hk] == 5).all()
    return got


MASS = [
    # dim, page, heads, hk, lens, new, window, sinks
    (128, 64, 7, 1, [1], [1], 0, 0),
    (128, 64, 28, 4, [333], [1], 0, 0),
    (64, 16, 8, 8, [127, 128, 129, 1, 16, 0], [1, 1, 1, 1, 1, 1], 0, 0),
    (128, 16, 16, 1, [700, 0, 257], [1, 1, 1], 0, 0),
    (64, 128, 12, 1, [640, 5], [1, 1], 0, 0),
    (128, 32, 32, 1, [900], [1], 0, 0),
    (64, 32, 5, 1, [300, 90], [4, 6], 0, 0),
    (128, 32, 12, 2, [513, 40, 3], [5, 40, 7], 0, 0),          # up to 240 rows a head; padding rows
    (128, 128, 16, 2, [1300], [17], 0, 0),
    (64, 64, 16, 4, [200, 64], [64, 64], 0, 0),                # 256 rows exactly
    (64, 64, 16, 4, [200, 64], [65, 64], 0, 0),                # one token more: several row tiles
    (128, 32, 24, 2, [700, 130, 5], [150, 1, 5], 0, 0),
    (128, 64, 6, 2, [1000, 300, 64], [1, 3, 2], 100, 0),
    (64, 16, 8, 2, [1000, 150, 30], [1, 1, 1], 20, 3),
    (64, 32, 8, 1, [700, 400], [100, 90], 64, 130),            # several row tiles, windows and sinks
    (128, 64, 4, 4, [600], [300], 1, 1),
]


@pytest.mark.parametrize("dim,page,heads,hk,lens,new,window,sinks", MASS)
def test_mass(dim, page, heads, hk, lens, new, window, sinks):
    weigh(ref.Problem(dim, page, hk, lens, new, seed=sum(lens), heads_inside=len(lens) > 1), heads, window, sinks)


@pytest.mark.parametrize("dim,page,heads,hk,lens,new,window,sinks", [
    (128, 64, 28, 4, [300, 70], [7, 3], 0, 0),
    (64, 16, 8, 2, [260, 135, 128, 3], [25, 9, 1, 5], 0, 0),
    (128, 32, 8, 1, [500], [130], 40, 4),
])
def test_mass_of_trees(dim, page, heads, hk, lens, new, window, sinks):
    r = random.Random(1)
    trees = [mref.random_tree(n, r) for n in new]
    trees[0][-1] = []  # a row without bits; its own position gets nothing unless others see it
    weigh(ref.Problem(dim, page, hk, lens, new, seed=2), heads, window, sinks, trees)


@pytest.mark.parametrize("factor", [0.0, 30.0])
def test_mass_of_flat_and_sharp_scores(factor):
    weigh(ref.Problem(128, 64, 2, [1500, 90], [1, 2], seed=6), 8, factor=factor)


def test_mass_sums_to_the_number_of_rows():
    """With the log-sum-exp that the attention wrote, a row's weights over a long
    cache sum to one: 2^-15, some 30 times the sums' own errors."""
    pr = ref.Problem(128, 128, 2, [30001], [3], seed=8)
    cache, batch = pr.cache(sgr), pr.batch(sgr)
    q = (1.5 * pr.randn(3, 10, 128)).bfloat16().cuda()
    lse = torch.empty(3, 10, device="cuda")
    sgr.sgr_kv_attention(cache, batch, q, lse=lse)
    mass = cache.zero_mass()
    sgr.sgr_kv_mass(cache, batch, q, lse, mass)
    total = mass.double().sum((0, 2)).cpu()
    assert ((total - 15).abs() <= 15 * 2.0 ** -15).all(), total


def test_mass_of_new_positions_is_set_and_of_unseen_ones_kept():
    """NaN masses where the call sets or does not look, NaN keys where no row sees."""
    pr = ref.Problem(64, 32, 1, [200, 70], [4, 1], seed=3)
    for t in range(10, 200 - 4 - 50 + 1):  # between the sinks and the first window
        pr.codes[0][int(pr.block_table[0, t // 32]), 0, t % 32] = ref.NAN_CODE
    q, lse, _, mass = inputs(pr, 4, 50, 10)
    for b, (length, n) in enumerate(zip(pr.lens, pr.new)):
        for t in range(length):
            if t >= length - n or (10 <= t <= length - n - 50):
                mass[int(pr.block_table[b, t // 32]), 0, t % 32] = math.nan
    want, tol = mref.mass(mass.double(), q, pr.values(0), lse, pr.block_table, pr.seq_len, pr.q_start, 32, 0.125, 50, 10)
    got = sgr.sgr_kv_mass(pr.cache(sgr), pr.batch(sgr), q.cuda(), lse.cuda(), mass.cuda(), window=50, sinks=10)
    assert torch.equal(got.cpu().isnan(), want.isnan())
    mref.check_mass(got, want, tol)


@pytest.mark.parametrize("new", [1, 40, 100])
def test_mass_stream_replay_and_rows_of_no_sequence(new):
    pr = ref.Problem(64, 32, 2, [300, 200], [new, new], seed=21)
    q, lse, _, mass = inputs(pr, 8)
    rows = pr.tokens + 3  # three rows of nobody
    x = torch.full((rows, 8, 64), math.nan, dtype=torch.bfloat16, device="cuda")
    stat = torch.full((rows, 8), math.nan, device="cuda")
    x[:pr.tokens], stat[:pr.tokens] = q.cuda(), lse.cuda()
    cache = pr.cache(sgr)
    batch = sgr.KvBatch(pr.block_table.cuda(), pr.seq_len.cuda(), pr.q_start.cuda(), tokens=rows, max_new=new)
    work = sgr.kv_mass_workspace(cache, batch, 8)
    work.fill_(255)  # its contents do not matter
    got = mass.cuda()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    sgr.sgr_kv_mass(cache, batch, x, stat, got, workspace=work, stream=side)
    side.synchronize()
    mref.check_mass(got, *mref.mass(mass.double(), q, pr.values(0), lse, pr.block_table, pr.seq_len, pr.q_start, 32, 0.125))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sgr.sgr_kv_mass(cache, batch, x, stat, got, workspace=work)
    for lens in ([300, 200], [new, new + 33], [299, new - 1]):
        batch.seq_len.copy_(torch.tensor(lens, dtype=torch.int32))
        _, _, now, _ = mref.attention(q, pr.values(0), pr.values(1), pr.block_table, lens, pr.q_start, 32, 0.125)
        stat[:pr.tokens] = now.float().cuda()
        got.copy_(mass)
        graph.replay()
        torch.cuda.synchronize()
        mref.check_mass(got, *mref.mass(mass.double(), q, pr.values(0), now.float(), pr.block_table, lens, pr.q_start, 32, 0.125),
                        f"replay {lens}")


def test_mass_bad_device_data_is_recorded():
    pr = ref.Problem(64, 16, 1, [40, 20], [1, 1], seed=5)
    q, lse, _, mass = inputs(pr, 4)
    whole = sgr.sgr_kv_mass(pr.cache(sgr), pr.batch(sgr), q.cuda(), lse.cuda(), mass.cuda())
    for change in ("page", "length", "rows"):
        table, lens, start = pr.block_table.clone(), pr.seq_len.clone(), pr.q_start.clone()
        if change == "page":
            table[0, 1] = pr.pages
        elif change == "length":
            lens[0] = 16 * table.shape[1] + 1
        else:
            start[0] = -5
        batch = sgr.KvBatch(table.cuda(), lens.cuda(), start.cuda(), tokens=2)
        got = sgr.sgr_kv_mass(pr.cache(sgr), batch, q.cuda(), lse.cuda(), mass.cuda())
        assert sgr.sgr_device_error(0) == 7, change
        for block in range(2):  # the other sequence's
            page = int(pr.block_table[1, block])
            assert torch.equal(got[page], whole[page]), change
        if change == "page":
            page = int(pr.block_table[0, 1])
            assert torch.equal(got[page].cpu(), mass[page])
    # more rows than max_new says
    pr = ref.Problem(64, 16, 1, [80], [70], seed=5)
    q, lse, _, mass = inputs(pr, 4)
    batch = sgr.KvBatch(pr.block_table.cuda(), pr.seq_len.cuda(), pr.q_start.cuda(), tokens=70, max_new=64)
    sgr.sgr_kv_mass(pr.cache(sgr), batch, q.cuda(), lse.cuda(), mass.cuda())
    assert sgr.sgr_device_error(0) == 7


# ----------------------------------------------------------------------- eviction
def fresh_table(pr, keeps, extra=0):
    """New pages behind the cache's own, in a shuffled order; -1 where none is needed."""
    need = [-(-min(k, l) // pr.page) + extra for k, l in zip(keeps, pr.lens)]
    order = torch.randperm(sum(need), generator=pr.g).int() + pr.pages
    table = torch.full((len(need), max(need + [1])), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table, sum(need)


def grown(pr, more):
    """The problem's cache with `more` pages behind it, whose contents show what is written."""
    for i in range(2):
        codes = torch.full((more, pr.hk, pr.page, pr.dim), 0x55, dtype=torch.uint8)
        pr.codes[i] = torch.cat([pr.codes[i], codes])
        pr.scale[i] = torch.cat([pr.scale[i], torch.full((more, pr.hk), 3.0)])
    pr.pages += more


def evict(pr, keeps, first, recent, mass=None, flags=0, odd=False):
    new_table, more = fresh_table(pr, keeps)
    grown(pr, more)
    if mass is None:
        mass = torch.rand(pr.pages, pr.hk, pr.page, generator=pr.g)
    else:
        mass = torch.cat([mass, torch.full((more, pr.hk, pr.page), 9.0)])
    cache, batch = pr.cache(sgr), pr.batch(sgr)
    kept = torch.full((len(pr.lens), pr.hk, new_table.shape[1] * pr.page), -7, dtype=torch.int32, device="cuda")
    got = mass.cuda()
    if odd:  # masses whose rows are not aligned to 16 bytes
        wide = torch.zeros(pr.pages, pr.hk, pr.page + 1, device="cuda")
        wide[:, :, 1:] = got
        got = wide[:, :, 1:]
    new_len, back = sgr.sgr_kv_evict(cache, batch, got, torch.tensor(keeps, dtype=torch.int32).cuda(), new_table.cuda(),
                                     first=first, recent=recent, kept=kept, flags=flags)
    assert back is kept
    want, scales, masses, stay = mref.evict(pr.codes, pr.scale, mass.double(), pr.block_table, pr.seq_len, new_table, pr.page,
                                            keeps, first, recent)
    assert new_len.tolist() == [min(k, l) for k, l in zip(keeps, pr.lens)]
    for b in range(len(pr.lens)):
        for h in range(pr.hk):
            n = len(stay[b][h])
            assert kept[b, h, :n].tolist() == stay[b][h].tolist(), (b, h)
            assert (kept[b, h, n:] == -7).all()
    assert torch.equal(got.double().cpu().nan_to_num(nan=-1.0), masses.nan_to_num(nan=-1.0))
    for i, (codes, scale) in enumerate(((cache.k, cache.k_scale), (cache.v, cache.v_scale))):
        there = ~scales[i].isnan()
        assert torch.equal(scale.cpu().isnan(), ~there)
        assert torch.equal(scale.double().cpu()[there], scales[i][there])
        still = want[i].isnan()
        codes = codes.view(torch.uint8).cpu()
        nan = torch.zeros_like(still)  # values that are NaN in the cache stay NaN
        for b in range(len(pr.lens)):
            for h in range(pr.hk):
                t = stay[b][h]
                src = pr.codes[i][pr.block_table[b].long()[t // pr.page], h, t % pr.page]
                at = torch.arange(len(t))
                nan[new_table[b].long()[at // pr.page], h, at % pr.page] = (src & 0x7F) == 0x7F
        assert ((codes[nan] & 0x7F) == 0x7F).all()
        same = still & ~nan
        assert torch.equal(codes[same], pr.codes[i][same])
        ok = ~still
        by = scales[i][:, :, None, None].expand_as(want[i])[ok]
        x = want[i][ok] / by
        step = ref.quantum(x)
        value = ref.e4m3_values()[codes[ok].long()]
        assert ((value - x).abs() <= 0.5 * step).all()
    return cache, new_table, new_len, kept


EVICT = [
    # dim, page, hk, lens, keep, first, recent
    (128, 64, 1, [1], [1], 0, 0),
    (128, 64, 4, [300, 70], [100, 70], 4, 20),
    (64, 16, 2, [260, 135, 128, 1, 0], [17, 100, 64, 5, 3], 1, 3),
    (128, 128, 2, [700, 140], [128, 129], 0, 0),
    (64, 32, 3, [500, 70], [33, 7], 30, 10),          # less room than the ends want
    (128, 32, 1, [1000], [999], 5, 100),
    (64, 128, 2, [400, 300], [0, 1], 4, 4),
    (128, 16, 1, [9000, 20], [1500, 20], 4, 64),      # a cluster of several CTAs
    (64, 64, 1, [20001], [5000], 0, 1),
]


@pytest.mark.parametrize("dim,page,hk,lens,keep,first,recent", EVICT)
def test_evict(dim, page, hk, lens, keep, first, recent):
    pr = ref.Problem(dim, page, hk, lens, [min(1, l) for l in lens], seed=sum(lens), heads_inside=hk == 2)
    evict(pr, keep, first, recent)


@pytest.mark.parametrize("lens,keep", [([700, 33], [100, 20]), ([40000], [7000])])
def test_evict_masses_of_odd_strides(lens, keep):
    evict(ref.Problem(64, 16, 1, lens, [1] * len(lens), seed=len(lens)), keep, 3, 9, odd=True)


@pytest.mark.parametrize("kind", ["equal", "few", "signs", "tiny"])
def test_evict_ties_and_special_masses(kind):
    """Equal masses (the first positions stay), zeros of both signs, infinities,
    NaN, negative and subnormal ones."""
    pr = ref.Problem(64, 16, 2, [777, 64, 40], [1, 1, 1], seed=4)
    m = {"equal": torch.full((pr.pages, 2, 16), 0.25),
         "few": torch.randint(0, 3, (pr.pages, 2, 16), generator=pr.g).float(),
         "signs": torch.tensor([0.0, -0.0, 1.0, -1.0, math.inf, -math.inf, math.nan, 2.0 ** -149, -(2.0 ** -149)])[
             torch.randint(0, 9, (pr.pages, 2, 16), generator=pr.g)],
         "tiny": torch.rand(pr.pages, 2, 16, generator=pr.g) * 2.0 ** -130}[kind]
    for keep in ([300, 10, 39], [1, 63, 2]):
        evict(ref.Problem(64, 16, 2, [777, 64, 40], [1, 1, 1], seed=4), keep, 2, 3, mass=m)


def test_evict_more_keys_than_shared_memory_holds():
    """A sequence past what a cluster keeps in shared memory, many equal keys around its end."""
    pr = ref.Problem(64, 128, 1, [140000], [1], seed=9)
    m = torch.randint(0, 50, (pr.pages, 1, 128), generator=pr.g).float()
    evict(pr, [70000], 4, 1000, mass=m)


def test_evict_page_scales_far_apart_zeros_and_nan():
    """Positions of pages whose scales differ by up to 2^40 on one page, pages of
    zeros, NaN codes."""
    pr = ref.Problem(128, 16, 1, [200], [1], seed=8)
    for i, f in ((0, (0, -3, 1, -40, 2, 0, 1)), (1, (0, 20, -20, 3, -40, 10, 0))):
        for block, e in enumerate(f):
            pr.scale[i][int(pr.block_table[0, block])] *= 2.0 ** e
    for block in (7, 8, 9):
        pr.codes[0][int(pr.block_table[0, block])] = 0x80 if block == 8 else 0
        pr.scale[0][int(pr.block_table[0, block])] = 2.0 ** (64 if block == 9 else -64)
    pr.codes[1][int(pr.block_table[0, 3]), 0, 2, 7] = 0xFF
    pr.codes[1][int(pr.block_table[0, 11]), 0, :] = ref.NAN_CODE
    m = torch.rand(pr.pages, 1, 16, generator=pr.g)
    for block in (7, 8, 9, 11):
        m[int(pr.block_table[0, block])] += 2
    evict(pr, [120], 0, 0, mass=m)


def test_evict_bad_device_data_is_recorded():
    for change in ("old page", "new page", "room", "keep", "length"):
        pr = ref.Problem(64, 16, 1, [60, 20], [1, 1], seed=5)
        new_table, more = fresh_table(pr, [30, 10])
        grown(pr, more)
        mass = torch.rand(pr.pages, 1, 16, generator=pr.g)
        keep, table, lens = [30, 10], pr.block_table.clone(), pr.seq_len.clone()
        if change == "old page":
            table[0, 3] = pr.pages  # the protected end's
        elif change == "new page":
            new_table[0, 1] = -1
        elif change == "room":
            keep[0] = 33
        elif change == "keep":
            keep[0] = -1
        else:
            lens[0] = 16 * table.shape[1] + 1
        cache = pr.cache(sgr)
        batch = sgr.KvBatch(table.cuda(), lens.cuda())
        got = mass.cuda()
        new_len, kept = sgr.sgr_kv_evict(cache, batch, got, torch.tensor(keep, dtype=torch.int32).cuda(), new_table.cuda(),
                                         first=2, recent=4)
        assert sgr.sgr_device_error(0) == 7, change
        assert new_len.tolist()[1] == 10
        want = mref.chosen(mass[pr.block_table[1].long()[:2], 0].flatten()[:20].tolist(), 10, 2, 4)
        assert kept[1, 0, :10].tolist() == want
        if change == "room":
            assert new_len.tolist()[0] == 32
        if change == "keep":
            assert new_len.tolist()[0] == 0


def test_evict_stream_and_replay():
    pr = ref.Problem(128, 32, 2, [300, 120], [1, 1], seed=31)
    keeps = [100, 100]
    new_table, more = fresh_table(pr, keeps)
    grown(pr, more)
    mass = torch.rand(pr.pages, 2, 32, generator=pr.g)
    cache, batch, got = pr.cache(sgr), pr.batch(sgr), mass.cuda()
    keep = torch.tensor(keeps, dtype=torch.int32).cuda()
    table = new_table.cuda()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    new_len, kept = sgr.sgr_kv_evict(cache, batch, got, keep, table, stream=side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sgr.sgr_kv_evict(cache, batch, got, keep, table, new_len=new_len, kept=kept)
    for lens, now in (([300, 120], [100, 100]), ([150, 119], [90, 3]), ([0, 40], [5, 100])):
        batch.seq_len.copy_(torch.tensor(lens, dtype=torch.int32))
        keep.copy_(torch.tensor(now, dtype=torch.int32))
        mass = torch.rand(pr.pages, 2, 32, generator=pr.g)
        got.copy_(mass)
        graph.replay()
        torch.cuda.synchronize()
        assert new_len.tolist() == [min(a, b) for a, b in zip(lens, now)]
        for b in range(2):
            for h in range(2):
                pages = pr.block_table[b].long()[torch.arange(lens[b]) // 32]
                want = mref.chosen(mass[pages, h, torch.arange(lens[b]) % 32].tolist(), now[b], 0, 0)
                assert kept[b, h, :len(want)].tolist() == want


def test_calls_on_two_streams_at_once():
    """Attention, masses and evictions of two caches on two streams, many times
    over, give the bits that they give one after the other."""
    jobs = []
    for k in range(2):
        pr = ref.Problem(128, 64, 2, [1500, 700], [60 + k, 3], seed=50 + k)
        keeps = [400, 300]
        new_table, more = fresh_table(pr, keeps)
        grown(pr, more)
        q = (1.5 * pr.randn(pr.tokens, 8, 128)).bfloat16().cuda()
        mass = torch.rand(pr.pages, 2, 64, generator=pr.g).cuda()
        jobs.append((pr, q, mass, torch.tensor(keeps, dtype=torch.int32).cuda(), new_table.cuda(), torch.cuda.Stream()))

    def run(job, stream):
        pr, q, mass, keep, table, _ = job
        cache, batch, mass = pr.cache(sgr), pr.batch(sgr), mass.clone()
        out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
        work = [sgr.kv_attention_workspace(cache, batch, 8), sgr.kv_mass_workspace(cache, batch, 8)]
        new_len = torch.empty(2, dtype=torch.int32, device="cuda")
        kept = torch.full((2, 2, table.shape[1] * 64), -1, dtype=torch.int32, device="cuda")
        torch.cuda.synchronize()

        def go():
            sgr.sgr_kv_attention(cache, batch, q, out=out, lse=lse, window=900, sinks=4, workspace=work[0], stream=stream)
            sgr.sgr_kv_mass(cache, batch, q, lse, mass, window=900, sinks=4, workspace=work[1], stream=stream)
            sgr.sgr_kv_evict(cache, batch, mass, keep, table, first=4, recent=70, new_len=new_len, kept=kept, stream=stream)

        return go, (out, lse, mass, kept, cache.k.view(torch.uint8), cache.v.view(torch.uint8), cache.k_scale.nan_to_num())

    want = []
    for job in jobs:
        go, outs = run(job, None)
        for _ in range(5):
            go()
        torch.cuda.synchronize()
        want.append([x.clone() for x in outs])
    both = [run(job, job[5]) for job in jobs]
    for _ in range(5):
        for go, _ in both:
            go()
    torch.cuda.synchronize()
    for (_, outs), w in zip(both, want):
        for x, y in zip(outs, w):
            assert torch.equal(x, y)


# ------------------------------------------------------------------- all together
def test_server_steps_of_trees_masses_and_evictions():
    """A prompt, its mass, an eviction, a tree of drafted tokens over what stayed,
    its accepted branch appended in its place, and a decode step with a window and
    sinks: each against the definition over the cache as it is then."""
    heads, hk, dim, page = 8, 2, 64, 16
    g = torch.Generator().manual_seed(1)
    cache = sgr.KvCache.empty(80, hk, page, dim)
    mass = cache.zero_mass()
    mass.fill_(math.nan)  # nothing needs clearing
    table = ref.rope_table(400, dim)
    rope = sgr.RopeNorm(table.cuda())
    lens = [150, 70]
    order = torch.randperm(80, generator=g).int()
    old = order[:30].view(2, 15).cuda()

    def values():
        return [(c.float() * s[:, :, None, None]).double().cpu() for c, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale))]

    def qkv(n):
        return torch.randn(n, heads + 2 * hk, dim, generator=g).bfloat16().cuda().split((heads, hk, hk), 1)

    def attend(batch, q, what, window=0, sinks=0, trees=None, words=None):
        lse = torch.empty(q.shape[:2], device="cuda")
        out = sgr.sgr_kv_attention(cache, batch, q, window=window, sinks=sinks, tree=words, lse=lse)
        k, v = values()
        start = batch.q_start.cpu() if batch.q_start is not None else None
        want, mag, want_lse, reach = mref.attention(q.cpu(), k, v, batch.block_table.cpu(), batch.seq_len.cpu(), start, page,
                                                    dim ** -0.5, window, sinks, trees)
        ref.check_attention(out, want, mag, what)
        mref.check_lse(lse, want_lse, reach, what)
        return lse

    # the prompt
    q, k, v = qkv(220)
    batch = sgr.KvBatch(old, torch.tensor(lens, dtype=torch.int32).cuda(), torch.tensor([0, 150, 220], dtype=torch.int32).cuda(),
                        tokens=220, max_new=150)
    q = sgr.sgr_kv_append(cache, batch, k, v, rope, q=q)
    lse = attend(batch, q, "prompt")
    sgr.sgr_kv_mass(cache, batch, q, lse, mass)
    before = torch.zeros(mass.shape, dtype=torch.float64)
    want, tol = mref.mass(before, q.cpu(), values()[0], lse.cpu(), old.cpu(), lens, batch.q_start.cpu(), page, dim ** -0.5)
    live = torch.zeros(mass.shape, dtype=torch.bool)
    for b in range(2):
        t = torch.arange(lens[b])
        live[old[b].cpu().long()[t // page], :, t % page] = True
    mref.check_mass(torch.where(live, mass.cpu(), 0.0), want, tol, "prompt")
    # what stays: 48 positions each, room for 16 more and a tree
    new = order[30:50].view(2, 10).cuda()
    keep = torch.tensor([48, 48], dtype=torch.int32).cuda()
    masses = mass.cpu()
    new_len, kept = sgr.sgr_kv_evict(cache, batch, mass, keep, new, first=2, recent=8)
    assert new_len.tolist() == [48, 48]
    k_old, v_old = values()
    for b in range(2):
        t = torch.arange(lens[b])
        pages = old[b].cpu().long()[t // page]
        for h in range(hk):
            stay = mref.chosen(masses[pages, h, t % page].tolist(), 48, 2, 8)
            assert kept[b, h, :48].tolist() == stay
            at = torch.arange(48)
            to = new[b].cpu().long()[at // page]
            for x in (k_old, v_old):  # the values moved, to a code's rounding (2^-4) or the least code
                a, c = x[to, h, at % page], x[pages[stay], h, torch.tensor(stay) % page]
                assert ((a - c).abs() <= 2.0 ** -4 * c.abs() + 2.0 ** -9).all()
    # a tree of 7 drafted tokens each
    r = random.Random(5)
    trees = [mref.random_tree(7, r) for _ in range(2)]
    words = torch.cat([mref.tree_words(t, 1) for t in trees]).cuda()
    depth = torch.tensor([lens[b] + len(path) - 1 for b in range(2) for path in trees[b]], dtype=torch.int32)
    batch = sgr.KvBatch(new, new_len + 7, torch.tensor([0, 7, 14], dtype=torch.int32).cuda(), tokens=14, max_new=7)
    q, k, v = qkv(14)
    q = sgr.sgr_kv_append(cache, batch, k, v, rope, q=q, positions=depth.cuda())
    k_want = ref.norm_rope(k.cpu(), None, depth, table, False, 0.0)
    for b in range(2):
        at = 48 + torch.arange(7)
        got = values()[0][new[b].cpu().long()[at // page], :, at % page]
        c = k_want[7 * b:7 * b + 7]
        assert ((got - c).abs() <= 2.0 ** -4 * c.abs() + 2.0 ** -6).all()
    attend(batch, q, "tree", trees=trees, words=words)
    # the longest branch is accepted: its tokens take the places behind the 48
    paths = [max(t, key=len) for t in trees]
    rows = torch.tensor([7 * b + j for b in range(2) for j in paths[b]]).cuda()
    count = [len(p) for p in paths]
    n = sum(count)
    batch = sgr.KvBatch(new, new_len + torch.tensor(count, dtype=torch.int32).cuda(),
                        torch.tensor([0, count[0], n], dtype=torch.int32).cuda(), tokens=n, max_new=max(count))
    q_in = torch.randn(n, heads, dim, generator=g).bfloat16().cuda()
    q = sgr.sgr_kv_append(cache, batch, k[rows], v[rows], rope, q=q_in, positions=depth.cuda()[rows])
    attend(batch, q, "accepted")
    # a decode step that sees the sinks and the last 20
    batch = sgr.KvBatch(new, new_len + torch.tensor(count, dtype=torch.int32).cuda() + 1)
    q, k, v = qkv(2)
    at = torch.tensor([lens[b] + count[b] for b in range(2)], dtype=torch.int32).cuda()
    q = sgr.sgr_kv_append(cache, batch, k, v, rope, q=q, positions=at)
    lse = attend(batch, q, "decode", window=20, sinks=3)
    before = mass.double().cpu().nan_to_num(nan=0.0)
    want, tol = mref.mass(before, q.cpu(), values()[0], lse.cpu(), new.cpu(), batch.seq_len.cpu(), None, page, dim ** -0.5, 20, 3)
    sgr.sgr_kv_mass(cache, batch, q, lse, mass, window=20, sinks=3)
    for b in range(2):
        length = int(batch.seq_len[b])
        t = torch.tensor([0, 1, 2] + list(range(length - 20, length)))
        pages = new[b].cpu().long()[t // page]
        got = mass.double().cpu()[pages, :, t % page]
        seen_before = t < 48
        w, e = want[pages, :, t % page], tol[pages, :, t % page]
        ok = seen_before | (t == length - 1)  # (the accepted ones' own masses were not asked for)
        assert ((got - w).abs() <= e)[ok].all()
