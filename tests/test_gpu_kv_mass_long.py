"""Accumulated attention weight where every CTA takes many tiles of keys: rings
that wrap, accumulators and slots of queries used again, sums of two warp groups
that meet once a tile.  Against the definition in 64 bits (tests/kv_mask_ref.py)."""
import math
import random

import pytest
import torch

import kv_mask_ref as mref
import kv_ref as ref
import skinny_bf16_gemm_residual_gb300 as sgr

pytestmark = pytest.mark.gpu

LENS = [9000, 4001, 8777, 6500, 129, 7990, 3333, 8192]


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


# rows a key/value head: new tokens of a sequence (at most) times 4
ROWS = [
    # new, window, sinks, tree
    (2, 0, 0, False),      # 8 rows
    (4, 0, 0, False),      # 16
    (5, 0, 0, False),      # 20: two groups of weighing warps from here on
    (8, 0, 0, False),      # 32
    (15, 0, 0, False),     # 60: one product of 64
    (32, 0, 0, False),     # 128: two products
    (75, 0, 0, False),     # 300: three row tiles, joined
    (8, 5000, 300, False),
    (32, 5000, 300, False),
    (32, 6000, 4, True),
]


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("new,window,sinks,tree", ROWS)
def test_mass_of_many_tiles_a_cta(dim, new, window, sinks, tree):
    hk, heads, page = 4, 16, 64
    r = random.Random(new + dim)
    count = [new] + [r.randint(max(new // 2, 1), new) for _ in LENS[1:]]
    pr = ref.Problem(dim, page, hk, LENS, count, seed=new)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    most = window + sinks if window else max(LENS)
    assert hk * sum(min(l, most) // 128 for l in LENS) > 3 * 2 * sms  # tiles of keys; two CTAs an SM
    trees = [mref.random_tree(n, r) for n in count] if tree else None
    words = torch.cat([mref.tree_words(t, -(-new // 64)) for t in trees]).cuda() if tree else None
    cache, batch = pr.cache(sgr), pr.batch(sgr)
    q = (1.5 * pr.randn(pr.tokens, heads, dim)).bfloat16()
    lse = torch.empty(pr.tokens, heads, device="cuda")
    masks = dict(window=window, sinks=sinks, tree=words)
    sgr.sgr_kv_attention(cache, batch, q.cuda(), lse=lse, **masks)
    before = torch.rand(pr.pages, hk, page, generator=pr.g)
    got = sgr.sgr_kv_mass(cache, batch, q.cuda(), lse, before.cuda(), **masks)
    for _ in range(20):  # the same bits on every run
        again = sgr.sgr_kv_mass(cache, batch, q.cuda(), lse, before.cuda(), **masks)
        assert torch.equal(again, got)
    assert lse.isfinite().all() and math.isfinite(float(got.sum()))
    mref.check_mass(got, *mref.mass(before.double(), q, pr.values(0), lse.cpu(), pr.block_table, pr.seq_len, pr.q_start, page,
                                    dim ** -0.5, window, sinks, trees))


@pytest.mark.parametrize("page,window,sinks", [(16, 70, 5), (32, 1, 33), (64, 300, 0)])
@pytest.mark.parametrize("entry", ["another page", "none"])
def test_mass_follows_no_entry_of_a_page_that_no_row_sees(page, window, sinks, entry):
    """Several row tiles under a window: entries between the sinks and the first
    window name a page that is another's (its masses are -0.0, which an addition of
    zero would make +0.0), or none (which would be recorded)."""
    new = 180
    pr = ref.Problem(64, page, 2, [1000, 700], [new, new - 1], seed=window, extra_pages=3)
    other = pr.pages - 1
    while other in pr.block_table.tolist()[0] or other in pr.block_table.tolist()[1]:
        other -= 1
    table = pr.block_table.clone()
    hidden = 0
    for b in range(2):
        first = pr.lens[b] - pr.new[b]
        for block in range(pr.max_pages):
            if block * page >= sinks and (block + 1) * page <= first - window + 1:
                table[b, block] = other if entry == "another page" else -1
                hidden += 1
    assert hidden > 4
    q = (1.5 * pr.randn(pr.tokens, 4, 64)).bfloat16()
    batch = sgr.KvBatch(table.cuda(), pr.seq_len.cuda(), pr.q_start.cuda(), tokens=pr.tokens, max_new=new)
    cache = pr.cache(sgr)
    lse = torch.empty(pr.tokens, 4, device="cuda")
    sgr.sgr_kv_attention(cache, batch, q.cuda(), lse=lse, window=window, sinks=sinks)
    assert sgr.kv_mass_workspace(cache, batch, 4).numel() > 0
    before = torch.rand(pr.pages, 2, page, generator=pr.g)
    before[other] = -0.0
    got = sgr.sgr_kv_mass(cache, batch, q.cuda(), lse, before.cuda(), window=window, sinks=sinks)
    assert (got[other].signbit() & (got[other] == 0)).all()
    mref.check_mass(got, *mref.mass(before.double(), q, pr.values(0), lse.cpu(), pr.block_table, pr.seq_len, pr.q_start, page,
                                    0.125, window, sinks))


@pytest.mark.parametrize("new", [1, 9, 100])  # rows a head: 4, 36, 400 (the last: several row tiles, joined)
def test_mass_of_shared_pages(new):
    """Twelve sequences with a common prompt, and pages of their own behind it: a
    shared position gets the weights of all.  The error allowed is the sum of the
    sequences' own."""
    page, heads, hk, shared, count = 32, 8, 2, 20, 12
    lens = [shared * page + r for r in range(new, new + 7 * count, 7)]
    pr = ref.Problem(128, page, hk, lens, [new] * count, seed=new)
    pr.block_table[:, :shared] = pr.block_table[0, :shared]
    q = (1.5 * pr.randn(pr.tokens, heads, 128)).bfloat16()
    cache, batch = pr.cache(sgr), pr.batch(sgr)
    lse = torch.empty(pr.tokens, heads, device="cuda")
    sgr.sgr_kv_attention(cache, batch, q.cuda(), lse=lse)
    before = torch.rand(pr.pages, hk, page, generator=pr.g)
    want, tol = before.double(), torch.zeros_like(before, dtype=torch.float64)
    for b in range(count):
        rows = slice(new * b, new * (b + 1))
        want, more = mref.mass(want, q[rows], pr.values(0), lse[rows].cpu(), pr.block_table[b:b + 1], pr.seq_len[b:b + 1],
                               torch.tensor([0, new]), page, 128 ** -0.5)
        tol += more
    for _ in range(5):
        got = sgr.sgr_kv_mass(cache, batch, q.cuda(), lse, before.cuda())
        mref.check_mass(got, want, tol)
