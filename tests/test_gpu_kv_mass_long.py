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
