"""Attention under windows with sinks and over trees of drafted tokens, its
log-sum-exp, and the append to given positions, on the GPU against their
definitions in 64 bits (tests/kv_mask_ref.py)."""
import math
import random

import pytest
import torch

import kv_mask_ref as mref
import kv_ref as ref
import skinny_bf16_gemm_residual_gb300 as sgr

pytestmark = pytest.mark.gpu
FEW, MANY = sgr.SGR_FLAG_KV_FEW_ROWS, sgr.SGR_FLAG_KV_MANY_ROWS


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


def attend(pr, heads, flags=0, window=0, sinks=0, trees=None, words=None, factor=1.5, q=None, check=True):
    """One call against the definition; rows of NaN beforehand show what is not written."""
    if q is None:
        q = (factor * pr.randn(pr.tokens, heads, pr.dim)).bfloat16()
    tree = None
    if trees is not None:
        tree = torch.cat([mref.tree_words(t, words) for t in trees]).cuda()
    out = torch.full((pr.tokens, heads, pr.dim), math.nan, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((pr.tokens, heads), math.nan, device="cuda")
    got = sgr.sgr_kv_attention(pr.cache(sgr), pr.batch(sgr), q.cuda(), out=out, window=window, sinks=sinks, tree=tree,
                               lse=lse, flags=flags)
    assert got is out
    if check:
        want, mag, want_lse, reach = mref.attention(q, pr.values(0), pr.values(1), pr.block_table, pr.seq_len, pr.q_start,
                                                    pr.page, pr.dim ** -0.5, window, sinks, trees)
        ref.check_attention(out, want, mag)
        mref.check_lse(lse, want_lse, reach)
    return out, lse


def hide_gap(pr, window, sinks, trees=False):
    """Pages that no row sees get no entry in the table: reading it would be recorded."""
    for b, (length, n) in enumerate(zip(pr.lens, pr.new)):
        first = max(length - n, 0)
        for block in range(-(-length // pr.page)):
            if block * pr.page >= sinks and (block + 1) * pr.page <= first - window + 1:
                pr.block_table[b, block] = -1


SINKS = [
    # dim, page, heads, hk, lens, new, window, sinks
    (128, 64, 7, 1, [1], [1], 1, 1),
    (128, 64, 28, 4, [2000, 333, 90], [1, 1, 1], 100, 4),
    (64, 16, 8, 2, [1000, 150, 140, 129, 1], [1, 1, 1, 1, 1], 20, 1),        # sinks and window in one tile, with a gap
    (64, 16, 8, 2, [700, 400], [1, 1], 129, 200),                            # sinks past a tile, window inside them
    (128, 128, 8, 2, [1500, 385, 0], [3, 2, 1], 128, 128),                   # both on tile borders
    (64, 32, 6, 2, [900, 30], [40, 35], 33, 300),                            # more rows; padding rows
    (128, 32, 24, 1, [1100, 200], [70, 200], 64, 7),                         # a chunk, a whole prompt
    (128, 16, 4, 4, [3000], [130], 1000, 1024),
    (64, 64, 16, 4, [640], [64], 1, 2),
    (64, 128, 3, 1, [500], [2], 600, 8),                                     # a window that leaves nothing out
    (128, 64, 2, 2, [777], [1], 10, 5000),                                   # sinks past the end
]


@pytest.mark.parametrize("flags", [FEW, MANY, 0])
@pytest.mark.parametrize("dim,page,heads,hk,lens,new,window,sinks", SINKS)
def test_sinks(dim, page, heads, hk, lens, new, window, sinks, flags):
    pr = ref.Problem(dim, page, hk, lens, new, seed=window + sinks)
    hide_gap(pr, window, sinks)
    attend(pr, heads, flags, window, sinks)


@pytest.mark.parametrize("flags", [FEW, MANY])
def test_sinks_of_nothing_are_a_window(flags):
    """sinks = 0, and sinks without a window: the bits of the calls without them."""
    pr = ref.Problem(64, 32, 2, [900, 130], [3, 20], seed=5)
    q = pr.randn(23, 8, 64).bfloat16()
    for window, sinks in ((100, 0), (0, 0), (0, 9)):
        out, _ = attend(pr, 8, flags, window, sinks, q=q)
        plain = sgr.sgr_kv_attention(pr.cache(sgr), pr.batch(sgr), q.cuda(), window=window, flags=flags)
        assert torch.equal(out, plain)


@pytest.mark.parametrize("flags", [FEW, MANY])
def test_nan_between_sinks_and_window_has_no_influence(flags):
    """NaN codes and scales between the sinks and the first window, in tiles and
    pages that hold sinks or windows too, and NaN that one row sees and another does not."""
    for window, sinks, n in ((40, 10, 1), (40, 10, 3), (150, 70, 30)):
        pr = ref.Problem(128, 64, 1, [400], [n], seed=n)
        first = 400 - n
        for which in (0, 1):
            for t in range(sinks, first - window + 1):
                pr.codes[which][int(pr.block_table[0, t // 64]), 0, t % 64] = ref.NAN_CODE
        out, lse = attend(pr, 6, flags, window, sinks)
        assert out.isfinite().all() and lse.isfinite().all()
        t = first - window + 1  # the first row's window begins here; later rows do not see it
        pr.codes[1][int(pr.block_table[0, t // 64]), 0, t % 64, 3] = ref.NAN_CODE
        out, _ = attend(pr, 6, flags, window, sinks)
        assert out[0, :, 3].isnan().all() and out[1:].isfinite().all() and out[0, :, :3].isfinite().all()


TREES = [
    # dim, page, heads, hk, lens, new, window, sinks
    (128, 64, 7, 1, [5], [5], 0, 0),                           # nothing before the tree
    (128, 64, 28, 4, [300, 70], [7, 3], 0, 0),
    (64, 16, 8, 2, [260, 135, 128], [25, 9, 1], 0, 0),         # trees across tiles and pages
    (128, 128, 16, 2, [700, 140], [64, 40], 0, 0),             # one word exactly
    (64, 32, 4, 1, [500, 70], [65, 70], 0, 0),                 # two words
    (128, 32, 8, 1, [1000], [150], 0, 0),                      # three, rows in many tiles
    (64, 64, 12, 2, [3, 0, 200], [5, 2, 4], 0, 0),             # padding rows
    (128, 16, 6, 2, [900, 300], [20, 33], 64, 5),              # a window with sinks
    (64, 128, 32, 4, [600], [30], 1, 0),                       # a window that leaves the tree and its root's place
    (128, 64, 3, 3, [400], [12], 3, 130),
]


@pytest.mark.parametrize("flags", [FEW, MANY, 0])
@pytest.mark.parametrize("dim,page,heads,hk,lens,new,window,sinks", TREES)
def test_tree(dim, page, heads, hk, lens, new, window, sinks, flags):
    pr = ref.Problem(dim, page, hk, lens, new, seed=sum(new))
    r = random.Random(sum(lens))
    attend(pr, heads, flags, window, sinks, [mref.random_tree(n, r) for n in new], -(-max(new) // 64))


@pytest.mark.parametrize("flags", [FEW, MANY])
def test_tree_of_any_bits(flags):
    """Bits that are no tree: rows that see others but not themselves, later
    ones, none at all; bits past the new tokens and words past them do not count."""
    pr = ref.Problem(64, 32, 2, [180, 4], [60, 4], seed=7)
    r = random.Random(3)
    trees = [[sorted(r.sample(range(n), r.randint(0, n))) for _ in range(n)] for n in pr.new]
    trees[0][5] = []
    trees[1] = [[], [1, 3], [], [0]]  # of a sequence that is all new: rows that see nothing
    q = pr.randn(64, 8, 64).bfloat16()
    q[60] = math.nan  # the first row of the second sequence, which sees nothing
    attend(pr, 8, flags, trees=trees, words=1, q=q)
    beyond = [[t + [n, n + 1, 63, 100] if n < 60 else t + [60, 61, 70] for t in paths] for n, paths in zip(pr.new, trees)]
    tree = torch.cat([mref.tree_words(t, 3) for t in beyond]).cuda()
    want = torch.cat([mref.tree_words(t, 1) for t in trees]).cuda()
    for window in (0, 20):
        a, b = (sgr.sgr_kv_attention(pr.cache(sgr), pr.batch(sgr), q.cuda(), tree=t, window=window, flags=flags)
                for t in (tree, want))
        assert torch.equal(a, b)


@pytest.mark.parametrize("flags", [FEW, MANY])
def test_chain_is_the_causal_mask(flags):
    """A tree without branches gives the bits of the call without a tree."""
    pr = ref.Problem(128, 64, 2, [500, 130, 40], [70, 3, 50], seed=11)
    q = pr.randn(pr.tokens, 8, 128).bfloat16().cuda()
    tree = torch.cat([mref.tree_words([list(range(i + 1)) for i in range(n)], 2) for n in pr.new]).cuda()
    for window, sinks in ((0, 0), (200, 0), (200, 20)):
        a = sgr.sgr_kv_attention(pr.cache(sgr), pr.batch(sgr), q, window=window, sinks=sinks, flags=flags)
        b = sgr.sgr_kv_attention(pr.cache(sgr), pr.batch(sgr), q, window=window, sinks=sinks, tree=tree, flags=flags)
        rows = slice(0, pr.tokens) if not window else slice(70, pr.tokens)  # (a window counts between a tree's tokens nowhere)
        assert torch.equal(a[rows], b[rows]), (window, sinks)


@pytest.mark.parametrize("flags", [FEW, MANY])
@pytest.mark.parametrize("dim", [64, 128])
def test_nan_of_another_branch(dim, flags):
    """A NaN key or value of one branch reaches the rows of its own branch only."""
    for which in (0, 1):
        pr = ref.Problem(dim, 32, 1, [139], [12], seed=4 + which)  # positions 127 .. 138
        trees = [mref.random_tree(12, random.Random(5))]
        at = 127 + 3
        pr.codes[which][int(pr.block_table[0, at // 32]), 0, at % 32, 5] = ref.NAN_CODE
        out, _ = attend(pr, 5, flags, trees=trees, words=1)
        hit = torch.tensor([3 in path for path in trees[0]])
        assert 0 < int(hit.sum()) < 12
        assert torch.equal(out.isnan().any(-1).any(-1).cpu(), hit)


@pytest.mark.parametrize("flags", [FEW, MANY])
def test_log_sum_exp_of_split_and_far_scores(flags):
    """The log-sum-exp of sequences over the whole GPU and of scores far from zero."""
    pr = ref.Problem(128, 128, 2, [20001, 3000, 0], [1, 2, 1], seed=13)
    for factor in (0.0, 1.5, 40.0):
        attend(pr, 8, flags, factor=factor)


@pytest.mark.parametrize("flags", [FEW, MANY])
def test_strided_tree_other_stream_and_replay(flags):
    """Tree words of a wider buffer; a captured call replays with another tree and lengths."""
    pr = ref.Problem(64, 32, 2, [300, 100], [30, 30], seed=21)
    r = random.Random(2)
    q = pr.randn(60, 8, 64).bfloat16()
    cache, batch, x = pr.cache(sgr), pr.batch(sgr), q.cuda()
    wide = torch.full((60, 5), -1, dtype=torch.int64, device="cuda")
    tree = wide[:, 1:3]
    trees = [mref.random_tree(30, r) for _ in range(2)]
    tree.copy_(torch.cat([mref.tree_words(t, 2) for t in trees]))
    out, lse = torch.empty_like(x), torch.empty(60, 8, device="cuda")
    work = sgr.kv_attention_workspace(cache, batch, 8, flags)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    sgr.sgr_kv_attention(cache, batch, x, out=out, tree=tree, lse=lse, workspace=work, flags=flags, stream=side)
    side.synchronize()

    def check(what):
        want, mag, want_lse, reach = mref.attention(q, pr.values(0), pr.values(1), pr.block_table, batch.seq_len.cpu(),
                                                    pr.q_start, 32, 0.125, 50, 4, trees) if what != "side" else mref.attention(
            q, pr.values(0), pr.values(1), pr.block_table, pr.seq_len, pr.q_start, 32, 0.125, 0, 0, trees)
        ref.check_attention(out, want, mag, what)
        mref.check_lse(lse, want_lse, reach, what)

    check("side")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sgr.sgr_kv_attention(cache, batch, x, out=out, tree=tree, lse=lse, workspace=work, flags=flags, window=50, sinks=4)
    for lens in ([299, 31], [40, 12]):
        trees = [mref.random_tree(30, r) for _ in range(2)]
        tree.copy_(torch.cat([mref.tree_words(t, 2) for t in trees]))
        batch.seq_len.copy_(torch.tensor(lens, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        check(f"replay {lens}")


def test_log_sum_exp_rows_of_no_sequence_are_left():
    pr = ref.Problem(64, 16, 2, [40, 21], [3, 1])
    batch = sgr.KvBatch(pr.block_table.cuda(), pr.seq_len.cuda(), pr.q_start.cuda(), tokens=6, max_new=3)
    x = pr.randn(6, 2, 64).bfloat16().cuda()
    for flags in (FEW, MANY):
        lse = torch.full((6, 2), 7.0, device="cuda")
        sgr.sgr_kv_attention(pr.cache(sgr), batch, x, lse=lse, flags=flags)
        assert (lse[4:] == 7).all() and not (lse[:4] == 7).any()


@pytest.mark.parametrize("dim,page,heads,hk,lens,new", [
    (128, 32, 4, 2, [13, 319], [2, 107]), (64, 16, 24, 2, [2000] * 5, [30] * 5), (128, 64, 28, 4, [9000], [7]),
    (128, 128, 8, 1, [5000, 70], [200, 3]), (64, 64, 8, 8, [4000] * 40, [5] * 40)])
def test_workspace_is_enough_for_any_window(dim, page, heads, hk, lens, new):
    """The workspace depends on the sizes alone; a window may change the row tiles."""
    pr = ref.Problem(dim, page, hk, [1] * len(lens), [1] * len(lens), extra_pages=4)  # (no position is looked at)
    cache = pr.cache(sgr)
    table = torch.zeros(len(lens), -(-max(lens) // page), dtype=torch.int32, device="cuda")
    start = torch.zeros(len(lens) + 1, dtype=torch.int32, device="cuda")  # no rows
    batch = sgr.KvBatch(table, torch.zeros(len(lens), dtype=torch.int32, device="cuda"), start, tokens=sum(new), max_new=max(new))
    q = torch.zeros(sum(new), heads, dim, dtype=torch.bfloat16, device="cuda")
    for flags in (0, FEW, MANY):
        work = sgr.kv_attention_workspace(cache, batch, heads, flags)
        for window in (0, 1, 30, 100, 300, 700, 1000, 2000, 4000, 100000):
            for sinks in (0, 4, 600):
                sgr.sgr_kv_attention(cache, batch, q, window=window, sinks=sinks, workspace=work, flags=flags)


# ------------------------------------------------------------------------- append
@pytest.mark.parametrize("dim,interleaved", [(64, True), (128, False)])
def test_append_to_given_positions(dim, interleaved):
    """Queries and keys rotated to other positions than their places; codes and
    scales where the call without positions puts them."""
    pr = ref.Problem(dim, 32, 2, [100, 3, 64], [37, 5, 1], seed=dim)  # (the second: two padding rows)
    table = ref.rope_table(400, dim)
    w = (1 + 0.3 * pr.randn(dim)).bfloat16()
    on = sgr.RopeNorm(table.cuda(), k_weight=w.cuda(), eps=1e-6, interleaved=interleaved)
    qkv = pr.randn(pr.tokens, 8, dim).bfloat16()
    pos = torch.randint(0, 400, (pr.tokens,), generator=pr.g, dtype=torch.int32)
    cache, batch = pr.cache(sgr), pr.batch(sgr)
    q, k, v = qkv.cuda().split((4, 2, 2), 1)
    q_out = sgr.sgr_kv_append(cache, batch, k, v, on, q=q, positions=pos.cuda())
    want_q = ref.norm_rope(qkv[:, :4], None, pos, table, interleaved, 1e-6)
    want_q[37:39] = 0
    ref.check_bf16(q_out, want_q, "q")
    k_new = ref.norm_rope(qkv[:, 4:6], w, pos, table, interleaved, 1e-6)
    for i, (x, got, scale) in enumerate(((k_new, cache.k, cache.k_scale), (qkv[:, 6:].double(), cache.v, cache.v_scale))):
        want, want_scale = ref.append(pr.codes[i], pr.scale[i], x, pr.block_table, pr.seq_len, pr.q_start, 32)
        used = ~want_scale.isnan().any(1)
        ref.check_append(got.view(torch.uint8).cpu()[used], scale.cpu()[used], pr.codes[i][used], want[used], want_scale[used])
    # the places themselves as positions: the bits of the call without
    place = torch.cat([torch.arange(l - n, l) for l, n in zip(pr.lens, pr.new)]).int()
    a, b = pr.cache(sgr), pr.cache(sgr)
    qa = sgr.sgr_kv_append(a, batch, k, v, on, q=q, positions=place.cuda())
    qb = sgr.sgr_kv_append(b, batch, k, v, on, q=q)
    assert torch.equal(qa, qb) and torch.equal(a.k.view(torch.uint8), b.k.view(torch.uint8))


def test_append_to_a_bad_position_is_recorded():
    pr = ref.Problem(64, 16, 1, [20], [2])
    on = sgr.RopeNorm(ref.rope_table(8, 64).cuda())
    x = pr.randn(2, 2, 1, 64).bfloat16().cuda()
    for bad in (-1, 8, -(1 << 31), (1 << 31) - 1):
        cache = pr.cache(sgr)
        sgr.sgr_kv_append(cache, pr.batch(sgr), x[0], x[1], on, positions=torch.tensor([3, bad], dtype=torch.int32).cuda())
        assert sgr.sgr_device_error(0) == 7
        other = pr.cache(sgr)
        sgr.sgr_kv_append(other, pr.batch(sgr), x[0], x[1], on,
                          positions=torch.tensor([3, 0 if bad < 0 else 7], dtype=torch.int32).cuda())
        assert torch.equal(cache.k.view(torch.uint8), other.k.view(torch.uint8))
