"""The attention operators on the GPU against their 64-bit definitions
(tests/kv_ref.py): head norms with rotation, append, attention."""
import math

import pytest
import torch

import kv_ref as ref
import skinny_bf16_gemm_residual_gb300 as sgr

pytestmark = pytest.mark.gpu
EPS = 1e-6
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


def norm_rope_args(dim, rot, interleaved, norm, rows, g):
    w = [(1 + 0.3 * torch.randn(dim, generator=g)).bfloat16() if n else None for n in norm]
    table = ref.rope_table(rows, rot) if rot else None
    on = sgr.RopeNorm(None if table is None else table.cuda(), *(None if x is None else x.cuda() for x in w), eps=EPS,
                      interleaved=interleaved)
    return w, table, on


# ---------------------------------------------------------------- norm + rotation
@pytest.mark.parametrize("dim,rot,interleaved,norm", [
    (128, 128, False, (True, True)), (128, 64, True, (True, False)), (128, 96, False, (False, True)),
    (64, 64, True, (True, True)), (64, 16, False, (False, False)), (64, 0, False, (True, True)),
    (128, 0, False, (False, True)),
])
@pytest.mark.parametrize("tokens,heads,hk", [(1, 1, 1), (3, 28, 4), (37, 5, 0), (200, 24, 8)])
def test_qk_norm_rope(dim, rot, interleaved, norm, tokens, heads, hk):
    g = torch.Generator().manual_seed(tokens + heads)
    w, table, on = norm_rope_args(dim, rot, interleaved, norm, 517, g)
    qkv = torch.randn(tokens, heads + 2 * hk, dim, generator=g).bfloat16()
    pos = torch.randint(0, 517, (tokens,), generator=g, dtype=torch.int32)
    dev = qkv.cuda()
    k = dev[:, heads:heads + hk] if hk else None
    q, k = sgr.sgr_qk_norm_rope(dev[:, :heads], k, pos.cuda(), on)
    ref.check_bf16(q, ref.norm_rope(qkv[:, :heads], w[0], pos, table, interleaved, EPS), "q")
    if hk:
        ref.check_bf16(k, ref.norm_rope(qkv[:, heads:heads + hk], w[1], pos, table, interleaved, EPS), "k")


def test_qk_norm_rope_in_place_head_major_and_padding():
    g = torch.Generator().manual_seed(5)
    w, table, on = norm_rope_args(128, 128, False, (True, True), 64, g)
    q0, k0 = (torch.randn(h, 9, 128, generator=g).bfloat16() for h in (6, 2))
    pos = torch.tensor([3, -1, 63, 0, 1, 2, -7, 5, 6], dtype=torch.int32)
    q, k = q0.cuda().transpose(0, 1), k0.cuda().transpose(0, 1)  # [heads, tokens, dim] in memory
    a, b = sgr.sgr_qk_norm_rope(q, k, pos.cuda(), on, q_out=q, k_out=k)
    assert a is q and b is k
    for got, x, wt in ((q, q0, w[0]), (k, k0, w[1])):
        want = ref.norm_rope(x.transpose(0, 1), wt, pos, table, False, EPS)
        want[pos < 0] = 0
        ref.check_bf16(got, want)


def test_position_beyond_the_table_is_recorded():
    g = torch.Generator().manual_seed(6)
    _, _, on = norm_rope_args(64, 64, False, (False, False), 8, g)
    q = torch.randn(2, 1, 64, generator=g).bfloat16().cuda()
    sgr.sgr_qk_norm_rope(q, None, torch.tensor([7, 8], dtype=torch.int32).cuda(), on)
    assert sgr.sgr_device_error(0) == 7


# ------------------------------------------------------------------------- append
APPEND = [
    # dim, page, hk, lens (with the new tokens), new
    (128, 64, 4, [1], [1]),
    (128, 16, 1, [16, 17, 18, 31, 33], [1, 1, 1, 1, 1]),
    (64, 16, 3, [5, 90, 47], [5, 40, 16]),
    (128, 32, 2, [100, 3, 64], [100, 2, 33]),
    (64, 128, 2, [130, 128, 127, 300], [3, 1, 127, 290]),
    (128, 128, 1, [129, 256, 1000], [2, 128, 999]),
    (64, 64, 2, [0, 3, 70, 2], [1, 5, 0, 3]),  # padding rows, a sequence without rows
]


@pytest.mark.parametrize("heads_inside", [False, True])
@pytest.mark.parametrize("dim,page,hk,lens,new", APPEND)
def test_append(dim, page, hk, lens, new, heads_inside):
    pr = ref.Problem(dim, page, hk, lens, new, seed=sum(lens), heads_inside=heads_inside)
    heads = 3 * hk
    w, table, on = norm_rope_args(dim, dim // 2, heads_inside, (True, True), max(lens) + 1, pr.g)
    qkv = (pr.randn(pr.tokens, heads + 2 * hk, dim) * torch.exp2(3 * pr.randn(pr.tokens, heads + 2 * hk, 1))).bfloat16()
    pos = torch.cat([torch.arange(l - n, l) for l, n in zip(lens, new)])
    cache, batch, dev = pr.cache(sgr), pr.batch(sgr), qkv.cuda()
    q, k, v = dev.split((heads, hk, hk), 1)
    before = [c.clone() for c in pr.codes]
    for again in range(2):  # the same rows again change nothing
        q_out = sgr.sgr_kv_append(cache, batch, k, v, on, q=q)
        want_q = ref.norm_rope(qkv[:, :heads], w[0], pos, table, heads_inside, EPS)
        want_q[pos < 0] = 0
        ref.check_bf16(q_out, want_q, "q")
        k_new = ref.norm_rope(qkv[:, heads:heads + hk], w[1], pos, table, heads_inside, EPS)
        for i, (x, got, scale) in enumerate(((k_new, cache.k, cache.k_scale), (qkv[:, heads + hk:].double(), cache.v, cache.v_scale))):
            want, want_scale = ref.append(before[i], pr.scale[i], x, pr.block_table, pr.seq_len, pr.q_start, page)
            used = ~want_scale.isnan().any(1)  # pages of nobody keep their NaN scales
            assert torch.equal(scale.cpu().isnan().any(1), ~used)
            ref.check_append(got.view(torch.uint8).cpu()[used], scale.cpu()[used], before[i][used], want[used], want_scale[used],
                             f"{'kv'[i]} {again}")
            assert torch.equal(got.view(torch.uint8).cpu()[~used], before[i][~used])


def test_append_without_queries_norm_or_rotation():
    pr = ref.Problem(128, 32, 2, [40, 5], [3, 5])
    x = pr.randn(2, pr.tokens, 2, 128).bfloat16()
    cache, batch = pr.cache(sgr), pr.batch(sgr)
    assert sgr.sgr_kv_append(cache, batch, x[0].cuda(), x[1].cuda(), sgr.RopeNorm()) is None
    for i, (got, scale) in enumerate(((cache.k, cache.k_scale), (cache.v, cache.v_scale))):
        want, want_scale = ref.append(pr.codes[i], pr.scale[i], x[i].double(), pr.block_table, pr.seq_len, pr.q_start, 32)
        used = ~want_scale.isnan().any(1)
        ref.check_append(got.view(torch.uint8).cpu()[used], scale.cpu()[used], pr.codes[i][used], want[used], want_scale[used])


def test_append_scale_boundaries_and_non_finite_values():
    """Powers of two exactly at the largest code, zeros, the clamped ends, and
    infinities and NaN, which do not count for the scale."""
    rows = [448.0, 449.0, 447.0 * 2.0 ** -10, 0.0, 2.0 ** -90, 3e38, math.inf, math.nan]
    n = len(rows)
    cache = sgr.KvCache.empty(n, 1, 16, 64)
    table = torch.arange(n, dtype=torch.int32).view(n, 1).cuda()
    batch = sgr.KvBatch(table, torch.ones(n, dtype=torch.int32).cuda())
    x = torch.ones(n, 1, 64)
    x[:, 0, 3] = torch.tensor(rows)
    x[3:5] = x[3:5] * 0 + torch.tensor(rows)[3:5, None, None]
    x = x.bfloat16()
    sgr.sgr_kv_append(cache, batch, x.cuda(), -x.cuda(), sgr.RopeNorm())
    top = [float(r[torch.isfinite(r)].abs().max()) for r in x[:, 0].double()]
    want = torch.tensor([2.0 ** ref.scale_exp(t) for t in top])
    for codes, scale, sign in ((cache.k, cache.k_scale, 1), (cache.v, cache.v_scale, -1)):
        assert torch.equal(scale[:, 0].cpu(), want)
        got = codes[:, 0, 0].float().cpu()
        assert torch.equal(got[0, :4], sign * torch.tensor([1.0, 1.0, 1.0, 448.0]))
        assert (got[3] == 0).all() and (got[4] == 0).all()
        assert got[5, 3] == sign * 448 and got[6, 3] == sign * 448 and got[7, 3].isnan()
        assert torch.equal(got[6, 4:], sign * torch.full((60,), 256.0)) and not got[7, 4:].isnan().any()


def test_bad_pages_and_rows_are_recorded_and_skipped():
    pr = ref.Problem(64, 16, 1, [20, 20], [1, 1])
    x = pr.randn(2, 2, 1, 64).bfloat16().cuda()
    on = sgr.RopeNorm()
    before = pr.cache(sgr)
    for change in ("page", "length", "rows"):
        cache = pr.cache(sgr)
        table, lens, start = pr.block_table.clone(), pr.seq_len.clone(), pr.q_start.clone()
        if change == "page":
            table[0, 1] = pr.pages
        elif change == "length":
            lens[0] = 16 * table.shape[1] + 1
        else:
            start[0] = -5
        batch = sgr.KvBatch(table.cuda(), lens.cuda(), start.cuda(), tokens=2)
        sgr.sgr_kv_append(cache, batch, x[0], x[1], on)
        assert sgr.sgr_device_error(0) == 7, change
        page = int(pr.block_table[1, 1])  # the other sequence's token is there
        assert not torch.equal(cache.k[page].view(torch.uint8), before.k[page].view(torch.uint8))
        if change != "rows":
            page = int(pr.block_table[0, 1])
            if change == "page":
                assert torch.equal(cache.k[page].view(torch.uint8), before.k[page].view(torch.uint8))
        o = sgr.sgr_kv_attention(cache, batch, x[0])
        assert sgr.sgr_device_error(0) == 7, change
        assert o[1].isfinite().all()


# ---------------------------------------------------------------------- attention
ATTEND = [
    # dim, page, heads, hk, lens, new, window
    (128, 64, 7, 1, [1], [1], 0),
    (128, 64, 28, 4, [333], [1], 0),
    (64, 16, 8, 8, [127, 128, 129, 1, 16], [1, 1, 1, 1, 1], 0),
    (128, 16, 16, 1, [700, 0, 257], [1, 1, 1], 0),
    (128, 128, 8, 2, [5, 640, 641], [1, 1, 1], 0),
    (64, 32, 5, 1, [300, 90], [4, 6], 0),
    (128, 32, 12, 2, [513, 40, 3], [5, 40, 7], 0),     # a prompt, rows before the first position
    (128, 64, 6, 2, [1000, 300, 64], [1, 3, 2], 100),
    (64, 64, 4, 4, [2000], [70], 129),
    (64, 128, 32, 2, [290, 140], [33, 9], 0),
    (128, 32, 40, 1, [400], [2], 1),
    (128, 16, 24, 1, [900, 200], [30, 200], 0),        # rows in many row tiles, a whole prompt
    (64, 32, 9, 3, [700, 130, 5], [100, 1, 5], 64),
    (128, 128, 16, 2, [1300], [17], 1000),
]


@pytest.mark.parametrize("dim,page,heads,hk,lens,new,window", ATTEND)
@pytest.mark.parametrize("heads_inside,flags", [(False, FEW), (True, 0), (False, MANY)])
def test_attention(dim, page, heads, hk, lens, new, window, heads_inside, flags):
    pr = ref.Problem(dim, page, hk, lens, new, seed=heads, heads_inside=heads_inside)
    q = (2 * pr.randn(pr.tokens, heads + 2, dim)).bfloat16()
    want, mag = ref.attention(q[:, :heads], pr.values(0), pr.values(1), pr.block_table, pr.seq_len, pr.q_start, page,
                              dim ** -0.5, window)
    cache, batch = pr.cache(sgr), pr.batch(sgr)
    got = sgr.sgr_kv_attention(cache, batch, q.cuda()[:, :heads], window=window, flags=flags)
    ref.check_attention(got, want, mag)
    again = torch.full((heads, pr.tokens, dim), 7.0, dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    sgr.sgr_kv_attention(cache, batch, q.cuda()[:, :heads], out=again, window=window, flags=flags)
    assert torch.equal(again, got)  # the same bits in another layout


@pytest.mark.parametrize("flags", [FEW, MANY])
def test_attention_sharp_and_shifted_scores(flags):
    """Scores far apart (one position takes nearly all the weight), far from
    zero, and a spike over a long flat tail."""
    pr = ref.Problem(128, 64, 2, [3000, 500], [1, 1], seed=3)
    q = pr.randn(2, 8, 128)
    for factor, what in ((60.0, "sharp"), (0.0, "flat"), (1e4, "one position"), (1e-30, "tiny")):
        x = (q * factor).bfloat16()
        want, mag = ref.attention(x, pr.values(0), pr.values(1), pr.block_table, pr.seq_len, None, 64, 128 ** -0.5, 0)
        got = sgr.sgr_kv_attention(pr.cache(sgr), pr.batch(sgr, False), x.cuda(), flags=flags)
        if factor <= 60:
            ref.check_attention(got, want, mag, what)
        else:
            assert got.isfinite().all()
    # spike: position 0 has 13 nats more than 2999 equal others
    cache = sgr.KvCache.empty(50, 1, 64, 64)
    n = 3000
    k, v = torch.zeros(n, 1, 64), torch.randn(n, 1, 64, generator=pr.g)
    k[0, 0, 0] = 13.0
    batch = sgr.KvBatch(torch.arange(50, dtype=torch.int32).view(1, 50).cuda(), torch.tensor([n], dtype=torch.int32).cuda(),
                        torch.tensor([0, n], dtype=torch.int32).cuda(), tokens=n, max_new=n)
    sgr.sgr_kv_append(cache, batch, k.bfloat16().cuda(), v.bfloat16().cuda(), sgr.RopeNorm())
    x = torch.zeros(1, 1, 64)
    x[0, 0, 0] = 8.0
    kk, vv = (c.float().double().cpu() * s.double().cpu()[:, :, None, None] for c, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)))
    want, mag = ref.attention(x, kk, vv, batch.block_table.cpu(), [n], None, 64, 0.125, 0)
    got = sgr.sgr_kv_attention(cache, sgr.KvBatch(batch.block_table, batch.seq_len), x.bfloat16().cuda(), flags=flags)
    ref.check_attention(got, want, mag, "spike")


@pytest.mark.parametrize("flags", [FEW, MANY])
@pytest.mark.parametrize("scale", [-0.3, 0.0, 1.0])
def test_other_scales(scale, flags):
    """Negative, zero and unit factors of the scores, few rows and many."""
    pr = ref.Problem(64, 32, 1, [300], [11], seed=9)
    q = (0.4 * pr.randn(11, 8, 64)).bfloat16()
    for heads in (1, 8):
        x = q[:, :heads].contiguous()
        want, mag = ref.attention(x, pr.values(0), pr.values(1), pr.block_table, pr.seq_len, pr.q_start, 32, scale, 0)
        got = sgr.sgr_kv_attention(pr.cache(sgr), pr.batch(sgr), x.cuda(), scale=scale, flags=flags)
        ref.check_attention(got, want, mag)


@pytest.mark.parametrize("heads,flags", [(4, FEW), (80, FEW), (4, MANY)])
def test_page_scales_far_apart(heads, flags):
    """Scales of neighbouring pages that differ by up to 2^40."""
    pr = ref.Problem(128, 16, 1, [100], [1], seed=8)
    for i, f in ((0, (0, -3, 1, -40, 2, 0, 1)), (1, (0, 20, -20, 3, -40, 10, 0))):
        for block, e in enumerate(f):
            pr.scale[i][int(pr.block_table[0, block])] *= 2.0 ** e
    q = (0.3 * pr.randn(1, heads, 128)).bfloat16()
    want, mag = ref.attention(q, pr.values(0), pr.values(1), pr.block_table, pr.seq_len, None, 16, 128 ** -0.5, 0)
    got = sgr.sgr_kv_attention(pr.cache(sgr), pr.batch(sgr, False), q.cuda(), flags=flags)
    ref.check_attention(got, want, mag)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("heads,flags", [(1, FEW), (3, FEW), (5, FEW), (1, MANY), (30, MANY)])
def test_nan_reaches_only_rows_that_see_it(dim, heads, flags):
    """A NaN key or value at a position that the later rows see and the
    earlier ones do not; a NaN before every window."""
    for which in (0, 1):
        for window in (0, 20):
            pr = ref.Problem(dim, 32, 1, [150], [6], seed=4 + which)
            at = [147] + ([100, 128] if window else [])
            for t in at:
                pr.codes[which][int(pr.block_table[0, t // 32]), 0, t % 32, 5] = ref.NAN_CODE
            q = pr.randn(6, heads, dim).bfloat16()
            want, mag = ref.attention(q, pr.values(0), pr.values(1), pr.block_table, pr.seq_len, pr.q_start, 32,
                                      dim ** -0.5, window)
            got = sgr.sgr_kv_attention(pr.cache(sgr), pr.batch(sgr), q.cuda(), window=window, flags=flags).cpu()
            assert torch.equal(got.isnan(), want.isnan())
            ref.check_attention(got, want, mag)


def test_large_offsets():
    """Pages more than 2^32 bytes apart, and tables with a long row stride."""
    pages, page, dim = 3, 16, 64
    stride = (1 << 31) + 4096
    store = torch.empty(pages * stride + (1 << 20), dtype=torch.uint8, device="cuda")
    kv = [torch.as_strided(store, (pages, 1, page, dim), (stride, page * dim, dim, 1), off) for off in (0, 1 << 19)]
    scales = torch.ones(2, pages, 1, device="cuda")
    cache = sgr.KvCache(kv[0], kv[1], scales[0], scales[1])
    wide = torch.full((2, 1000), -1, dtype=torch.int32, device="cuda")
    wide[0, :2] = torch.tensor([2, 0], dtype=torch.int32)
    wide[1, 0] = 1
    lens = torch.tensor([20, 9], dtype=torch.int32, device="cuda")
    batch = sgr.KvBatch(wide[:, :5], lens, torch.tensor([0, 20, 29], dtype=torch.int32, device="cuda"), tokens=29, max_new=20)
    g = torch.Generator().manual_seed(1)
    x = torch.randn(3, 29, 1, dim, generator=g).bfloat16()
    sgr.sgr_kv_append(cache, batch, x[0].cuda(), x[1].cuda(), sgr.RopeNorm())
    got = sgr.sgr_kv_attention(cache, batch, x[2].cuda())
    k, v = (c.float().double().cpu() * s.double().cpu()[:, :, None, None]
            for c, s in zip((t.view(torch.float8_e4m3fn) for t in kv), scales))
    want, mag = ref.attention(x[2], k, v, wide.cpu(), lens.cpu(), batch.q_start.cpu(), page, dim ** -0.5, 0)
    ref.check_attention(got, want, mag)


@pytest.mark.parametrize("flags", [FEW, MANY])
def test_long_context_split_and_repeatable(flags):
    """One long sequence over the whole GPU: against the definition, and the
    same bits every time."""
    pr = ref.Problem(128, 128, 2, [20001, 300], [1, 1], seed=12)
    q = (2 * pr.randn(2, 8, 128)).bfloat16()
    want, mag = ref.attention(q, pr.values(0), pr.values(1), pr.block_table, pr.seq_len, None, 128, 128 ** -0.5, 0)
    cache, batch = pr.cache(sgr), pr.batch(sgr, False)
    work = sgr.kv_attention_workspace(cache, batch, 8, flags)
    work.fill_(255)  # its contents do not matter
    first = sgr.sgr_kv_attention(cache, batch, q.cuda(), workspace=work, flags=flags)
    ref.check_attention(first, want, mag)
    for _ in range(5):
        assert torch.equal(sgr.sgr_kv_attention(cache, batch, q.cuda(), workspace=work, flags=flags), first)


def test_other_stream_and_graph_replay():
    """A step captured once replays with new lengths, tables and rows."""
    pr = ref.Problem(128, 64, 2, [200, 70, 129], [1, 1, 1], seed=20)
    cache, batch = pr.cache(sgr), pr.batch(sgr, False)
    qkv = pr.randn(3, 8 + 4, 128).bfloat16().cuda()
    w, table, on = norm_rope_args(128, 128, False, (True, True), 400, pr.g)
    q_out, out = torch.empty(3, 8, 128, dtype=torch.bfloat16, device="cuda"), torch.empty(3, 8, 128, dtype=torch.bfloat16, device="cuda")
    work = sgr.kv_attention_workspace(cache, batch, 8)
    side = torch.cuda.Stream()

    def step(stream=None):
        q, k, v = qkv.split((8, 2, 2), 1)
        sgr.sgr_kv_append(cache, batch, k, v, on, q=q, q_out=q_out, stream=stream)
        sgr.sgr_kv_attention(cache, batch, q_out, out=out, workspace=work, stream=stream)

    def want():
        k, v = (c.float().double().cpu() * s.double().cpu()[:, :, None, None]
                for c, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)))
        return ref.attention(q_out.cpu(), k, v, batch.block_table.cpu(), batch.seq_len.cpu(), None, 64, 128 ** -0.5, 0)

    torch.cuda.synchronize()
    step(side)
    side.synchronize()
    ref.check_attention(out, *want(), "side stream")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for lens in ([130, 1, 128], [0, 66, 190]):
        batch.seq_len.copy_(torch.tensor(lens, dtype=torch.int32))
        batch.block_table.copy_(batch.block_table.flip(0).roll(1, 0).clamp(min=0))
        table0 = torch.arange(12, dtype=torch.int32).view(3, 4)[:, :batch.max_pages] % pr.pages
        batch.block_table.copy_(table0)
        cache.k.view(torch.uint8).fill_(0x38), cache.v.view(torch.uint8).fill_(0x30)
        cache.k_scale.fill_(1.0), cache.v_scale.fill_(1.0)
        qkv.copy_(torch.randn(qkv.shape, generator=pr.g))
        graph.replay()
        torch.cuda.synchronize()
        ref.check_attention(out, *want(), f"replay {lens}")


def test_decode_block_with_projection():
    """Append, attention and the output projection with its residual, as a
    layer runs them."""
    pr = ref.Problem(128, 64, 4, [100, 300], [1, 1], seed=30)
    heads, hidden = 28, 7168
    cache, batch = pr.cache(sgr), pr.batch(sgr, False)
    qkv = pr.randn(2, heads + 8, 128).bfloat16().cuda()
    w_out = (pr.randn(hidden, heads * 128) / 60).bfloat16().cuda()
    residual = pr.randn(2, hidden).bfloat16().cuda()
    q, k, v = qkv.split((heads, 4, 4), 1)
    q = sgr.sgr_kv_append(cache, batch, k, v, sgr.RopeNorm(), q=q)
    o = sgr.sgr_kv_attention(cache, batch, q)
    y = sgr.skinny_gemm_residual(o.flatten(1), w_out, residual)
    kk, vv = (c.float().double().cpu() * s.double().cpu()[:, :, None, None]
              for c, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)))
    want, _ = ref.attention(q.cpu(), kk, vv, pr.block_table, pr.seq_len, None, 64, 128 ** -0.5, 0)
    want = want.flatten(1) @ w_out.cpu().double().T + residual.cpu().double()
    err = (y.cpu().double() - want).abs()
    assert (err <= 1e-2 * want.abs() + 2e-2).all()


def test_library_takes_the_kernel_for_many_rows():
    """A chunk large enough for the library's own choice: the bits of the
    forced one."""
    pr = ref.Problem(64, 64, 4, [1500, 700], [150, 90], seed=40)
    q = pr.randn(pr.tokens, 32, 64).bfloat16()
    cache, batch, x = pr.cache(sgr), pr.batch(sgr), q.cuda()
    assert torch.equal(sgr.sgr_kv_attention(cache, batch, x), sgr.sgr_kv_attention(cache, batch, x, flags=MANY))
    assert not torch.equal(sgr.sgr_kv_attention(cache, batch, x, flags=FEW), sgr.sgr_kv_attention(cache, batch, x, flags=MANY))
    want, mag = ref.attention(q, pr.values(0), pr.values(1), pr.block_table, pr.seq_len, pr.q_start, 64, 0.125, 0)
    ref.check_attention(sgr.sgr_kv_attention(cache, batch, x), want, mag)


def test_workspace_refusals():
    pr = ref.Problem(128, 64, 2, [3000], [1])
    cache, batch = pr.cache(sgr), pr.batch(sgr, False)
    q = torch.zeros(1, 8, 128, dtype=torch.bfloat16, device="cuda")
    work = sgr.kv_attention_workspace(cache, batch, 8)
    for kw, status in ((dict(workspace=work[:-1]), sgr.SGR_ERR_UNSUPPORTED), (dict(workspace=work[8:]), sgr.SGR_ERR_ALIGN),
                       (dict(flags=FEW | MANY, workspace=work), sgr.SGR_ERR_UNSUPPORTED)):
        with pytest.raises(sgr.SgrError) as e:
            sgr.sgr_kv_attention(cache, batch, q, **kw)
        assert e.value.status == status
    with pytest.raises(ValueError):
        sgr.sgr_kv_attention(cache, batch, q, workspace=work.cpu())
    with pytest.raises(ValueError):
        sgr.sgr_kv_attention(cache, batch, q[:, :, :64])


def test_empty_calls():
    cache = sgr.KvCache.empty(2, 1, 16, 64)
    none = torch.empty(0, 3, dtype=torch.int32, device="cuda"), torch.empty(0, dtype=torch.int32, device="cuda")
    batch = sgr.KvBatch(*none)
    x = torch.empty(0, 1, 64, dtype=torch.bfloat16, device="cuda")
    assert sgr.sgr_kv_attention(cache, batch, x).shape == (0, 1, 64)
    assert sgr.sgr_kv_append(cache, batch, x, x, sgr.RopeNorm(), q=x).shape == (0, 1, 64)
    pos = torch.empty(0, dtype=torch.int32, device="cuda")
    assert sgr.sgr_qk_norm_rope(x, x, pos, sgr.RopeNorm())[0].shape == (0, 1, 64)


@pytest.mark.parametrize("flags", [FEW, MANY])
def test_rows_of_no_sequence_are_left(flags):
    pr = ref.Problem(64, 16, 2, [40, 21], [3, 1])
    cache = pr.cache(sgr)
    batch = sgr.KvBatch(pr.block_table.cuda(), pr.seq_len.cuda(), pr.q_start.cuda(), tokens=pr.tokens + 2, max_new=3)
    x = pr.randn(3, pr.tokens + 2, 2, 64).bfloat16().cuda()
    q_out, out = torch.full_like(x[0], 7.0), torch.full_like(x[0], 7.0)
    sgr.sgr_kv_append(cache, batch, x[1], x[2], sgr.RopeNorm(), q=x[0], q_out=q_out)
    sgr.sgr_kv_attention(cache, batch, x[0], out=out, flags=flags)
    for t in (q_out, out):
        assert (t[pr.tokens:] == 7).all() and not (t[:pr.tokens] == 7).all(-1).any()


@pytest.mark.parametrize("flags", [FEW, MANY])
def test_join_with_pieces_that_see_nothing(flags):
    """Rows whose few positions lie in one piece of a split cache, with scores
    far below zero: the other pieces have no part in the maximum."""
    pr = ref.Problem(128, 128, 2, [1035], [26], seed=3)
    q = (8 * pr.randn(26, 16, 128)).bfloat16()
    want, mag = ref.attention(q, pr.values(0), pr.values(1), pr.block_table, pr.seq_len, pr.q_start, 128, 4.0, 1)
    got = sgr.sgr_kv_attention(pr.cache(sgr), pr.batch(sgr), q.cuda(), scale=4.0, window=1, flags=flags)
    ref.check_attention(got, want, mag)
