"""Attention over the paged cache where the range of its intermediate values
ends: factors of scores that underflow, rows that see nothing, weights at the
top of a code's range and far below the largest, errors of all outputs
together."""
import math

import pytest
import torch

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


def check(got, want, mag, grid=0.0, what=""):
    """BF16 rounding (half a step is at most 2^-8 of the value) and, on the sum
    p |v|, 2^-11 for the weights and 2^-11 for the scores; `grid`: what the
    smallest step of a weight adds up to."""
    got = got.double().cpu()
    bad = ~((got - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -10 * mag + grid)
    bad &= ~(got.isnan() & want.isnan())
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} off, first {tuple(bad.nonzero()[0].tolist())}: "
                           f"got {got[bad][0]} want {want[bad][0]}")


def values(cache):
    return [c.float().double().cpu() * s.double().cpu()[:, :, None, None]
            for c, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale))]


# ------------------------------------------------- factors of the scores near zero
@pytest.mark.parametrize("flags", [FEW, MANY, 0])
@pytest.mark.parametrize("window", [0, 37])
@pytest.mark.parametrize("dim,page,heads,hk", [(128, 64, 8, 2), (64, 16, 3, 1)])
def test_zero_queries_over_zero_keys(dim, page, heads, hk, window, flags):
    """A prompt of zeros: the append gives its pages the least scale, every
    position that a row sees has the same weight, and what it does not see
    none."""
    g = torch.Generator().manual_seed(heads)
    lens, new = [200, 131, 3], [130, 131, 3]
    pages = [-(-n // page) for n in lens]
    table = torch.full((3, max(pages)), -1, dtype=torch.int32)
    for b, n in enumerate(pages):
        table[b, :n] = torch.arange(sum(pages[:b]), sum(pages[:b]) + n)
    cache = sgr.KvCache.empty(sum(pages), hk, page, dim)
    for rows in ([n - m for n, m in zip(lens, new)], new):
        if rows is not new:  # the earlier positions of the first sequence
            start = torch.tensor([0, rows[0], rows[0], rows[0]], dtype=torch.int32)
            length = torch.tensor([rows[0], 0, 0], dtype=torch.int32)
        else:
            start = torch.tensor([0] + [sum(new[:i + 1]) for i in range(3)], dtype=torch.int32)
            length = torch.tensor(lens, dtype=torch.int32)
        batch = sgr.KvBatch(table.cuda(), length.cuda(), start.cuda(), tokens=int(start[-1]), max_new=max(rows))
        zero = torch.zeros(batch.tokens, heads + hk, dim, dtype=torch.bfloat16, device="cuda")
        v = torch.randn(batch.tokens, hk, dim, generator=g).bfloat16().cuda()
        q = sgr.sgr_kv_append(cache, batch, zero[:, heads:], v, sgr.RopeNorm(), q=zero[:, :heads])
    assert (cache.k_scale == 2.0 ** -64).all()
    want, mag = ref.attention(q.cpu(), *values(cache), table, lens, start, page, dim ** -0.5, window)
    check(sgr.sgr_kv_attention(cache, batch, q, window=window, flags=flags), want, mag)


@pytest.mark.parametrize("flags", [FEW, MANY])
@pytest.mark.parametrize("factor,scale", [(1.0, 0.0), (0.0, 1.0), (2.0 ** -100, -1.0)])
def test_small_factors_over_small_scales(factor, scale, flags):
    """Scores of nothing: a scale of zero, queries of (almost) zero, over keys
    whose pages have the least scale, partly masked."""
    pr = ref.Problem(128, 32, 2, [300, 40], [70, 9], seed=5)
    pr.scale[0] = torch.where(pr.scale[0].isnan(), pr.scale[0], 2.0 ** -64)
    q = (pr.randn(pr.tokens, 6, 128) * factor).bfloat16()
    for window in (0, 50):
        want, mag = ref.attention(q, pr.values(0), pr.values(1), pr.block_table, pr.seq_len, pr.q_start, 32, scale, window)
        got = sgr.sgr_kv_attention(pr.cache(sgr), pr.batch(sgr), q.cuda(), scale=scale, window=window, flags=flags)
        check(got, want, mag)


# --------------------------------------------------------------- rows that see nothing
@pytest.mark.parametrize("flags", [FEW, MANY])
@pytest.mark.parametrize("window", [0, 20])
@pytest.mark.parametrize("bad", [math.nan, math.inf, 3e38])
def test_padding_rows_get_zeros_whatever_their_query(bad, window, flags):
    """Rows before a sequence's first position, next to rows of the same tile
    that see something."""
    pr = ref.Problem(64, 32, 1, [200, 6], [220, 9], seed=7)
    q = pr.randn(pr.tokens, 3, 64).bfloat16()
    for first, n in ((0, 20), (220, 3)):
        q[first:first + n, :, 5] = bad
    clean = torch.where(q.isfinite() & (q.abs() < 1e30), q, 0.0)
    want, mag = ref.attention(clean, pr.values(0), pr.values(1), pr.block_table, pr.seq_len, pr.q_start, 32, 0.125, window)
    got = sgr.sgr_kv_attention(pr.cache(sgr), pr.batch(sgr), q.cuda(), window=window, flags=flags)
    assert (want[:20] == 0).all() and (want[220:223] == 0).all()
    assert (got[:20] == 0).all() and (got[220:223] == 0).all()
    check(got, want, mag)


# ---------------------------------------------------------------- range of the weights
@pytest.mark.parametrize("flags", [FEW, MANY])
def test_later_score_above_the_largest_so_far(flags):
    """A position of the second tile that takes most of the weight, 1.5 to 2.8
    binades above the one that set the reference in the first."""
    bits = [1.5 + 0.02 * i for i in range(64)]
    n, dim = 129, 64
    k, v = torch.zeros(n, 1, dim), torch.zeros(n, 1, dim)
    k[:, 0, 2] = -224.0  # no weight
    k[0, 0, :3] = torch.tensor([1.0, 0.0, 0.0])
    k[n - 1, 0, :3] = torch.tensor([0.0, 1.0, 0.0])
    v[n - 1] = 1.0 + torch.arange(dim) / 64.0
    v[1] = v[n - 1]  # (both pages with one scale)
    cache = sgr.KvCache.empty(2, 1, 128, dim)
    table = torch.arange(2, dtype=torch.int32).view(1, 2)
    whole = sgr.KvBatch(table.cuda(), torch.tensor([n], dtype=torch.int32).cuda(),
                        torch.tensor([0, n], dtype=torch.int32).cuda(), tokens=n, max_new=n)
    sgr.sgr_kv_append(cache, whole, k.bfloat16().cuda(), v.bfloat16().cuda(), sgr.RopeNorm())
    q = torch.zeros(1, len(bits), dim)
    q[0, :, 0] = 0.01 * math.log(2)  # just above a whole number of binades
    q[0, :, 1] = torch.tensor(bits) * math.log(2)
    q[0, :, 2] = 1.0
    q = q.bfloat16()
    for heads in (1, 8, 13, 24, 64):  # row tiles of every size
        for first in range(0, len(bits), heads):
            x = q[:, first:first + heads].contiguous()
            want, mag = ref.attention(x, *values(cache), table, [n], None, 128, 1.0, 0)
            got = sgr.sgr_kv_attention(cache, sgr.KvBatch(table.cuda(), whole.seq_len), x.cuda(), scale=1.0, flags=flags)
            check(got, want, mag, what=f"heads {first}..")


@pytest.mark.parametrize("flags", [FEW, MANY])
@pytest.mark.parametrize("heads", [1, 20])
def test_long_flat_tail_far_below_one_position(heads, flags):
    """One position of no value 14 nats above 131071 others that hold an
    eighth of the weight together, a whole sequence to each CTA: the others
    still add up."""
    n, dim, page = 131072, 64, 128
    g = torch.Generator().manual_seed(1)
    pages = n // page
    k = torch.zeros(pages, 1, page, dim)
    k[..., 0] = 0.375
    k[0, 0, 0, :2] = torch.tensor([14.0, 0.25])
    v = (1 + 0.25 * torch.randn(pages, 1, page, dim, generator=g)).to(torch.float8_e4m3fn)
    v[0, 0, 0] = 0.0
    scales = torch.ones(2, pages, 1)
    cache = sgr.KvCache(k.to(torch.float8_e4m3fn).cuda(), v.cuda(), scales[0].cuda(), scales[1].cuda())
    table = torch.arange(pages, dtype=torch.int32).view(1, pages)
    batch = 2 * torch.cuda.get_device_properties(0).multi_processor_count
    q = torch.zeros(batch, heads, dim)
    q[..., :2] = 1.0
    q = q.bfloat16()
    want, mag = ref.attention(q[:1, :1], k.double(), v.double(), table, [n], None, page, 1.0, 0)
    assert 0.07 < float(want.mean()) < 0.15
    on = sgr.KvBatch(table.expand(batch, -1).contiguous().cuda(), torch.full((batch,), n, dtype=torch.int32).cuda())
    got = sgr.sgr_kv_attention(cache, on, q.cuda(), scale=1.0, flags=flags)
    # Weights below 2^-17 of the largest are multiples of 2^-25 of it: half of that each
    check(got, want.expand(batch, heads, -1), mag.expand(batch, heads, -1), grid=n * 2.0 ** -26)


# -------------------------------------------------------------- all outputs together
@pytest.mark.parametrize("dim,page,heads,hk,lens,new,size", [
    (128, 64, 28, 4, [3000, 1201, 77], [1, 1, 1], 1.0),
    (128, 64, 28, 4, [3000, 1201, 77], [1, 1, 1], 0.0),
    (64, 32, 32, 8, [2500, 640], [5, 3], 2.0),
    (128, 32, 14, 2, [900, 1500], [100, 70], 1.0),
])
@pytest.mark.parametrize("flags", [FEW, MANY])
def test_root_mean_square_error(dim, page, heads, hk, lens, new, size, flags):
    """Of all outputs of a case: that of rounding them to BF16, and 2^-11 each
    of the outputs' own size for the weights and for the scores."""
    pr = ref.Problem(dim, page, hk, lens, new, seed=dim + heads)
    q = (size * pr.randn(pr.tokens, heads, dim)).bfloat16()
    want, _ = ref.attention(q, pr.values(0), pr.values(1), pr.block_table, pr.seq_len, pr.q_start, page, dim ** -0.5, 0)
    got = sgr.sgr_kv_attention(pr.cache(sgr), pr.batch(sgr), q.cuda(), flags=flags).double().cpu()

    def rms(x):
        return float(x.square().mean().sqrt())

    bound = math.sqrt(rms(want.bfloat16().double() - want) ** 2 + 2 * (2.0 ** -11 * rms(want)) ** 2)
    assert rms(got - want) <= 1.02 * bound


@pytest.mark.parametrize("flags", [FEW, MANY])
def test_one_position_takes_all_the_weight(flags):
    """Scores of thousands: the value of the largest, wherever it is ahead by
    more than 12 and twice a score's error (2^-16 of |q| |k| scale)."""
    pr = ref.Problem(128, 64, 2, [3000, 500, 130], [1, 1, 1], seed=3)
    q = (1e4 * pr.randn(3, 8, 128)).bfloat16()
    want, mag = ref.attention(q, pr.values(0), pr.values(1), pr.block_table, pr.seq_len, None, 64, 128 ** -0.5, 0)
    got = sgr.sgr_kv_attention(pr.cache(sgr), pr.batch(sgr, False), q.cuda(), flags=flags).double().cpu()
    checked = 0
    for b, n in enumerate(pr.lens):
        t = torch.arange(n)
        k = pr.values(0)[pr.block_table[b].long()[t // 64], :, t % 64]  # [n, heads, dim]
        score = torch.einsum("kgd,tkd->kgt", q[b].double().view(2, 4, 128), k).reshape(8, n) * 128 ** -0.5
        top = score.topk(2, -1).values
        error = 2.0 ** -16 * q[b].double().norm(dim=-1) * k.norm(dim=-1).max() * 128 ** -0.5
        ahead = top[:, 0] - top[:, 1] > 12 + 2 * error
        check(got[b][ahead], want[b][ahead], mag[b][ahead])
        checked += int(ahead.sum())
    assert checked >= 12
