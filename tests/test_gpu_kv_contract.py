"""What the header says of the attention operators' arguments where no other test
looks, on the GPU against the header's own formulas."""
import pytest
import torch

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
