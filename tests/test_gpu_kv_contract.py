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
