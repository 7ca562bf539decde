"""Sizes and numbers at the ends of what the attention operators take (no GPU)."""
import ctypes

import pytest

import skinny_bf16_gemm_residual_gb300 as sgr
from test_kv_host import BASE, GIB, batch, cache


def mass_workspace(c, b, q_heads):
    n = ctypes.c_int64(-1)
    rc = sgr.load().sgr_kv_mass_workspace(ctypes.byref(c), ctypes.byref(b), q_heads, ctypes.byref(n))
    return rc, n.value


@pytest.mark.parametrize("kw,ckw,q_heads", [
    (dict(tokens=1 << 20, max_new=1 << 20, max_pages=1 << 24, table_stride=1 << 24), {}, 4096),  # more than 2^31 units
    (dict(tokens=600, max_new=300, batch=2), {}, 1 << 30),                                       # heads; 2^64 bytes and more
    (dict(tokens=600, max_new=300, batch=2), {}, 8192),
    (dict(tokens=70000, max_new=300, batch=70000, max_pages=1, table_stride=1), {}, 4),          # more sequences than a join takes
    (dict(max_pages=1 << 24, table_stride=1 << 24), dict(page_size=128, page_stride=4 * 128 * 128, head_stride=128 * 128), 4),  # tiles of a sequence
])
def test_mass_workspace_refuses_what_the_call_refuses(kw, ckw, q_heads):
    b = dict(q_start=BASE + 112 * GIB)
    assert mass_workspace(cache(**ckw), batch(**dict(b, **kw)), q_heads) == (sgr.SGR_ERR_UNSUPPORTED, -1)


def test_mass_workspace_of_nothing():
    assert mass_workspace(cache(), batch(tokens=0, batch=0), 4) == (sgr.SGR_OK, 0)
    assert mass_workspace(cache(), batch(tokens=70000, max_new=32, batch=70000, q_start=BASE + 112 * GIB), 16) == (sgr.SGR_OK, 0)


def test_numbers_past_32_bits_are_value_errors():
    from skinny_bf16_gemm_residual_gb300 import attention

    for window, sinks in ((1 << 31, 0), (0, 1 << 31), (1 << 70, 4), (-(1 << 31) - 1, 0), (3.5, 0)):
        with pytest.raises(ValueError, match="32 bits"):
            attention._mask(None, window, sinks, None, 0)
    assert len(attention._mask(None, (1 << 31) - 1, (1 << 31) - 1, None, 0)) == 32
