"""Arrays that the attention operators read, within the memory that they write:
refused before anything is enqueued (no GPU; addresses are never dereferenced)."""
import ctypes

import pytest

import skinny_bf16_gemm_residual_gb300 as sgr
from test_kv_host import BASE, GIB, H, batch, cache, heads, nr

TOKENS = 16
Q_OUT = BASE + 3 * GIB
Q_BYTES = TOKENS * 28 * 128 * 2
CODES = 1000 * 4 * 64 * 128


@pytest.mark.parametrize("pos,status", [
    (BASE + 170 * GIB, sgr.SGR_OK),
    (Q_OUT - 4 * TOKENS, sgr.SGR_OK),                                  # right before the rotated queries
    (Q_OUT + Q_BYTES, sgr.SGR_OK),                                     # right behind them
    (BASE, sgr.SGR_OK),                                                # the queries, which are not written
    (Q_OUT, sgr.SGR_ERR_ALIAS),
    (Q_OUT - 4 * TOKENS + 4, sgr.SGR_ERR_ALIAS),                       # the last position in the first query
    (Q_OUT + Q_BYTES - 4, sgr.SGR_ERR_ALIAS),
    (BASE + 100 * GIB, sgr.SGR_ERR_ALIAS),                             # the keys' codes
    (BASE + 101 * GIB + CODES - 4, sgr.SGR_ERR_ALIAS),                 # the values'
    (BASE + 102 * GIB, sgr.SGR_ERR_ALIAS),                             # the scales
    (BASE + 103 * GIB + 4 * 4 * 1000 - 4, sgr.SGR_ERR_ALIAS),
])
def test_positions_within_what_an_append_writes(pos, status):
    c, b, n = cache(), batch(), nr()
    assert sgr.load().sgr_validate_kv_append_at(ctypes.byref(c), ctypes.byref(b), H(heads()), H(heads(1, 512, 128, 4)),
                                                H(heads(2, 512, 128, 4)), H(heads(3)), ctypes.byref(n), pos) == status


def test_positions_of_an_append_without_queries():
    c, b, n = cache(), batch(), nr()
    for pos, status in ((Q_OUT, sgr.SGR_OK), (BASE + 100 * GIB, sgr.SGR_ERR_ALIAS)):
        assert sgr.load().sgr_validate_kv_append_at(ctypes.byref(c), ctypes.byref(b), None, H(heads(1, 512, 128, 4)),
                                                    H(heads(2, 512, 128, 4)), None, ctypes.byref(n), pos) == status


LSE, MASS, TREE = BASE + 130 * GIB, BASE + 140 * GIB, BASE + 150 * GIB
OUT = BASE + GIB
WORDS = 15 * 3 + 2  # of 16 rows of two words, three apart


def mask(at):
    return sgr.binding.sgr_kv_mask(tree=at, tree_stride=3, tree_words=2, window=0, sinks=0, reserved=0)


@pytest.mark.parametrize("at,status", [
    (TREE, sgr.SGR_OK),
    (OUT - 8 * WORDS, sgr.SGR_OK),
    (OUT - 8 * WORDS + 8, sgr.SGR_ERR_ALIAS),
    (OUT + Q_BYTES, sgr.SGR_OK),
    (OUT + Q_BYTES - 8, sgr.SGR_ERR_ALIAS),
    (LSE - 8 * WORDS, sgr.SGR_OK),
    (LSE - 8 * WORDS + 8, sgr.SGR_ERR_ALIAS),
    (LSE + 4 * TOKENS * 28 - 8, sgr.SGR_ERR_ALIAS),
    (LSE + 4 * TOKENS * 28, sgr.SGR_OK),
    (BASE, sgr.SGR_OK),                                                # the queries and the keys are not written
    (BASE + 100 * GIB, sgr.SGR_OK),
])
def test_trees_within_what_attention_writes(at, status):
    c, b, m = cache(), batch(), mask(at)
    assert sgr.load().sgr_validate_kv_attention_masked(ctypes.byref(c), ctypes.byref(b), H(heads()), H(heads(1)), LSE, 0.1,
                                                       ctypes.byref(m)) == status


@pytest.mark.parametrize("at,status", [
    (TREE, sgr.SGR_OK),
    (MASS - 8 * WORDS, sgr.SGR_OK),
    (MASS - 8 * WORDS + 8, sgr.SGR_ERR_ALIAS),
    (MASS + 4 * 1000 * 4 * 64 - 8, sgr.SGR_ERR_ALIAS),
    (MASS + 4 * 1000 * 4 * 64, sgr.SGR_OK),
    (LSE, sgr.SGR_OK),                                                 # not written by this call
])
def test_trees_within_masses(at, status):
    c, b, m = cache(), batch(), mask(at)
    to = sgr.binding.sgr_kv_masses(data=MASS, page_stride=4 * 64, head_stride=64)
    assert sgr.load().sgr_validate_kv_mass(ctypes.byref(c), ctypes.byref(b), H(heads()), LSE, ctypes.byref(to), 0.1,
                                           ctypes.byref(m)) == status
