"""The example of the attention block: prompts in chunks, then steps from one graph."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

EXAMPLE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "decode_block.py")


@pytest.mark.parametrize("heads, kv_heads, dim, page", [(4, 2, 64, 16), (7, 1, 128, 64)])
def test_decode_block_example(heads, kv_heads, dim, page):
    spec = importlib.util.spec_from_file_location("decode_block", EXAMPLE)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    error, largest, _ = m.run(batch=3, prompt=90, chunk=33, steps=5, heads=heads, kv_heads=kv_heads, dim=dim, page=page)
    # E4M3 keys and values: 2.6% rms each of a score's and a value's unit
    # variance, so 3.7% of the attention's rms, which is at most 0.36 here (21
    # or more positions whose weights vary by e: 8 in effect).  Six standard
    # deviations of that, 0.08, and half a BF16 step of an output below 8.
    assert largest < 8
    assert error <= 0.08 + 2.0 ** -6
