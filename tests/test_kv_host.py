"""Host side of the attention operators (no GPU): structure layouts, argument
checks on addresses that are never dereferenced, and the binding's refusals."""
import ctypes
import glob
import os
import re

import pytest
import torch

import skinny_bf16_gemm_residual_gb300 as sgr
from skinny_bf16_gemm_residual_gb300 import attention, binding

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BASE = 1 << 40
GIB = 1 << 30


def test_structs_match_header():
    text = "".join(open(h).read() for h in glob.glob(os.path.join(ROOT, "include", "*.h")))
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    for name, size in (("sgr_heads", 32), ("sgr_kv_cache", 80), ("sgr_kv_batch", 48), ("sgr_norm_rope", 40)):
        body = re.search(r"typedef struct\s*\{([^{}]*)\}\s*" + name + r"\s*;", text).group(1)
        fields = [m.group(1) for m in re.finditer(r"(\w+)\s*(?:\[\s*\d+\s*\])?\s*;", body)]
        assert fields == [f[0] for f in getattr(binding, name)._fields_]
        assert ctypes.sizeof(getattr(binding, name)) == size


def heads(at=0, ts=28 * 128, hs=128, n=28, reserved=0):
    return dict(data=BASE + at * GIB if at is not None else None, token_stride=ts, head_stride=hs, heads=n, reserved=reserved)


def cache(**kw):
    d = dict(k=BASE + 100 * GIB, v=BASE + 101 * GIB, k_scale=BASE + 102 * GIB, v_scale=BASE + 103 * GIB,
             page_stride=4 * 64 * 128, head_stride=64 * 128, token_stride=128, scale_stride=4, num_pages=1000,
             page_size=64, heads=4, head_dim=128)
    d.update(kw)
    return binding.sgr_kv_cache(**d)


def batch(**kw):
    d = dict(block_table=BASE + 110 * GIB, seq_len=BASE + 111 * GIB, q_start=None, table_stride=32, batch=16, max_pages=32,
             tokens=16, max_new=1)
    d.update(kw)
    return binding.sgr_kv_batch(**d)


def nr(**kw):
    d = dict(q_weight=None, k_weight=None, table=BASE + 120 * GIB, eps=1e-6, table_rows=100, rot_dim=128, interleaved=0)
    d.update(kw)
    return binding.sgr_norm_rope(**d)


def H(d):
    return None if d is None else ctypes.byref(binding.sgr_heads(**d))


def rope(q=heads(), k=heads(1, 512, 128, 4), qo=heads(2), ko=heads(3, 512, 128, 4), pos=BASE + 120 * GIB, tokens=5, dim=128, n=nr()):
    return sgr.load().sgr_validate_qk_norm_rope(H(q), H(k), H(qo), H(ko), pos, tokens, dim, ctypes.byref(n) if n else None)


def append(c=cache(), b=batch(), q=heads(), k=heads(1, 512, 128, 4), v=heads(2, 512, 128, 4), qo=heads(3), n=nr()):
    return sgr.load().sgr_validate_kv_append(ctypes.byref(c), ctypes.byref(b), H(q), H(k), H(v), H(qo), ctypes.byref(n))


def attend(c=cache(), b=batch(), q=heads(), out=heads(1), scale=0.1, window=0):
    return sgr.load().sgr_validate_kv_attention(ctypes.byref(c), ctypes.byref(b), H(q), H(out), scale, window)


@pytest.mark.parametrize("kw,status", [
    ({}, sgr.SGR_OK),
    (dict(k=None, ko=None), sgr.SGR_OK),
    (dict(qo=heads(), ko=heads(1, 512, 128, 4)), sgr.SGR_OK),                      # in place
    (dict(tokens=0, pos=None), sgr.SGR_OK),
    (dict(qo=heads(2, 128, 5 * 128)), sgr.SGR_OK),                                 # [heads, tokens, dim]
    (dict(ko=None), sgr.SGR_ERR_NULL),
    (dict(pos=None), sgr.SGR_ERR_NULL),
    (dict(q=None), sgr.SGR_ERR_NULL),
    (dict(n=None), sgr.SGR_ERR_NULL),
    (dict(q=heads(None)), sgr.SGR_ERR_NULL),
    (dict(tokens=-1), sgr.SGR_ERR_SHAPE),
    (dict(qo=heads(2, n=27)), sgr.SGR_ERR_SHAPE),
    (dict(qo=heads(2, ts=27 * 128)), sgr.SGR_ERR_SHAPE),                           # rows overlap
    (dict(n=nr(rot_dim=144)), sgr.SGR_ERR_SHAPE),
    (dict(n=nr(rot_dim=24)), sgr.SGR_ERR_SHAPE),
    (dict(n=nr(q_weight=BASE, eps=float("nan"))), sgr.SGR_ERR_SHAPE),
    (dict(dim=96), sgr.SGR_ERR_UNSUPPORTED),
    (dict(q=heads(reserved=1)), sgr.SGR_ERR_UNSUPPORTED),
    (dict(q=heads(ts=28 * 128 + 4)), sgr.SGR_ERR_ALIGN),
    (dict(q=dict(heads(), data=BASE + 8)), sgr.SGR_ERR_ALIGN),
    (dict(n=nr(k_weight=BASE + 2)), sgr.SGR_ERR_ALIGN),
    (dict(qo=dict(heads(), data=BASE + 16)), sgr.SGR_ERR_ALIAS),
    (dict(qo=heads(1)), sgr.SGR_ERR_ALIAS),                                        # over k
    (dict(ko=heads(2, 512, 128, 4)), sgr.SGR_ERR_ALIAS),                           # the two outputs
])
def test_validate_qk_norm_rope(kw, status):
    assert rope(**kw) == status


PACKED = 36 * 128


def part(first, n, at=0):
    return dict(heads(at, PACKED, 128, n), data=BASE + at * GIB + first * 256)


@pytest.mark.parametrize("kw,status", [
    ({}, sgr.SGR_OK),
    (dict(q=None, qo=None), sgr.SGR_OK),
    (dict(q=part(0, 28), k=part(28, 4), v=part(32, 4), qo=part(0, 28)), sgr.SGR_OK),  # in place in a packed row
    (dict(b=batch(tokens=0)), sgr.SGR_OK),
    (dict(c=cache(head_stride=128, token_stride=512)), sgr.SGR_OK),                   # [pages, page, heads, dim]
    (dict(c=cache(page_stride=2 * 4 * 64 * 128, v=BASE + 100 * GIB + 4 * 64 * 128)), sgr.SGR_OK),  # k and v in turn
    (dict(q=part(0, 28), k=part(28, 4), v=part(32, 4), qo=part(4, 28)), sgr.SGR_ERR_ALIAS),
    (dict(qo=heads(1)), sgr.SGR_ERR_ALIAS),
    (dict(qo=heads(100)), sgr.SGR_ERR_ALIAS),
    (dict(k=heads(103, 512, 128, 4)), sgr.SGR_ERR_ALIAS),
    (dict(qo=None), sgr.SGR_ERR_NULL),
    (dict(k=None), sgr.SGR_ERR_NULL),
    (dict(c=cache(k_scale=None)), sgr.SGR_ERR_NULL),
    (dict(b=batch(seq_len=None)), sgr.SGR_ERR_NULL),
    (dict(k=heads(1, 512, 128, 5)), sgr.SGR_ERR_SHAPE),
    (dict(c=cache(token_stride=112)), sgr.SGR_ERR_SHAPE),
    (dict(c=cache(page_stride=4 * 64 * 128 - 16)), sgr.SGR_ERR_SHAPE),
    (dict(c=cache(scale_stride=3)), sgr.SGR_ERR_SHAPE),
    (dict(b=batch(tokens=17)), sgr.SGR_ERR_SHAPE),
    (dict(b=batch(batch=-1)), sgr.SGR_ERR_SHAPE),
    (dict(b=batch(table_stride=31)), sgr.SGR_ERR_SHAPE),
    (dict(c=cache(token_stride=136)), sgr.SGR_ERR_ALIGN),
    (dict(c=cache(v=BASE + 101 * GIB + 8)), sgr.SGR_ERR_ALIGN),
    (dict(b=batch(q_start=BASE + 1)), sgr.SGR_ERR_ALIGN),
    (dict(c=cache(page_size=48)), sgr.SGR_ERR_UNSUPPORTED),
    (dict(c=cache(head_dim=96)), sgr.SGR_ERR_UNSUPPORTED),
    (dict(c=cache(page_stride=1 << 37)), sgr.SGR_ERR_UNSUPPORTED),
    (dict(b=batch(tokens=(1 << 20) + 1, batch=(1 << 20) + 1)), sgr.SGR_ERR_UNSUPPORTED),
])
def test_validate_kv_append(kw, status):
    assert append(**kw) == status


@pytest.mark.parametrize("kw,status", [
    ({}, sgr.SGR_OK),
    (dict(window=7), sgr.SGR_OK),
    (dict(c=cache(num_pages=0, k=None)), sgr.SGR_OK),
    (dict(window=-1), sgr.SGR_ERR_SHAPE),
    (dict(scale=float("inf")), sgr.SGR_ERR_SHAPE),
    (dict(q=heads(n=27, ts=27 * 128), out=heads(1, n=27, ts=27 * 128)), sgr.SGR_ERR_SHAPE),
    (dict(out=heads(1, n=24)), sgr.SGR_ERR_SHAPE),
    (dict(out=None), sgr.SGR_ERR_NULL),
    (dict(b=batch(max_new=0)), sgr.SGR_ERR_SHAPE),
    (dict(out=heads(0)), sgr.SGR_ERR_ALIAS),
    (dict(out=heads(101)), sgr.SGR_ERR_ALIAS),
])
def test_validate_kv_attention(kw, status):
    assert attend(**kw) == status


def test_binding_refuses_cpu_tensors_and_wrong_types():
    x = torch.zeros(2, 4, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        attention._heads(x, "q", (2, 4, 128), 0)
    with pytest.raises(TypeError):
        attention._heads(x.float(), "q", (2, 4, 128), 0)
    with pytest.raises(ValueError):
        sgr.KvCache(torch.zeros(1, 1, 16, 64, dtype=torch.uint8), torch.zeros(1, 1, 16, 64, dtype=torch.uint8), x, x)
    with pytest.raises(TypeError):
        sgr.KvCache(x[None], x[None], x, x)
    with pytest.raises(ValueError):
        sgr.KvBatch(torch.zeros(1, 1, dtype=torch.int32), torch.zeros(1, dtype=torch.int32))
    with pytest.raises(ValueError):
        sgr.RopeNorm(torch.zeros(4, 64))
