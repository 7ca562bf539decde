"""Host side of masked attention, appends to given positions, accumulated weight
and eviction (no GPU): structure layouts, argument checks on addresses that are
never dereferenced, the binding's refusals, and the kernels' index arithmetic
compiled for the host."""
import ctypes
import glob
import os
import re
import shutil
import subprocess

import pytest
import torch

import skinny_bf16_gemm_residual_gb300 as sgr
from skinny_bf16_gemm_residual_gb300 import attention, binding
from test_kv_host import BASE, GIB, H, ROOT, batch, cache, heads, nr

LSE = BASE + 130 * GIB
MASS = BASE + 140 * GIB


def test_structs_match_header():
    text = "".join(open(h).read() for h in glob.glob(os.path.join(ROOT, "include", "*.h")))
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    for name, size in (("sgr_kv_mask", 32), ("sgr_kv_masses", 24), ("sgr_kv_eviction", 56)):
        body = re.search(r"typedef struct\s*\{([^{}]*)\}\s*" + name + r"\s*;", text).group(1)
        fields = [m.group(1) for m in re.finditer(r"(\w+)\s*(?:\[\s*\d+\s*\])?\s*;", body)]
        assert fields == [f[0] for f in getattr(binding, name)._fields_]
        assert ctypes.sizeof(getattr(binding, name)) == size


def mask(**kw):
    return binding.sgr_kv_mask(**dict(dict(tree=None, tree_stride=0, tree_words=0, window=0, sinks=0, reserved=0), **kw))


def tree(at=150, stride=1, words=1, **kw):
    return mask(tree=BASE + at * GIB, tree_stride=stride, tree_words=words, **kw)


def masses(**kw):
    return binding.sgr_kv_masses(**dict(dict(data=MASS, page_stride=4 * 64, head_stride=64), **kw))


def eviction(**kw):
    return binding.sgr_kv_eviction(**dict(dict(keep=BASE + 160 * GIB, table=BASE + 161 * GIB, kept=BASE + 162 * GIB,
                                               new_len=BASE + 163 * GIB, table_stride=8, max_pages=8, first=4, recent=100,
                                               reserved=0), **kw))


def ref_of(x):
    return None if x is None else ctypes.byref(x)


def attend(c=cache(), b=batch(), q=heads(), out=heads(1), lse=LSE, scale=0.1, m=mask()):
    return sgr.load().sgr_validate_kv_attention_masked(ctypes.byref(c), ctypes.byref(b), H(q), H(out), lse, scale, ref_of(m))


@pytest.mark.parametrize("kw,status", [
    ({}, sgr.SGR_OK),
    (dict(m=None, lse=None), sgr.SGR_OK),
    (dict(m=mask(window=7, sinks=4)), sgr.SGR_OK),
    (dict(m=mask(sinks=1 << 30)), sgr.SGR_OK),
    (dict(m=tree()), sgr.SGR_OK),
    (dict(m=tree(stride=5, words=3, window=9, sinks=2), b=batch(max_new=192, q_start=BASE + 112 * GIB)), sgr.SGR_OK),
    (dict(m=mask(window=-1)), sgr.SGR_ERR_SHAPE),
    (dict(m=mask(sinks=-1)), sgr.SGR_ERR_SHAPE),
    (dict(m=tree(words=0)), sgr.SGR_ERR_SHAPE),
    (dict(m=tree(words=2)), sgr.SGR_ERR_SHAPE),                                             # rows closer than their words
    (dict(m=tree(), b=batch(max_new=65, q_start=BASE + 112 * GIB)), sgr.SGR_ERR_SHAPE),     # more new tokens than bits
    (dict(m=tree(stride=1 << 37)), sgr.SGR_ERR_UNSUPPORTED),
    (dict(m=mask(reserved=1)), sgr.SGR_ERR_UNSUPPORTED),
    (dict(m=mask(tree=BASE + 150 * GIB + 4, tree_stride=1, tree_words=1)), sgr.SGR_ERR_ALIGN),
    (dict(lse=LSE + 2), sgr.SGR_ERR_ALIGN),
    (dict(lse=BASE + 100), sgr.SGR_ERR_ALIAS),                                              # within the queries
    (dict(lse=BASE + GIB - 16 * 28 * 4 + 4), sgr.SGR_ERR_ALIAS),                            # runs into the outputs
    (dict(lse=BASE + 102 * GIB), sgr.SGR_ERR_ALIAS),                                        # the key scales
    (dict(scale=float("nan")), sgr.SGR_ERR_SHAPE),
    (dict(out=None), sgr.SGR_ERR_NULL),
    (dict(b=batch(tokens=0), out=None, m=tree(words=0)), sgr.SGR_OK),                       # nothing to do
])
def test_validate_kv_attention_masked(kw, status):
    assert attend(**kw) == status


@pytest.mark.parametrize("pos,status", [(None, sgr.SGR_OK), (BASE + 170 * GIB, sgr.SGR_OK), (BASE + 170 * GIB + 2, sgr.SGR_ERR_ALIGN)])
def test_validate_kv_append_at(pos, status):
    c, b, n = cache(), batch(), nr()
    assert sgr.load().sgr_validate_kv_append_at(ctypes.byref(c), ctypes.byref(b), H(heads()), H(heads(1, 512, 128, 4)),
                                                H(heads(2, 512, 128, 4)), H(heads(3)), ctypes.byref(n), pos) == status


def weigh(c=cache(), b=batch(), q=heads(), lse=LSE, mass=masses(), scale=0.1, m=mask()):
    return sgr.load().sgr_validate_kv_mass(ctypes.byref(c), ctypes.byref(b), H(q), lse, ref_of(mass), scale, ref_of(m))


@pytest.mark.parametrize("kw,status", [
    ({}, sgr.SGR_OK),
    (dict(m=tree(window=5)), sgr.SGR_OK),
    (dict(mass=masses(page_stride=64, head_stride=64 * 1000)), sgr.SGR_OK),                 # [heads, pages, page]
    (dict(c=cache(num_pages=0, k=None), mass=masses(data=None)), sgr.SGR_OK),
    (dict(b=batch(tokens=0), lse=None, mass=None), sgr.SGR_OK),
    (dict(q=None), sgr.SGR_ERR_NULL),
    (dict(lse=None), sgr.SGR_ERR_NULL),
    (dict(mass=None), sgr.SGR_ERR_NULL),
    (dict(mass=masses(data=None)), sgr.SGR_ERR_NULL),
    (dict(scale=float("inf")), sgr.SGR_ERR_SHAPE),
    (dict(q=heads(n=27, ts=27 * 128)), sgr.SGR_ERR_SHAPE),
    (dict(mass=masses(head_stride=63)), sgr.SGR_ERR_SHAPE),                                 # positions overlap
    (dict(mass=masses(page_stride=3 * 64)), sgr.SGR_ERR_SHAPE),
    (dict(mass=masses(page_stride=-256)), sgr.SGR_ERR_SHAPE),
    (dict(mass=masses(page_stride=1 << 37)), sgr.SGR_ERR_UNSUPPORTED),
    (dict(mass=masses(data=MASS + 2)), sgr.SGR_ERR_ALIGN),
    (dict(lse=LSE + 1), sgr.SGR_ERR_ALIGN),
    (dict(mass=masses(data=BASE + 100 * GIB)), sgr.SGR_ERR_ALIAS),                          # the keys
    (dict(mass=masses(data=LSE)), sgr.SGR_ERR_ALIAS),
    (dict(mass=masses(data=BASE)), sgr.SGR_ERR_ALIAS),                                      # the queries
])
def test_validate_kv_mass(kw, status):
    assert weigh(**kw) == status


def test_mass_workspace_sizes():
    n = ctypes.c_int64(-1)

    def size(c, b, q_heads):
        rc = sgr.load().sgr_kv_mass_workspace(ctypes.byref(c), ctypes.byref(b), q_heads, ctypes.byref(n))
        return rc, n.value

    assert size(cache(), batch(), 28) == (sgr.SGR_OK, 0)
    chunk = dict(q_start=BASE + 112 * GIB, tokens=600, batch=2)
    assert size(cache(), batch(max_new=18, **chunk), 28) == (sgr.SGR_OK, 0)  # 126 rows a head
    # 19 tokens of 7 heads: at most (600 * 7 / 128 + 2) row tiles of 4 heads over 16 tiles of 128 positions
    assert size(cache(), batch(max_new=19, **chunk), 28) == (sgr.SGR_OK, (600 * 7 // 128 + 2) * 4 * 16 * 128 * 4)
    assert size(cache(), batch(), 27)[0] == sgr.SGR_ERR_SHAPE
    assert sgr.load().sgr_kv_mass_workspace(ctypes.byref(cache()), ctypes.byref(batch()), 28, None) == sgr.SGR_ERR_NULL


def evict(c=cache(), b=batch(), mass=masses(), e=eviction()):
    return sgr.load().sgr_validate_kv_evict(ctypes.byref(c), ctypes.byref(b), ref_of(mass), ref_of(e))


@pytest.mark.parametrize("kw,status", [
    ({}, sgr.SGR_OK),
    (dict(b=batch(tokens=99, max_new=0)), sgr.SGR_OK),                                      # rows do not matter
    (dict(e=eviction(max_pages=0, table=None, kept=None)), sgr.SGR_OK),
    (dict(b=batch(batch=0, tokens=0), e=eviction(keep=None)), sgr.SGR_OK),
    (dict(e=None), sgr.SGR_ERR_NULL),
    (dict(mass=None), sgr.SGR_ERR_NULL),
    (dict(e=eviction(keep=None)), sgr.SGR_ERR_NULL),
    (dict(e=eviction(new_len=None)), sgr.SGR_ERR_NULL),
    (dict(e=eviction(kept=None)), sgr.SGR_ERR_NULL),
    (dict(e=eviction(table=None)), sgr.SGR_ERR_NULL),
    (dict(b=batch(seq_len=None)), sgr.SGR_ERR_NULL),
    (dict(e=eviction(first=-1)), sgr.SGR_ERR_SHAPE),
    (dict(e=eviction(recent=-1)), sgr.SGR_ERR_SHAPE),
    (dict(e=eviction(max_pages=-1)), sgr.SGR_ERR_SHAPE),
    (dict(e=eviction(table_stride=7)), sgr.SGR_ERR_SHAPE),
    (dict(b=batch(batch=-1)), sgr.SGR_ERR_SHAPE),
    (dict(e=eviction(reserved=1)), sgr.SGR_ERR_UNSUPPORTED),
    (dict(e=eviction(max_pages=(1 << 24) + 1, table_stride=1 << 25)), sgr.SGR_ERR_UNSUPPORTED),
    (dict(e=eviction(kept=BASE + 162 * GIB + 2)), sgr.SGR_ERR_ALIGN),
    (dict(e=eviction(new_len=BASE + 111 * GIB)), sgr.SGR_ERR_ALIAS),                        # the lengths in use
    (dict(e=eviction(kept=BASE + 110 * GIB)), sgr.SGR_ERR_ALIAS),                           # the table in use
    (dict(e=eviction(kept=BASE + 163 * GIB - 4)), sgr.SGR_ERR_ALIAS),                       # runs into the new lengths
    (dict(e=eviction(kept=MASS)), sgr.SGR_ERR_ALIAS),
    (dict(e=eviction(new_len=BASE + 101 * GIB)), sgr.SGR_ERR_ALIAS),                        # the values
    (dict(e=eviction(table=BASE + 100 * GIB)), sgr.SGR_ERR_ALIAS),                          # a table within what is written
    (dict(mass=masses(data=BASE + 103 * GIB)), sgr.SGR_ERR_ALIAS),
])
def test_validate_kv_evict(kw, status):
    assert evict(**kw) == status


def test_binding_refuses_wrong_trees_and_masses():
    class Sizes:
        tokens, max_new = 6, 70

    for t in (torch.zeros(6, 2, dtype=torch.int32), torch.zeros(6, dtype=torch.int64), torch.zeros(6, 4, dtype=torch.int64)[:, ::2]):
        with pytest.raises(ValueError, match="int64"):
            attention._mask(Sizes, 0, 0, t, 0)
    with pytest.raises(ValueError, match="CUDA"):
        attention._mask(Sizes, 0, 0, torch.zeros(6, 2, dtype=torch.int64), 0)
    for shape in ((5, 2), (6, 1), (6, 0)):
        with pytest.raises(ValueError, match="at least 2"):
            attention._mask(Sizes, 0, 0, torch.zeros(shape, dtype=torch.int64), -1)
    assert len(attention._mask(Sizes, 5, 4, None, 0)) == ctypes.sizeof(binding.sgr_kv_mask)
    with pytest.raises(ValueError, match="float32"):
        attention._row_stats(torch.zeros(6, 8, dtype=torch.float64), "lse", (6, 8), -1)
    with pytest.raises(ValueError, match="float32"):
        attention._row_stats(torch.zeros(8, 6).t(), "lse", (6, 8), -1)


def test_masks_of_the_kernels_on_the_host(tmp_path):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("nvcc not available")
    exe = str(tmp_path / "kv_mask_probe")
    subprocess.run([nvcc, "-std=c++17", "--expt-relaxed-constexpr", "-gencode", "arch=compute_103a,code=sm_103a",
                    "-Xcompiler", "-fsanitize=signed-integer-overflow", "-Xcompiler", "-fno-sanitize-recover=all",
                    f"-I{os.path.join(ROOT, 'skinny_bf16_gemm_residual_gb300', 'csrc')}", f"-I{os.path.join(ROOT, 'include')}",
                    os.path.join(ROOT, "tests", "kv_mask_probe.cu"), "-o", exe, "-lubsan"], check=True)
    out = subprocess.run([exe], capture_output=True, text=True)
    assert out.returncode == 0, out.stdout + out.stderr
    assert int(out.stdout) > 100000
