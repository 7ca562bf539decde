"""Tensor-level calls of the attention operators (include/sgr_attention.h).

A program keeps a ``KvCache`` (the pages), a ``KvBatch`` (the sequences of a
step; its tensors are updated in place from step to step) and a ``RopeNorm``
(rotation table and norm weights), and calls per layer and step

    q = sgr_kv_append(cache, batch, k, v, rope, q=q)     # norm, rotation, append
    o = sgr_kv_attention(cache, batch, q)                # attention over the cache
    y = skinny_gemm_residual(o.flatten(1), w_out, residual)

Rows of heads (q, k, v and outputs) are CUDA bfloat16 tensors
[tokens, heads, head_dim] with unit inner stride and token and head strides
that are multiples of 8 elements: slices of a packed projection output fit as
they are.  Calls run on the tensors' device, on its current stream unless
``stream=`` is given.  As everywhere in this package there is no CPU fallback.
"""
from __future__ import annotations

import ctypes
import struct

from .binding import (SGR_OK, SgrError, _common_device, load, sgr_heads, sgr_kv_batch, sgr_kv_cache, sgr_norm_rope)


class _Torch:
    """Stands for torch until its first use (importing the package does not import torch)."""

    def __getattr__(self, name):
        global torch
        import torch

        return getattr(torch, name)


torch = _Torch()

# A call of a few microseconds on the GPU should not wait for its arguments:
# sgr_heads structures go as packed bytes, devices are compared by index, the
# current stream is asked for as a number, and torch is looked up in this
# module.
_pack_heads = struct.Struct("@Pqqii").pack
assert struct.calcsize("@Pqqii") == ctypes.sizeof(sgr_heads)


def _check(rc: int, what: str) -> None:
    if rc != SGR_OK:
        raise SgrError(rc, what)


def _wrong_heads(t, name: str, shape, index: int):
    if t.dtype is not torch.bfloat16:
        raise TypeError(f"{name} must be torch.bfloat16, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.get_device() != index:
        raise ValueError(f"{name}: all tensors must be on one CUDA device, got {t.device} and cuda:{index}")
    if t.dim() != 3:
        raise ValueError(f"{name} must be [tokens, heads, head_dim]")
    if tuple(t.shape) != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    raise ValueError(f"{name} must have unit inner stride")


def _heads(t, name: str, shape, index: int) -> bytes:
    """The sgr_heads of a tensor of this shape on this device."""
    if t.dtype is not torch.bfloat16 or t.get_device() != index or t.shape != shape:
        _wrong_heads(t, name, shape, index)
    ts, hs, es = t.stride()
    if es != 1:
        _wrong_heads(t, name, shape, index)
    tokens, heads, dim = shape
    # Strides of axes with one element are arbitrary in torch.
    return _pack_heads(t.data_ptr(), ts if tokens > 1 else heads * dim, hs if heads > 1 else dim, heads, 0)


def _shape3(t, name: str):
    if t.dim() != 3:
        raise ValueError(f"{name} must be [tokens, heads, head_dim]")
    return t.shape


def _int32(t, name: str, dim: int):
    if t.dtype is not torch.int32 or not t.is_cuda or t.dim() != dim or (t.shape[-1] > 1 and t.stride(-1) != 1):
        raise ValueError(f"{name} must be a {dim}-D CUDA int32 tensor with unit inner stride")
    return t


class KvCache:
    """A paged cache of E4M3 codes with one power-of-two scale for each page and head.

    k, v: [pages, heads, page_size, head_dim] CUDA float8_e4m3fn (or uint8)
    tensors with unit inner stride and the same strides; a view
    ``.transpose(1, 2)`` of [pages, page_size, heads, head_dim] fits as well.
    k_scale, v_scale: [pages, heads] float32, unit inner stride."""

    def __init__(self, k, v, k_scale, v_scale):
        for t, n in ((k, "k"), (v, "v")):
            if t.dtype not in (torch.float8_e4m3fn, torch.uint8):
                raise TypeError(f"{n} must be torch.float8_e4m3fn or torch.uint8, got {t.dtype}")
            if not t.is_cuda or t.dim() != 4 or t.stride(3) != 1:
                raise ValueError(f"{n} must be a CUDA tensor [pages, heads, page_size, head_dim] with unit inner stride")
        if k.shape != v.shape or k.stride() != v.stride():
            raise ValueError("k and v must have the same shape and strides")
        for t, n in ((k_scale, "k_scale"), (v_scale, "v_scale")):
            if t.dtype != torch.float32 or not t.is_cuda or t.shape != k.shape[:2] or (t.shape[1] > 1 and t.stride(1) != 1):
                raise ValueError(f"{n} must be a CUDA float32 tensor [pages, heads] with unit inner stride")
        if k_scale.stride(0) != v_scale.stride(0):
            raise ValueError("k_scale and v_scale must have the same strides")
        self.device = _common_device((k, v, k_scale, v_scale))
        self.index = self.device.index
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        pages, self.heads, self.page_size, self.head_dim = k.shape
        self.c = sgr_kv_cache(k.data_ptr(), v.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), k.stride(0),
                              k.stride(1), k.stride(2), k_scale.stride(0) if pages > 1 else self.heads, pages,
                              self.page_size, self.heads, self.head_dim)
        self.ref = ctypes.addressof(self.c)

    @classmethod
    def empty(cls, pages: int, heads: int, page_size: int, head_dim: int, device="cuda") -> "KvCache":
        """A cache without contents: pages count from the first append to them."""
        kv = torch.zeros(2, pages, heads, page_size, head_dim, dtype=torch.uint8, device=device)
        scale = torch.ones(2, pages, heads, dtype=torch.float32, device=device)
        kv = kv.view(torch.float8_e4m3fn)
        return cls(kv[0], kv[1], scale[0], scale[1])


class KvBatch:
    """The sequences of a step: block_table [batch, max_pages], seq_len
    [batch] (positions in the cache, this step's new tokens among them) and
    q_start [batch + 1] (first row of each sequence; None: one row each), all
    CUDA int32.  tokens: rows in all; max_new: the most rows of a sequence
    (both are read on the host, q_start is not)."""

    def __init__(self, block_table, seq_len, q_start=None, tokens: int | None = None, max_new: int = 1):
        _int32(block_table, "block_table", 2)
        _int32(seq_len, "seq_len", 1)
        batch, max_pages = block_table.shape
        if seq_len.shape[0] != batch:
            raise ValueError(f"seq_len must have {batch} elements, got {seq_len.shape[0]}")
        if q_start is not None:
            _int32(q_start, "q_start", 1)
            if q_start.shape[0] != batch + 1:
                raise ValueError(f"q_start must have {batch + 1} elements, got {q_start.shape[0]}")
        if tokens is None:
            if q_start is not None:
                raise ValueError("tokens is needed with q_start")
            tokens = batch
        self.block_table, self.seq_len, self.q_start = block_table, seq_len, q_start
        self.device = _common_device([t for t in (block_table, seq_len, q_start) if t is not None])
        self.index = self.device.index
        self.batch, self.max_pages, self.tokens, self.max_new = batch, max_pages, int(tokens), int(max_new)
        self.c = sgr_kv_batch(block_table.data_ptr(), seq_len.data_ptr(),
                              q_start.data_ptr() if q_start is not None else None,
                              block_table.stride(0) if batch > 1 else max_pages, batch, max_pages, self.tokens,
                              self.max_new)
        self.ref = ctypes.addressof(self.c)


class RopeNorm:
    """Rotation table [positions, rot_dim] float32 (rot_dim / 2 cosines, then
    the sines; None: no rotation) and the norm weights of queries and keys
    [head_dim] bfloat16 (None: no norm)."""

    def __init__(self, table=None, q_weight=None, k_weight=None, eps: float = 1e-6, interleaved: bool = False):
        if table is not None and (table.dtype != torch.float32 or not table.is_cuda or table.dim() != 2
                                  or not table.is_contiguous()):
            raise ValueError("table must be a contiguous 2-D CUDA float32 tensor")
        for w, n in ((q_weight, "q_weight"), (k_weight, "k_weight")):
            if w is not None and (w.dtype != torch.bfloat16 or not w.is_cuda or w.dim() != 1 or not w.is_contiguous()):
                raise ValueError(f"{n} must be a contiguous 1-D CUDA bfloat16 tensor")
        self.table, self.q_weight, self.k_weight = table, q_weight, k_weight
        tensors = [t for t in (table, q_weight, k_weight) if t is not None]
        self.index = _common_device(tensors).index if tensors else None
        dims = {w.shape[0] for w in (q_weight, k_weight) if w is not None}
        if len(dims) > 1:
            raise ValueError("q_weight and k_weight must have the same number of elements")
        self.head_dim = dims.pop() if dims else None
        rows, rot = table.shape if table is not None else (0, 0)
        self.c = sgr_norm_rope(*(t.data_ptr() if t is not None else None for t in (q_weight, k_weight, table)),
                               float(eps), rows, rot, int(interleaved))
        self.ref = ctypes.addressof(self.c)


def _on(index: int, other, what: str):
    if other is not None and other != index:
        raise ValueError(f"{what}: all tensors must be on one CUDA device, got cuda:{index} and cuda:{other}")


def _launch(index: int, stream, what: str, fn, *args):
    """fn(*args, stream handle) with device `index` current."""
    if stream is None:
        handle = torch._C._cuda_getCurrentRawStream(index)
    elif isinstance(stream, int):
        handle = stream
    elif stream.device.index != index:
        raise ValueError(f"stream is on {stream.device}, tensors on cuda:{index}")
    else:
        handle = stream.cuda_stream
    if torch._C._cuda_getDevice() == index:
        rc = fn(*args, handle)
    else:
        with torch.cuda.device(index):
            rc = fn(*args, handle)
    if rc != SGR_OK:
        raise SgrError(rc, what)


def _new(index: int, stream, make):
    """A tensor allocated for use on `stream`."""
    if stream is None:
        return make()
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device=index)
    with torch.cuda.stream(stream):
        return make()


def _like(t, stream):
    return _new(t.get_device(), stream, lambda: torch.empty(t.shape, dtype=t.dtype, device=t.device))


def sgr_qk_norm_rope(q, k, positions, rope: RopeNorm, q_out=None, k_out=None, flags: int = 0, stream=None):
    """Queries and keys normalised per head and rotated to positions [tokens]
    (int32; a negative one gives a row of zeros); k may be None.  The outputs
    may be the inputs.  Returns (q_out, k_out)."""
    shape = _shape3(q, "q")
    tokens, _, dim = shape
    index = q.get_device()
    hq = _heads(q, "q", shape, index)
    if (positions.dtype is not torch.int32 or positions.shape != (tokens,) or positions.get_device() != index
            or not positions.is_contiguous()):
        _int32(positions, "positions", 1)
        if positions.shape[0] != tokens:
            raise ValueError(f"positions must have {tokens} elements, got {positions.shape[0]}")
        _on(index, positions.get_device(), "sgr_qk_norm_rope")
    if rope.head_dim is not None and rope.head_dim != dim:
        raise ValueError(f"norm weights must have {dim} elements")
    if q_out is None:
        q_out = _like(q, stream)
    hqo = _heads(q_out, "q_out", shape, index)
    hk = hko = None
    if k is not None:
        shape = (tokens, _shape3(k, "k")[1], dim)
        hk = _heads(k, "k", shape, index)
        if k_out is None:
            k_out = _like(k, stream)
        hko = _heads(k_out, "k_out", shape, index)
    if rope.index != index:
        _on(index, rope.index, "sgr_qk_norm_rope")
    _launch(index, stream, "sgr_qk_norm_rope", load().sgr_qk_norm_rope, hq, hk, hqo, hko, positions.data_ptr(), tokens,
            dim, rope.ref, flags)
    return q_out, k_out


def sgr_kv_append(cache: KvCache, batch: KvBatch, k, v, rope: RopeNorm, q=None, q_out=None, flags: int = 0,
                  stream=None):
    """Append the new tokens' keys (normalised, rotated to their positions)
    and values [tokens, heads, head_dim] to the cache; with q, also normalise
    and rotate their queries into q_out (which may be q).  Returns q_out."""
    index = cache.index
    shape = (batch.tokens, cache.heads, cache.head_dim)
    hk, hv = _heads(k, "k", shape, index), _heads(v, "v", shape, index)
    if rope.head_dim is not None and rope.head_dim != cache.head_dim:
        raise ValueError(f"norm weights must have {cache.head_dim} elements")
    hq = hqo = None
    if q is not None:
        shape = (batch.tokens, _shape3(q, "q")[1], cache.head_dim)
        hq = _heads(q, "q", shape, index)
        if q_out is None:
            q_out = _like(q, stream)
        hqo = _heads(q_out, "q_out", shape, index)
    elif q_out is not None:
        raise ValueError("q_out without q")
    if batch.index != index or rope.index != index:
        _on(index, batch.index, "sgr_kv_append")
        _on(index, rope.index, "sgr_kv_append")
    _launch(index, stream, "sgr_kv_append", load().sgr_kv_append, cache.ref, batch.ref, hq, hk, hv, hqo, rope.ref, flags)
    return q_out


def kv_attention_workspace(cache: KvCache, batch: KvBatch, q_heads: int, flags: int = 0):
    """A workspace for sgr_kv_attention calls of these sizes and flags (one for each call that may overlap with others on the GPU)."""
    n = ctypes.c_int64(0)
    _check(load().sgr_kv_attention_workspace(cache.index, cache.ref, batch.ref, q_heads, flags, ctypes.byref(n)),
           "sgr_kv_attention_workspace")
    return torch.empty(n.value, dtype=torch.uint8, device=cache.device)


def sgr_kv_attention(cache: KvCache, batch: KvBatch, q, out=None, scale: float | None = None, window: int = 0,
                     workspace=None, flags: int = 0, stream=None):
    """Attention of the new tokens' queries [tokens, q_heads, head_dim] over
    the cached positions up to their own (the last `window` of them where
    window > 0), scores times `scale` (1/sqrt(head_dim) by default).
    Returns out."""
    index = cache.index
    shape = (batch.tokens, _shape3(q, "q")[1], cache.head_dim)
    hq = _heads(q, "q", shape, index)
    if out is None:
        out = _like(q, stream)
    ho = _heads(out, "out", shape, index)
    if workspace is None:
        workspace = _new(index, stream, lambda: kv_attention_workspace(cache, batch, shape[1], flags))
    elif not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    if batch.index != index or workspace.get_device() != index:
        _on(index, batch.index, "sgr_kv_attention")
        _on(index, workspace.get_device(), "sgr_kv_attention")
    _launch(index, stream, "sgr_kv_attention", load().sgr_kv_attention, cache.ref, batch.ref, hq, ho,
            shape[2] ** -0.5 if scale is None else scale, window, workspace.data_ptr(), workspace.nbytes, flags)
    return out
