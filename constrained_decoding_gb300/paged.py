"""Rotary positions and the 8-bit paged K/V cache on torch tensors: the calls
of include/pcd_kernels.h under their C names.

A serving layer runs them in this order, with one set of offsets, lengths and
block tables for the append and the attention::

    freqs, amp = paged.pcd_rope_freqs(128, 1e6)
    freqs = freqs.cuda()
    q = paged.pcd_k_rope(q, freqs, pos)
    paged.pcd_k_kv_append(k, v, k_cache, v_cache, k_scale, v_scale, q_off, kv_len, table, freqs=freqs)
    o = paged.pcd_k_paged_attention(q, k_cache, v_cache, k_scale, v_scale, q_off, kv_len, table)

Every call checks types, shapes and devices (ValueError), runs on its tensors'
device in torch's current stream there, and returns without synchronising; what
the library itself refuses raises PCDError.  A cache is two tensors [pages,
KV heads, page size, head dim] of torch.float8_e4m3fn or torch.int8 (any strides
that keep channels contiguous, the same for both) and two float32 scales
[pages, KV heads].

None of the calls records a gradient, so rows that require one are refused
unless gradients are off (torch.no_grad(), detach()); in a backward pass of
one's own, pcd_k_rope(..., transpose=True) is the rotation's gradient.  Writes to
`out`, the cache and its scales do not count as in-place changes that autograd
knows of: what it has saved must not be overwritten.
"""
from __future__ import annotations

import ctypes
import functools
import struct
from typing import Optional

import torch

from ._lib import load
from .pcd import PCDError, _check

_DTYPE = {torch.float32: 1, torch.bfloat16: 2, torch.float16: 3}
_FORMAT = {torch.float8_e4m3fn: 1, torch.int8: 2}
SCALING = {"none": 0, "linear": 1, "base": 2, "bands": 3, "ramp": 4}

_lib = load()
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)
_current_device = torch.cuda.current_device
_int32, _int64, _float32 = torch.int32, torch.int64, torch.float32
_INT = 0x7fffffff  # the library's sizes are C ints, which ctypes would fill with the low 32 bits of a larger one

# The checks below run on every call of a latency-bound loop, so a message is
# put together only when it is raised.


def _ints(t, dev: int, n: int, what: str) -> int:
    """The pointer of a contiguous int32 tensor of n elements on device `dev` (0 for None)."""
    if t is None:
        return 0
    if t.dtype is not _int32 or t.get_device() != dev or t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{what}: {n} contiguous int32 values on cuda:{dev}")
    return t.data_ptr()


def _rope(freqs, dev: int, dim: int):
    """(pointer, rot_dim) of a frequency tensor (0, 0 for None)."""
    if freqs is None:
        return 0, 0
    rot = 2 * freqs.numel()
    if freqs.dtype is not _int64 or freqs.get_device() != dev or freqs.dim() != 1 or not freqs.is_contiguous():
        raise ValueError(f"freqs: contiguous int64 values on cuda:{dev}")
    if not 0 < rot <= dim:
        raise ValueError("freqs: one value for each pair, 2 * pairs <= head_dim")
    return freqs.data_ptr(), rot


def _too_many():
    raise ValueError("under 2^31 tokens, heads, sequences and pages a sequence")


def _strides(t, dev: int, dim: int, what: str):
    """The strides of a [tokens, heads, dim] tensor on device `dev`."""
    st = t.stride()
    if t.get_device() != dev or (st[2] != 1 and dim != 1):
        raise ValueError(f"{what}: on cuda:{dev}, channels contiguous")
    if t.requires_grad and torch.is_grad_enabled():
        raise ValueError(f"{what}: requires a gradient, which this call does not record")
    return st


def _rows(t, dev: int, shape, dtype, what: str):
    """... that has this shape and type too."""
    if t.shape != shape or t.dtype is not dtype:
        raise ValueError(f"{what}: {list(shape)} of {dtype}")
    return _strides(t, dev, shape[2], what)


def _launch(dev: int, where: str, fn, *args) -> None:
    """fn(*args, stream) with `dev` the current device, in torch's current stream there."""
    cur = _current_device()
    if cur == dev:
        rc = fn(*args, _raw_stream(dev))
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, _raw_stream(dev))
    if rc:
        raise PCDError(rc, where)


def pcd_rope_freqs(rot_dim: int, theta: float, scaling: str = "none", factor: float = 1.0, orig_len: float = 0.0,
                   lo_turns: float = 1.0, hi_turns: Optional[float] = None):
    """(freqs, amp): an int64 CPU tensor of rot_dim / 2 turn fractions a position
    in units of 2^-64 (move it to the device once), and the factor on cos and
    sin.  scaling: "none", "linear", "base", "bands" or "ramp" for contexts
    `factor` times longer than orig_len; hi_turns defaults to 4 for "bands" and
    32 for "ramp"."""
    if scaling not in SCALING:
        raise ValueError(f"unknown scaling {scaling!r}")
    if hi_turns is None:
        hi_turns = 32.0 if scaling == "ramp" else 4.0
    out = torch.zeros(max(int(rot_dim) // 2, 1), dtype=torch.int64)
    amp = ctypes.c_float()
    _check(_lib.pcd_rope_freqs(int(rot_dim), float(theta), SCALING[scaling], float(factor), float(orig_len),
                                 float(lo_turns), float(hi_turns), out.data_ptr(), ctypes.byref(amp)), "pcd_rope_freqs")
    return out, amp.value


def pcd_k_rope(x, freqs, pos=None, *, base: int = 0, interleaved: bool = False, amp: float = 1.0,
               transpose: bool = False, out=None):
    """x [tokens, heads, head_dim] with its first 2 * len(freqs) channels rotated
    by each token's position (`pos`, int32, or base + row).  `transpose` turns
    back with the same amp: the gradient with respect to x.  `out` may be x."""
    shape, dtype, dev = x.shape, x.dtype, x.get_device()
    code = _DTYPE.get(dtype)
    if code is None or dev < 0 or len(shape) != 3:
        raise ValueError("x: a float32, float16 or bfloat16 CUDA tensor [tokens, heads, dim]")
    n, heads, dim = shape
    if n > _INT or heads > _INT:
        _too_many()
    xs = _strides(x, dev, dim, "x")
    f, rot = _rope(freqs, dev, dim)
    if base and not -0x80000000 <= base <= _INT:
        raise ValueError("base: a 32-bit integer")
    if out is None:
        out = torch.empty(shape, dtype=dtype, device=x.device)
        ys = (heads * dim, dim)
    else:
        ys = _rows(out, dev, shape, dtype, "out")
    _launch(dev, "pcd_k_rope", _lib.pcd_k_rope, x.data_ptr(), out.data_ptr(), code, n, heads, dim, xs[0], xs[1], ys[0],
            ys[1], f, rot, interleaved, amp, _ints(pos, dev, n, "pos"), base, transpose)
    return out


_PAGES = struct.Struct("@4P3q5i4x")  # pcd_kv_pages


def _pages(k_cache, v_cache, k_scale, v_scale):
    """(pcd_kv_pages as bytes, device, page size, KV heads, head dim) of a cache."""
    shape, dtype, dev, st = k_cache.shape, k_cache.dtype, k_cache.get_device(), k_cache.stride()
    fmt = _FORMAT.get(dtype)
    if fmt is None or dev < 0 or len(shape) != 4:
        raise ValueError("k_cache: a float8_e4m3fn or int8 CUDA tensor [pages, KV heads, page size, head dim]")
    if v_cache.dtype is not dtype or v_cache.get_device() != dev or v_cache.shape != shape or v_cache.stride() != st or st[3] != 1:
        raise ValueError("v_cache: k_cache's type, device, shape and strides; channels contiguous")
    two = shape[:2]
    for t in (k_scale, v_scale):
        if t.dtype is not _float32 or t.get_device() != dev or t.shape != two or not t.is_contiguous():
            raise ValueError("scales: contiguous float32 [pages, KV heads] on the cache's device")
    pages, heads, size, dim = shape
    return _PAGES.pack(k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), st[0], st[1], st[2],
                       pages, size, heads, dim, fmt), dev, size, heads, dim


def _table(table, n_seq: int, dev: int):
    """(pointer, row stride, width) of a block table."""
    shape = table.shape
    if table.dtype is _int32 and table.get_device() == dev and len(shape) == 2:
        n, width = shape
        stride, step = table.stride()
        if n_seq < 2:
            stride = width
        if n == n_seq and (step == 1 or width < 2) and stride >= width:
            if n + stride > _INT:
                _too_many()
            return table.data_ptr(), stride, width
    raise ValueError(f"table: int32 [{n_seq}, pages] on cuda:{dev}, rows contiguous")


def pcd_k_kv_append(k, v, k_cache, v_cache, k_scale, v_scale, q_off, kv_len, table, *, freqs=None,
                    interleaved: bool = False, amp: float = 1.0, pos=None, err=None) -> None:
    """Writes new rows k, v [tokens, KV heads, head_dim] (float32, float16 or
    bfloat16) into the cache, the keys rotated on the way when `freqs` is given.
    Rows q_off[s] .. q_off[s + 1) become the last tokens of sequence s, which has
    kv_len[s] with them; token j of it lies in page table[s, j // page size].
    (`table` may be a column slice of a wider one: a length beyond its own columns
    is out of range.)  A page that the call writes to stands once in the table.
    `err` (int32, one element) is set nonzero when offsets, lengths or pages
    were out of range; without it, what was skipped goes unsaid."""
    c, dev, _, kv_heads, dim = _pages(k_cache, v_cache, k_scale, v_scale)
    dtype, shape, n_seq = k.dtype, k.shape, kv_len.numel()
    code = _DTYPE.get(dtype)
    if code is None or len(shape) != 3 or shape[1] != kv_heads or shape[2] != dim:
        raise ValueError("k: float32, float16 or bfloat16 [tokens, KV heads, head dim]")
    n = shape[0]
    if n > _INT:
        _too_many()
    ks, vs = _strides(k, dev, dim, "k"), _rows(v, dev, shape, dtype, "v")
    t, t_stride, width = _table(table, n_seq, dev)
    f, rot = _rope(freqs, dev, dim)
    _launch(dev, "pcd_k_kv_append", _lib.pcd_k_kv_append_cols, c, k.data_ptr(), v.data_ptr(), code, ks[0], ks[1],
            vs[0], vs[1], _ints(q_off, dev, n_seq + 1, "q_off"), _ints(kv_len, dev, n_seq, "kv_len"), t, n_seq, n, t_stride,
            width, f, rot, interleaved, amp, _ints(pos, dev, n, "pos"), _ints(err, dev, 1, "err"))


def pcd_k_paged_attention_scratch_bytes(n_tok: int, n_seq: int, n_q_heads: int, n_kv_heads: int, head_dim: int,
                                        max_kv: int) -> int:
    if max(n_tok, n_seq, n_q_heads, n_kv_heads, head_dim) > _INT:
        _too_many()
    return int(_lib.pcd_k_paged_attention_scratch_bytes(n_tok, n_seq, n_q_heads, n_kv_heads, head_dim, max_kv))


@functools.lru_cache(maxsize=1024)
def _scratch_bytes(dev: int, *sizes) -> int:
    """What a call of these sizes needs on this device: a function of them alone."""
    if _current_device() == dev:
        return _lib.pcd_k_paged_attention_scratch_bytes(*sizes)
    with torch.cuda.device(dev):
        return _lib.pcd_k_paged_attention_scratch_bytes(*sizes)


def pcd_k_paged_attention(q, k_cache, v_cache, k_scale, v_scale, q_off, kv_len, table, *, max_kv: Optional[int] = None,
                          causal: bool = True, scale: Optional[float] = None, out=None, return_lse: bool = False,
                          scratch=None, err=None):
    """softmax(scale q k^T) v of q [tokens, query heads, head_dim] (float16 or
    bfloat16) over the cached tokens.  Rows q_off[s] .. q_off[s + 1) are the last
    tokens of sequence s and see up to themselves (`causal`), or all kv_len[s]
    tokens.  Rows behind the last offset are not written.  max_kv: the longest
    kv_len, if the caller knows it (default: what the table holds); scale
    defaults to head_dim ** -0.5.  `out` may be q.  Returns the output, and with return_lse the
    log-sum-exp [tokens, query heads] too.  `scratch` (uint8) replaces the
    workspace that is otherwise taken from torch's allocator.  `err` (int32, one
    element) is set nonzero when offsets, lengths or pages were out of range (such
    keys are not seen, rows of bad offsets not written), or when a wait of the
    kernel's pipelines ran out (those rows are NaN); without it, nothing tells of
    the former."""
    c, dev, page, kv_heads, dim = _pages(k_cache, v_cache, k_scale, v_scale)
    dtype, shape, n_seq = q.dtype, q.shape, kv_len.numel()
    if (dtype is not torch.float16 and dtype is not torch.bfloat16) or len(shape) != 3 or shape[2] != dim:
        raise ValueError("q: float16 or bfloat16 [tokens, heads, head dim]")
    n, heads, _ = shape
    if n > _INT or heads > _INT:
        _too_many()
    qs = _strides(q, dev, dim, "q")
    t, t_stride, width = _table(table, n_seq, dev)
    if out is None:
        out = torch.empty(shape, dtype=dtype, device=q.device)
        os = (heads * dim, dim)
    else:
        os = _rows(out, dev, shape, dtype, "out")
    lse = torch.empty((n, heads), dtype=_float32, device=q.device) if return_lse else None
    if max_kv is None:
        max_kv = width * page
    if scratch is None:
        need = _scratch_bytes(dev, n, n_seq, heads, kv_heads, dim, max_kv)
        if need > 0:
            scratch = torch.empty(need, dtype=torch.uint8, device=q.device)
    elif scratch.get_device() != dev or not scratch.is_contiguous():
        raise ValueError(f"scratch: contiguous bytes on cuda:{dev}")
    else:
        need = scratch.numel() * scratch.element_size()
    _launch(dev, "pcd_k_paged_attention", _lib.pcd_k_paged_attention_cols, c, q.data_ptr(), out.data_ptr(),
            lse.data_ptr() if return_lse else 0, _DTYPE[dtype], heads, qs[0], qs[1], os[0], os[1],
            _ints(q_off, dev, n_seq + 1, "q_off"), _ints(kv_len, dev, n_seq, "kv_len"), t, n_seq, n, t_stride, width, max_kv,
            causal, dim ** -0.5 if scale is None else scale, 0 if scratch is None else scratch.data_ptr(), need,
            _ints(err, dev, 1, "err"))
    return (out, lse) if return_lse else out
