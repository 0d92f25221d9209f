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
"""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

from . import _decls as D
from ._lib import load
from .pcd import PCDError, _check

_DTYPE = {torch.float32: 1, torch.bfloat16: 2, torch.float16: 3}
_FORMAT = {torch.float8_e4m3fn: 1, torch.int8: 2}
SCALING = {"none": 0, "linear": 1, "base": 2, "bands": 3, "ramp": 4}

_lib = None


def _get():
    global _lib
    if _lib is None:
        _lib = load()
    return _lib


def _need(ok, what: str) -> None:
    if not ok:
        raise ValueError(what)


def _int32(t, device, n: int, what: str) -> int:
    """The pointer of a contiguous int32 tensor of n elements on `device` (0 for None)."""
    if t is None:
        return 0
    _need(t.dtype is torch.int32 and t.device == device and t.numel() == n and t.is_contiguous(),
          f"{what}: {n} contiguous int32 values on {device}")
    return t.data_ptr()


def _rope(freqs, device, dim: int):
    """(pointer, rot_dim) of a frequency tensor (0, 0 for None)."""
    if freqs is None:
        return 0, 0
    _need(freqs.dtype is torch.int64 and freqs.device == device and freqs.dim() == 1 and freqs.is_contiguous(),
          f"freqs: contiguous int64 values on {device}")
    rot = 2 * freqs.numel()
    _need(0 < rot <= dim, "freqs: one value for each pair, 2 * pairs <= head_dim")
    return freqs.data_ptr(), rot


def _rows(t, heads, dim, device, what: str) -> None:
    _need(t.device == device and t.dim() == 3 and t.shape[1] == heads and t.shape[2] == dim and
          (t.stride(2) == 1 or dim == 1), f"{what}: [tokens, {heads}, {dim}] on {device}, channels contiguous")


class _On:
    """Makes a tensor's device the current one (only when it is not), and gives its current stream."""
    __slots__ = ("index", "back")

    def __init__(self, device):
        self.index = device.index
        self.back = -1

    def __enter__(self):
        cur = torch.cuda.current_device()
        if cur != self.index:
            self.back = cur
            torch.cuda.set_device(self.index)
        return torch.cuda.current_stream(self.index).cuda_stream

    def __exit__(self, *exc):
        if self.back >= 0:
            torch.cuda.set_device(self.back)


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
    _check(_get().pcd_rope_freqs(int(rot_dim), float(theta), SCALING[scaling], float(factor), float(orig_len),
                                 float(lo_turns), float(hi_turns), out.data_ptr(), ctypes.byref(amp)), "pcd_rope_freqs")
    return out, amp.value


def pcd_k_rope(x, freqs, pos=None, *, base: int = 0, interleaved: bool = False, amp: float = 1.0,
               transpose: bool = False, out=None):
    """x [tokens, heads, head_dim] with its first 2 * len(freqs) channels rotated
    by each token's position (`pos`, int32, or base + row).  `transpose` turns
    back with the same amp: the gradient with respect to x.  `out` may be x."""
    _need(x.is_cuda and x.dim() == 3 and x.dtype in _DTYPE, "x: a float32, float16 or bfloat16 CUDA tensor [tokens, heads, dim]")
    n, heads, dim = x.shape
    dev = x.device
    _rows(x, heads, dim, dev, "x")
    f, rot = _rope(freqs, dev, dim)
    p = _int32(pos, dev, n, "pos")
    if out is None:
        out = torch.empty(x.shape, dtype=x.dtype, device=dev)
    else:
        _rows(out, heads, dim, dev, "out")
        _need(out.dtype is x.dtype and out.shape[0] == n, "out: x's shape and type")
    with _On(dev) as stream:
        rc = _get().pcd_k_rope(x.data_ptr(), out.data_ptr(), _DTYPE[x.dtype], n, heads, dim, x.stride(0), x.stride(1),
                               out.stride(0), out.stride(1), f, rot, interleaved, amp, p, base, transpose, stream)
    if rc:
        raise PCDError(rc, "pcd_k_rope")
    return out


def _pages(k_cache, v_cache, k_scale, v_scale) -> D.pcd_kv_pages:
    dev = k_cache.device
    _need(k_cache.is_cuda and k_cache.dim() == 4 and k_cache.dtype in _FORMAT,
          "k_cache: a float8_e4m3fn or int8 CUDA tensor [pages, KV heads, page size, head dim]")
    _need(v_cache.dtype is k_cache.dtype and v_cache.device == dev and v_cache.shape == k_cache.shape and
          v_cache.stride() == k_cache.stride() and k_cache.stride(3) == 1,
          "v_cache: k_cache's type, device, shape and strides; channels contiguous")
    pages, heads, size, dim = k_cache.shape
    for t in (k_scale, v_scale):
        _need(t.dtype is torch.float32 and t.device == dev and t.dim() == 2 and t.shape[0] == pages and
              t.shape[1] == heads and t.is_contiguous(), "scales: contiguous float32 [pages, KV heads] on the cache's device")
    st = k_cache.stride()
    return D.pcd_kv_pages(k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), st[0], st[1],
                          st[2], pages, size, heads, dim, _FORMAT[k_cache.dtype])


def _table(table, n_seq: int, dev):
    _need(table.dtype is torch.int32 and table.device == dev and table.dim() == 2 and table.shape[0] == n_seq and
          (table.stride(1) == 1 or table.shape[1] <= 1) and table.stride(0) >= table.shape[1],
          f"table: int32 [{n_seq}, pages] on {dev}, rows contiguous")
    return table.data_ptr(), table.stride(0) if n_seq > 1 else table.shape[1]


def pcd_k_kv_append(k, v, k_cache, v_cache, k_scale, v_scale, q_off, kv_len, table, *, freqs=None,
                    interleaved: bool = False, amp: float = 1.0, pos=None, err=None) -> None:
    """Writes new rows k, v [tokens, KV heads, head_dim] (float32, float16 or
    bfloat16) into the cache, the keys rotated on the way when `freqs` is given.
    Rows q_off[s] .. q_off[s + 1) become the last tokens of sequence s, which has
    kv_len[s] with them; token j of it lies in page table[s, j // page size].
    `err` (int32, one element) is set nonzero when offsets, lengths or pages
    were out of range."""
    c = _pages(k_cache, v_cache, k_scale, v_scale)
    dev = k_cache.device
    heads, dim = c.n_kv_heads, c.head_dim
    _need(k.dtype in _DTYPE and v.dtype is k.dtype, "k, v: float32, float16 or bfloat16, the same")
    _rows(k, heads, dim, dev, "k")
    _rows(v, heads, dim, dev, "v")
    n, n_seq = k.shape[0], kv_len.numel()
    _need(v.shape[0] == n, "k and v: the same tokens")
    t, t_stride = _table(table, n_seq, dev)
    f, rot = _rope(freqs, dev, dim)
    args = (_int32(q_off, dev, n_seq + 1, "q_off"), _int32(kv_len, dev, n_seq, "kv_len"), t, n_seq, n, t_stride, f, rot,
            interleaved, amp, _int32(pos, dev, n, "pos"), _int32(err, dev, 1, "err"))
    with _On(dev) as stream:
        rc = _get().pcd_k_kv_append(ctypes.byref(c), k.data_ptr(), v.data_ptr(), _DTYPE[k.dtype], k.stride(0),
                                    k.stride(1), v.stride(0), v.stride(1), *args, stream)
    if rc:
        raise PCDError(rc, "pcd_k_kv_append")


def pcd_k_paged_attention_scratch_bytes(n_tok: int, n_seq: int, n_q_heads: int, n_kv_heads: int, head_dim: int,
                                        max_kv: int) -> int:
    return int(_get().pcd_k_paged_attention_scratch_bytes(n_tok, n_seq, n_q_heads, n_kv_heads, head_dim, max_kv))


def pcd_k_paged_attention(q, k_cache, v_cache, k_scale, v_scale, q_off, kv_len, table, *, max_kv: Optional[int] = None,
                          causal: bool = True, scale: Optional[float] = None, out=None, return_lse: bool = False,
                          scratch=None, err=None):
    """softmax(scale q k^T) v of q [tokens, query heads, head_dim] (float16 or
    bfloat16) over the cached tokens.  Rows q_off[s] .. q_off[s + 1) are the last
    tokens of sequence s and see up to themselves (`causal`), or all kv_len[s]
    tokens.  Rows behind the last offset are not written.  max_kv: the longest
    kv_len, if the caller knows it (default: what the table holds); scale
    defaults to head_dim ** -0.5.  Returns the output, and with return_lse the
    log-sum-exp [tokens, query heads] too.  `scratch` (uint8) replaces the
    workspace that is otherwise taken from torch's allocator."""
    c = _pages(k_cache, v_cache, k_scale, v_scale)
    dev = k_cache.device
    dim = c.head_dim
    _need(q.dim() == 3 and (q.dtype is torch.float16 or q.dtype is torch.bfloat16),
          "q: a float16 or bfloat16 tensor [tokens, heads, dim]")
    n, heads, n_seq = q.shape[0], q.shape[1], kv_len.numel()
    _rows(q, heads, dim, dev, "q")
    t, t_stride = _table(table, n_seq, dev)
    if out is None:
        out = torch.empty(q.shape, dtype=q.dtype, device=dev)
    else:
        _rows(out, heads, dim, dev, "out")
        _need(out.dtype is q.dtype and out.shape[0] == n, "out: q's shape and type")
    lse = torch.empty((n, heads), dtype=torch.float32, device=dev) if return_lse else None
    if max_kv is None:
        max_kv = table.shape[1] * c.page_size
    args = (_int32(q_off, dev, n_seq + 1, "q_off"), _int32(kv_len, dev, n_seq, "kv_len"), t, n_seq, n, t_stride, max_kv,
            causal, dim ** -0.5 if scale is None else scale)
    e = _int32(err, dev, 1, "err")
    lib = _get()
    with _On(dev) as stream:
        need = lib.pcd_k_paged_attention_scratch_bytes(n, n_seq, heads, c.n_kv_heads, dim, max_kv)
        if scratch is None:
            if need:
                scratch = torch.empty(need, dtype=torch.uint8, device=dev)
        else:
            _need(scratch.device == dev and scratch.is_contiguous(), f"scratch: contiguous bytes on {dev}")
            need = scratch.numel() * scratch.element_size()
        rc = lib.pcd_k_paged_attention(ctypes.byref(c), q.data_ptr(), out.data_ptr(),
                                       lse.data_ptr() if return_lse else 0, _DTYPE[q.dtype], heads, q.stride(0),
                                       q.stride(1), out.stride(0), out.stride(1), *args,
                                       scratch.data_ptr() if scratch is not None else 0, need, e, stream)
    if rc:
        raise PCDError(rc, "pcd_k_paged_attention")
    return (out, lse) if return_lse else out
