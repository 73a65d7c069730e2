"""A serving step around a paged cache: the plan, rotary positions with the cache write, attention.

Marshals arguments for ``qaff_paged_plan``, ``qaff_rope_append`` and ``qaff_paged_attention`` of
``include/qaff.h``; every step of the computation runs in the library's kernels, on the current
stream. Caches are ``[pages, kv_heads, page_size, head_dim]`` in bf16 or float16, each page
contiguous (the pages may be strided: K and V pages may alternate in one tensor).

    plan = paged_plan(cached_lens, new_lens, free_pages, block_tables, page_size, tokens)  # once a step
    q = rope_append(q, k, v, plan.positions, inv_freq, plan.slots, k_cache, v_cache)       # per layer
    o = paged_attention(q, k_cache, v_cache, block_tables, plan.cu_new, plan.kv_lens)
"""
from __future__ import annotations

import contextlib
import ctypes
import math
from typing import NamedTuple

import torch

from . import _lib

__all__ = ["PagedPlan", "paged_plan", "rope_append", "paged_attention"]

_HALF = {torch.bfloat16: _lib.QAFF_BF16, torch.float16: _lib.QAFF_F16}


class PagedPlan(NamedTuple):
    """What a step's kernels need to know of its requests (``paged_plan``)."""

    cu_new: torch.Tensor      # int32 [requests + 1]: exclusive prefix sums of the new tokens
    kv_lens: torch.Tensor     # int32 [requests]: tokens in the cache once the step is written
    positions: torch.Tensor   # int32 [tokens]
    slots: torch.Tensor       # int64 [tokens]: page * page_size + offset, -1 where there is none
    pages_used: torch.Tensor  # int32 [1]: free pages the step takes


def _tensor(t, name, dtypes, device=None, dim=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be on a GPU device, got {t.device}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} has dtype {t.dtype}, expected one of {dtypes}")
    if dim is not None and t.dim() != dim:
        raise ValueError(f"{name} must have {dim} dimensions, got {t.dim()}")


def _flat(t, name, dtypes, device=None, dim=None):
    _tensor(t, name, dtypes, device, dim)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


_I32 = (torch.int32,)


def _on(dev):
    """The device to launch on: nothing to do where it is current already."""
    return contextlib.nullcontext() if torch.cuda.current_device() == dev.index else torch.cuda.device(dev)


def _stream(dev):
    return torch.cuda.current_stream(dev).cuda_stream


def _p(t):
    return t.data_ptr() if t.numel() else None


def _heads(t, name, dtypes, dev=None):
    """A [tokens, heads, head_dim] operand, its last axis contiguous; its token and head strides."""
    _tensor(t, name, dtypes, dev, 3)
    if t.stride(2) != 1 and t.shape[2] > 1:
        raise ValueError(f"the last axis of {name} must be contiguous")
    return t.stride(0), t.stride(1)


def _cache(k_cache, v_cache, dtype, dev):
    """Both caches: (pages, kv_heads, page_size, head_dim, page stride)."""
    for t, name in ((k_cache, "k_cache"), (v_cache, "v_cache")):
        _tensor(t, name, (dtype,), dev, 4)
    if k_cache.shape != v_cache.shape:
        raise ValueError(f"k_cache {list(k_cache.shape)} and v_cache {list(v_cache.shape)} differ")
    pages, heads, size, dim = k_cache.shape
    strides = k_cache.stride()
    if strides[1:] != (size * dim, dim, 1) and k_cache.numel():
        raise ValueError("each page of the caches must be contiguous: [kv_heads, page_size, head_dim]")
    if v_cache.stride() != strides:
        raise ValueError("k_cache and v_cache differ in their strides")
    return pages, heads, size, dim, strides[0] if pages > 1 else heads * size * dim


def paged_plan(cached_lens, new_lens, free_pages, block_tables, page_size: int, tokens: int) -> PagedPlan:
    """Block tables and slots of a step's new tokens, from the request lengths (all on the GPU).

    ``cached_lens`` and ``new_lens`` are int32 ``[requests]``: tokens each request has in the cache
    and tokens it brings. ``free_pages`` is int32, the pages no request holds: the step takes the
    first ``pages_used`` of them, in order, and writes them into ``block_tables`` (int32
    ``[requests, width]``, in place) behind the pages a request already has. ``tokens`` is the
    number of rows to describe: the step's tokens, or more (rows past them get slot -1). Where the
    free pages or a table's width run out, the entries and slots are -1."""
    lib = _lib.load()
    _flat(cached_lens, "cached_lens", _I32, None, 1)
    dev = cached_lens.device
    _flat(new_lens, "new_lens", _I32, dev, 1)
    _flat(free_pages, "free_pages", _I32, dev, 1)
    _flat(block_tables, "block_tables", _I32, dev, 2)
    requests = cached_lens.shape[0]
    if new_lens.shape[0] != requests or block_tables.shape[0] != requests:
        raise ValueError(f"cached_lens has {requests} requests, new_lens {new_lens.shape[0]}, block_tables "
                         f"{block_tables.shape[0]}")
    if tokens < 0:
        raise ValueError(f"tokens is {tokens}")
    ints = dict(dtype=torch.int32, device=dev)
    plan = PagedPlan(torch.empty(requests + 1, **ints), torch.empty(requests, **ints), torch.empty(tokens, **ints),
                     torch.empty(tokens, dtype=torch.int64, device=dev), torch.empty(1, **ints))
    with _on(dev):
        _lib.check(lib.qaff_paged_plan(_p(cached_lens), _p(new_lens), requests, _p(free_pages), free_pages.shape[0],
                                       _p(block_tables), block_tables.shape[1], page_size, tokens, _p(plan.cu_new),
                                       _p(plan.kv_lens), _p(plan.positions), _p(plan.slots), _p(plan.pages_used),
                                       _stream(dev)))
    return plan


def rope_append(q, k, v, positions, inv_freq, slots, k_cache, v_cache, sections=None, interleaved: bool = False,
                traditional: bool = False, out=None):
    """Turns q ``[tokens, heads, head_dim]`` and k ``[tokens, kv_heads, head_dim]`` by their rotary
    positions, writes the turned k and v to their slots of the caches (in place) and returns the
    turned q. q, k and v may be views of one projection's rows (any token and head strides).

    ``inv_freq`` (float32 ``[rot / 2]``) has an entry per pair of the first ``rot`` values of a head;
    the rest pass. Pair i is values i and i + rot / 2, or 2 i and 2 i + 1 with ``traditional``.
    ``positions`` is int32 ``[tokens]``, or ``[axes, tokens]`` with ``sections``, the pairs of each
    axis (time, height, width): in order, or ``interleaved`` (pair i to axis i % axes while that
    axis has pairs left, else to the first). A token whose slot is below 0 or past the caches is
    not written."""
    lib = _lib.load()
    q_ts, q_hs = _heads(q, "q", tuple(_HALF))
    dev, dt = q.device, q.dtype
    k_ts, k_hs = _heads(k, "k", (dt,), dev)
    v_ts, v_hs = _heads(v, "v", (dt,), dev)
    tokens, heads, dim = q.shape
    pages, kv_heads, size, cache_dim, page_stride = _cache(k_cache, v_cache, dt, dev)
    want = (tokens, kv_heads, dim)
    if cache_dim != dim or k.shape != want or v.shape != want:
        raise ValueError(f"q {list(q.shape)} with caches {list(k_cache.shape)} needs k and v {list(want)}, got "
                         f"{list(k.shape)} and {list(v.shape)}")
    _flat(positions, "positions", _I32, dev)
    axes = 1 if positions.dim() == 1 else positions.shape[0]
    if positions.dim() not in (1, 2) or positions.shape[-1] != tokens:
        raise ValueError(f"positions must be [{tokens}] or [axes, {tokens}], got {list(positions.shape)}")
    _flat(inv_freq, "inv_freq", (torch.float32,), dev, 1)
    _flat(slots, "slots", (torch.int64,), dev, 1)
    if slots.shape[0] != tokens:
        raise ValueError(f"slots must be [{tokens}], got {list(slots.shape)}")
    if sections is not None:
        if len(sections) != axes:
            raise ValueError(f"{len(sections)} sections for {axes} axes")
        sections = (ctypes.c_int32 * axes)(*sections)
    if out is None:
        out = torch.empty((tokens, heads, dim), dtype=dt, device=dev)
    else:
        _flat(out, "out", (dt,), dev)
        if out.shape != q.shape:
            raise ValueError(f"out must be {list(q.shape)}")
    with _on(dev):
        _lib.check(lib.qaff_rope_append(_p(q), _p(k), _p(v), _HALF[dt], tokens, heads, kv_heads, dim, q_ts, q_hs, k_ts,
                                        k_hs, v_ts, v_hs, _p(positions), axes, sections, interleaved, traditional,
                                        _p(inv_freq), 2 * inv_freq.shape[0], _p(slots), _p(k_cache), _p(v_cache),
                                        pages, page_stride, size, _p(out), _stream(dev)))
    return out


def paged_attention(q, k_cache, v_cache, block_tables, cu_new, kv_lens, max_new=None, scale=None, causal: bool = True,
                    window: int = 0, return_lse: bool = False, out=None):
    """Attention of the step's new tokens over the paged caches, which already hold their keys and
    values (``rope_append``): q ``[tokens, heads, head_dim]`` (any token and head strides), heads a
    multiple of the caches' kv_heads; returns ``[tokens, heads, head_dim]`` in q's dtype, and with
    ``return_lse`` also the float32 ``[tokens, heads]`` logarithm of each row's sum of exponentials.

    Request b's tokens are rows ``cu_new[b]`` to ``cu_new[b + 1]``, the last at position
    ``kv_lens[b] - 1``; its keys are in the pages of ``block_tables[b]``. A token at position p sees
    the keys up to p (``causal``), and with ``window`` only the last ``window`` of them. A token that
    sees none, and a row past every request, gets zeros (lse -inf). ``scale`` defaults to
    ``head_dim ** -0.5``. ``max_new``, the largest number of new tokens of any request or a bound of
    it, lets the library choose its kernels without reading ``cu_new`` back (default: all rows)."""
    lib = _lib.load()
    q_ts, q_hs = _heads(q, "q", tuple(_HALF))
    dev, dt = q.device, q.dtype
    tokens, heads, dim = q.shape
    pages, kv_heads, size, cache_dim, page_stride = _cache(k_cache, v_cache, dt, dev)
    if cache_dim != dim:
        raise ValueError(f"q has heads of {dim}, the caches of {cache_dim}")
    _flat(block_tables, "block_tables", _I32, dev, 2)
    _flat(cu_new, "cu_new", _I32, dev, 1)
    _flat(kv_lens, "kv_lens", _I32, dev, 1)
    requests, width = block_tables.shape
    if kv_lens.shape[0] != requests or cu_new.shape[0] != requests + 1:
        raise ValueError(f"block_tables has {requests} requests, kv_lens {kv_lens.shape[0]}, cu_new needs "
                         f"{requests + 1} entries and has {cu_new.shape[0]}")
    if scale is None:
        scale = 1.0 / math.sqrt(dim) if dim else 1.0
    max_new = tokens if max_new is None else max_new
    if out is None:
        out = torch.empty((tokens, heads, dim), dtype=dt, device=dev)
    else:
        _flat(out, "out", (dt,), dev)
        if out.shape != q.shape:
            raise ValueError(f"out must be {list(q.shape)}")
    lse = torch.empty((tokens, heads), dtype=torch.float32, device=dev) if return_lse else None
    nbytes = lib.qaff_paged_attention_workspace_size(tokens, heads, kv_heads, dim, size, width, requests, max_new)
    ws = torch.empty(nbytes, dtype=torch.uint8, device=dev) if nbytes else None
    with _on(dev):
        _lib.check(lib.qaff_paged_attention(_p(q), _HALF[dt], tokens, heads, q_ts, q_hs, _p(k_cache), _p(v_cache),
                                            pages, page_stride, kv_heads, dim, size, _p(block_tables), width,
                                            _p(cu_new), _p(kv_lens), requests, max_new, scale, causal, window,
                                            None if ws is None else ws.data_ptr(), nbytes, _p(out),
                                            None if lse is None else _p(lse), _stream(dev)))
    return (out, lse) if return_lse else out
