"""A serving step around a paged cache: the plan, rotary positions with the cache write, attention.

Calls ``qaff_paged_plan``, ``qaff_rope_append`` and ``qaff_paged_attention`` of ``include/qaff.h``
through ``_paged.so``, which checks and marshals the arguments; every step of the computation runs in
the library's kernels, on the current stream. Caches are ``[pages, kv_heads, page_size, head_dim]``
in bf16 or float16, each page contiguous (the pages may be strided: K and V pages may alternate in
one tensor).

    plan = paged_plan(cached_lens, new_lens, free_pages, block_tables, page_size, tokens)  # once a step
    q = rope_append(q, k, v, plan.positions, inv_freq, plan.slots, k_cache, v_cache)       # per layer
    o = paged_attention(q, k_cache, v_cache, block_tables, plan.cu_new, plan.kv_lens)
"""
from __future__ import annotations

import os
from typing import NamedTuple

import torch

from . import _lib

__all__ = ["PagedPlan", "paged_plan", "rope_append", "paged_attention"]

MODULE_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_paged.so")
_module = None


def _load():
    """The in-tree _paged.so (argument checks and marshalling in C++). Raises if it is not built."""
    global _module
    if _module is None:
        if not os.path.exists(MODULE_PATH):
            raise RuntimeError(f"{MODULE_PATH} is not built; run `python -m quantized_matmul_mlx_amd.build` "
                               "(or __graft_entry__.build()) first")
        _lib.load()
        from . import _paged
        _module = _paged
    return _module


class PagedPlan(NamedTuple):
    """What a step's kernels need to know of its requests (``paged_plan``)."""

    cu_new: torch.Tensor      # int32 [requests + 1]: exclusive prefix sums of the new tokens
    kv_lens: torch.Tensor     # int32 [requests]: tokens in the cache once the step is written
    positions: torch.Tensor   # int32 [tokens]
    slots: torch.Tensor       # int64 [tokens]: page * page_size + offset, -1 where there is none
    pages_used: torch.Tensor  # int32 [1]: free pages the step takes


def paged_plan(cached_lens, new_lens, free_pages, block_tables, page_size: int, tokens: int) -> PagedPlan:
    """Block tables and slots of a step's new tokens, from the request lengths (all on the GPU).

    ``cached_lens`` and ``new_lens`` are int32 ``[requests]``: tokens each request has in the cache
    and tokens it brings. ``free_pages`` is int32, the pages no request holds: the step takes the
    first ``pages_used`` of them, in order, and writes them into ``block_tables`` (int32
    ``[requests, width]``, in place) behind the pages a request already has. ``tokens`` is the
    number of rows to describe: the step's tokens, or more (rows past them get slot -1). Where the
    free pages or a table's width run out, the entries and slots are -1."""
    return PagedPlan(*_load().paged_plan(cached_lens, new_lens, free_pages, block_tables, page_size, tokens))


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
    return _load().rope_append(q, k, v, positions, inv_freq, slots, k_cache, v_cache, sections, interleaved, traditional,
                               out)


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
    it, lets the library choose its kernels without reading ``cu_new`` back (default: all rows, with
    which 64 decoding requests of up to 8192 keys take 250 us instead of 203). Where ``cu_new`` goes past
    the rows of q, only the rows that are there are computed."""
    return _load().paged_attention(q, k_cache, v_cache, block_tables, cu_new, kv_lens, max_new, scale, causal, window,
                                   return_lse, out)
