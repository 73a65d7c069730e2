"""A decoder's feed-forward over weights of few bits: the router and the experts of a mixture of experts,
and products in 8-bit floating point with a scale for each block of 128.

Calls ``qaff_moe_route``, ``qaff_moe_ffn``, ``qaff_block_quantize`` and ``qaff_block_qmm`` of
``include/qaff.h`` through ``_ffn.so``, which checks and marshals the arguments; every step of the
computation runs in the library's kernels, on the current stream.

    weights, experts = moe_route(router_logits, 8)
    y = moe_ffn(x, experts, weights, gate, up, down, group_size, bits, resid=x0)   # (packed, scales, biases) each

    w = BlockWeight(*block_quantize(weight, block_rows=128))                        # once
    y = w.mm(x)                                                                     # quantizes x, then the product
"""
from __future__ import annotations

import os

import torch

from . import _lib

__all__ = ["moe_route", "moe_ffn", "block_quantize", "block_qmm", "BlockWeight"]

MODULE_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_ffn.so")
_module = None


def _load():
    """The in-tree _ffn.so (argument checks and marshalling in C++). Raises if it is not built."""
    global _module
    if _module is None:
        if not os.path.exists(MODULE_PATH):
            raise RuntimeError(f"{MODULE_PATH} is not built; run `python -m quantized_matmul_mlx_amd.build` "
                               "(or __graft_entry__.build()) first")
        _lib.load()
        from . import _ffn
        _module = _ffn
    return _module


def moe_route(logits, top_k: int, bias=None, scoring: str = "softmax", renormalize: bool = True, scale: float = 1.0):
    """The experts of each token and their weights, from the router's logits ``[..., experts]`` (float32,
    bf16 or float16; a 2-D one may have any row stride): returns float32 weights and int32 experts, both
    ``[..., top_k]``, in falling order of the choice.

    The choice takes the largest logits (ties: the lowest index), or with ``bias`` (float32
    ``[experts]``) the largest ``score + bias``. The weight is the score without the bias,
    ``softmax(logits)`` or with ``scoring="sigmoid"`` ``sigmoid(logit)``, divided by the sum over the
    chosen ones with ``renormalize``, times ``scale``. A logit of -infinity (or NaN) is an expert that is
    switched off: it is chosen only where no others are left, with weight 0."""
    if scoring not in ("softmax", "sigmoid"):
        raise ValueError(f"scoring must be 'softmax' or 'sigmoid', got {scoring!r}")
    return _load().moe_route(logits, top_k, bias, scoring == "sigmoid", renormalize, scale)


def moe_ffn(x, experts, weights, gate, up, down, group_size: int, bits: int, resid=None, out=None):
    """The layer of a mixture of experts with quantized weights:

        y[t] = resid[t] + sum_j weights[t, j] * down[e] (silu(gate[e] x[t]) * (up[e] x[t])),  e = experts[t, j]

    x is bf16 or float16 ``[..., width]``; ``experts`` (int32) and ``weights`` (float32) are ``[..., top_k]``,
    as ``moe_route`` returns them. ``gate`` and ``up`` are ``(packed, scales, biases)`` of
    ``[n_experts, hidden, width]``, ``down`` of ``[n_experts, width, hidden]``, scales and biases in x's
    dtype (``quantize`` of a dense weight stack gives them). An expert outside ``0 .. n_experts - 1`` adds
    nothing: a share of the experts on one GPU, or a padded token. ``resid`` has x's shape."""
    return _load().moe_ffn(x, experts, weights, gate, up, down, group_size, bits, resid, out)


def block_quantize(x, block_rows: int = 1):
    """x ``[..., cols]`` (float32, bf16 or float16; a 2-D one may have any row stride) in 8-bit floating point
    with a float32 scale for each 128 columns: returns codes (``torch.float8_e4m3fn``, x's shape) and scales
    ``[..., ceil(cols / 128)]``; with ``block_rows=128`` (weights, 2-D) a scale for each 128 x 128 block,
    ``[ceil(rows / 128), ceil(cols / 128)]``. The scale is the block's largest magnitude / 448; a NaN or
    an infinity makes its block NaN."""
    return _load().block_quantize(x, block_rows)


def block_qmm(x, x_scales, w, w_scales, out_dtype=torch.bfloat16, out=None):
    """``x . w^T`` of operands in 8-bit floating point with block scales: x ``[..., k]`` with scales
    ``[..., ceil(k / 128)]``, w ``[n, k]`` with scales ``[ceil(n / 128), ceil(k / 128)]`` (``block_quantize``);
    returns ``[..., n]`` in ``out_dtype`` (float32, bf16 or float16)."""
    return _load().block_qmm(x, x_scales, w, w_scales, out_dtype, out)


class BlockWeight:
    """A weight ``[out, in]`` in 8-bit floating point with a scale for each 128 x 128 block. The caller owns
    the tensors."""

    __slots__ = ("codes", "scales", "shape")

    def __init__(self, codes, scales):
        self.codes, self.scales = codes, scales
        self.shape = tuple(codes.shape)
        want = tuple(-(-n // 128) for n in self.shape)
        if len(self.shape) != 2 or tuple(scales.shape) != want:
            raise ValueError(f"codes must be 2-D with scales {list(want)}, got {list(self.shape)} and {list(scales.shape)}")

    def mm(self, x, out_dtype=None):
        """x @ W.T, with x quantized on the way; the result has x's dtype unless ``out_dtype`` says another."""
        codes, scales = block_quantize(x)
        return block_qmm(codes, scales, self.codes, self.scales, out_dtype=out_dtype or x.dtype)
