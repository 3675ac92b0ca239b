"""Python binding of the routed experts (include/moe_experts.h), with the same entry-point
names: the router's choices sorted by expert, rows moved into that order and back, rows
quantised to e4m3 and the block-scaled 8-bit products.

Argument marshalling only, as in ``api``: tensors are checked (device, dtype, contiguity,
shape; ValueError) and their device pointers handed to the library, which runs on the
tensors' device and, unless ``stream`` is given (a torch stream or a handle), on torch's
current stream of that device; MlaError carries the library's code. The checks are native
(csrc/bind.cpp): the smallest of these kernels take less time than their checks took in
Python. Outputs and workspaces are the caller's; the calls can be captured into CUDA graphs.
"""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

from . import _lib
from ._lib import MlaError

SCALE_BLOCK = 128
E4M3 = torch.float8_e4m3fn

# In the order that _bind.set_entries takes.
_ENTRIES = ("mla_moe_sort", "mla_moe_gather", "mla_moe_combine", "mla_moe_combine_backward", "mla_fp8_quantize",
            "mla_fp8_matmul", "mla_fp8_grouped_matmul")
_bound = None


def _native():
    """The native marshalling module, bound to the loaded library; raises if either is missing, or if
    the module was built for another torch or Python (it reads tensors by their layout)."""
    global _bound
    if _bound is None:
        lib = _lib.lib()
        fix = "build it with `python -m sparse_mla_decode_front_b200.build`"
        try:
            from . import _bind
        except ImportError as e:
            raise ImportError(f"_bind.so is missing or cannot be loaded: {fix}") from e
        built_for = getattr(_bind, "built_for", "an unknown torch")
        if built_for != _lib.bind_tag():
            raise ImportError(f"_bind.so was built for {built_for}, this is {_lib.bind_tag()}: {fix}")
        _bind.set_entries(*[ctypes.cast(getattr(lib, n), ctypes.c_void_p).value for n in _ENTRIES])
        _bound = _bind
    return _bound


def scale_blocks(width: int) -> int:
    """Blocks of 128 elements in a row of ``width``."""
    return -(-int(width) // SCALE_BLOCK)


def mla_moe_sort_workspace_bytes(n_tokens: int, top_k: int, n_experts: int) -> int:
    return int(_lib.lib().mla_moe_sort_workspace_bytes(int(n_tokens), int(top_k), int(n_experts)))


def mla_moe_sort(topk_idx, expert_offsets, row_of, source_of, workspace=None, first_expert: int = 0,
                 affinities: Optional[torch.Tensor] = None, weights: Optional[torch.Tensor] = None,
                 normalize: bool = False, scale: float = 1.0, stream=None) -> None:
    """Sort the choices ``topk_idx`` [T, K] int32 by expert: ``expert_offsets`` [E + 1],
    ``row_of`` [T, K] and ``source_of`` [T * K] (int32) are written for the E experts from
    ``first_expert`` on. With ``affinities`` [T, E_total] bf16, ``weights`` [T, K] fp32 takes
    each choice's routing weight (``normalize``: divided by the token's sum; times ``scale``).
    ``workspace``: uint8, at least mla_moe_sort_workspace_bytes(T, K, E); None where that is 0."""
    rc = (_bound or _native()).moe_sort(topk_idx, expert_offsets, row_of, source_of, workspace, first_expert, affinities,
                                        weights, normalize, scale, stream)
    if rc:
        raise MlaError(rc, "mla_moe_sort")


def mla_moe_gather(x, row_of, rows, scales: Optional[torch.Tensor] = None, stream=None) -> None:
    """``rows``[row_of[t, k]] = ``x``[t]; with ``scales`` [ceil(H / 128), R] fp32, ``rows`` [R, H]
    is e4m3. ``row_of`` names a row at most once, as ``mla_moe_sort`` writes it. Its gradient is
    ``mla_moe_combine`` without weights."""
    rc = (_bound or _native()).moe_gather(x, row_of, rows, scales, stream)
    if rc:
        raise MlaError(rc, "mla_moe_gather")


def mla_moe_combine(rows, row_of, weights: Optional[torch.Tensor], out, stream=None) -> None:
    """``out``[t] = sum over k of ``weights``[t, k] * ``rows``[row_of[t, k]] (weights None: ones),
    choices without a row left out."""
    rc = (_bound or _native()).moe_combine(rows, row_of, weights, out, stream)
    if rc:
        raise MlaError(rc, "mla_moe_combine")


def mla_moe_combine_backward(grad_out, rows, row_of, weights: Optional[torch.Tensor],
                             grad_rows: Optional[torch.Tensor], grad_weights: Optional[torch.Tensor],
                             stream=None) -> None:
    """Gradients of ``mla_moe_combine``: ``grad_rows`` [R, H] (rows of no choice are left as they
    were) and ``grad_weights`` [T, K] fp32; either may be None. ``rows`` may be None without
    ``grad_weights``. ``row_of`` names a row at most once: the gradients of a row named twice are
    not added up."""
    rc = (_bound or _native()).moe_combine_backward(grad_out, rows, row_of, weights, grad_rows, grad_weights, stream)
    if rc:
        raise MlaError(rc, "mla_moe_combine_backward")


def mla_fp8_quantize(x, q, scales, gated: bool = False, valid_rows: Optional[torch.Tensor] = None,
                     stream=None) -> None:
    """Rows of ``x`` [R, C] to e4m3 ``q`` [R, C] with ``scales`` [ceil(C / 128), R] fp32; ``gated``:
    ``x`` is [R, 2 C] = [g | u] and silu(g) * u is quantised. ``valid_rows`` (int32, one element on
    the device): only that many rows, the others are left as they were."""
    rc = (_bound or _native()).fp8_quantize(x, q, scales, gated, valid_rows, stream)
    if rc:
        raise MlaError(rc, "mla_fp8_quantize")


def mla_fp8_matmul(x, x_scales, w, w_scales, out, status: Optional[torch.Tensor] = None, stream=None) -> None:
    """``out`` [M, N] (bf16, fp16 or fp32) = x w^T of e4m3 ``x`` [M, K] with ``x_scales``
    [ceil(K / 128), M] and e4m3 ``w`` [N, K] with ``w_scales`` [ceil(N / 128), ceil(K / 128)].
    ``status``: int32, one element, into which a wait that gave up is recorded."""
    rc = (_bound or _native()).fp8_matmul(x, x_scales, w, w_scales, out, status, stream)
    if rc:
        raise MlaError(rc, "mla_fp8_matmul")


def mla_fp8_grouped_matmul(x, x_scales, w, w_scales, expert_offsets, out, status: Optional[torch.Tensor] = None,
                           stream=None) -> None:
    """``mla_fp8_matmul`` with a weight for each expert: rows [expert_offsets[e], expert_offsets[e + 1])
    of ``x`` [R, K] with ``w``[e] ([E, N, K]; ``w_scales`` [E, ceil(N / 128), ceil(K / 128)]); rows
    of no expert are left as they were."""
    rc = (_bound or _native()).fp8_grouped_matmul(x, x_scales, w, w_scales, expert_offsets, out, status, stream)
    if rc:
        raise MlaError(rc, "mla_fp8_grouped_matmul")
