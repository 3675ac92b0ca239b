"""Python binding of the routed experts (include/moe_experts.h), with the same entry-point
names: the router's choices sorted by expert, rows moved into that order and back, rows
quantised to e4m3 and the block-scaled 8-bit products.

Argument marshalling only, as in ``api``: tensors are checked (device, dtype, contiguity,
shape) and their device pointers handed to the library, which runs on the tensors' device
and, unless ``stream`` is given, on torch's current stream of that device. Outputs and
workspaces are the caller's; the calls can be captured into CUDA graphs.
"""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

from . import _lib
from ._lib import MlaError

SCALE_BLOCK = 128
DTYPES = {torch.bfloat16: _lib.MLA_DTYPE_BF16, torch.float16: _lib.MLA_DTYPE_FP16,
          torch.float32: _lib.MLA_DTYPE_FP32}
E4M3 = torch.float8_e4m3fn
_MAX_DIM = 2 ** 31 - 1
_lib_of = _lib.lib
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)   # absent from a CPU-only torch
_get_device = getattr(torch._C, "_cuda_getDevice", None)


def scale_blocks(width: int) -> int:
    """Blocks of 128 elements in a row of ``width``."""
    return -(-int(width) // SCALE_BLOCK)


def _bad(name, t, dtype, shape, dev):
    """The reason why ``t`` is refused."""
    if not isinstance(t, torch.Tensor):
        return ValueError(f"{name} is {'None' if t is None else type(t).__name__}, expected a tensor")
    if not t.is_cuda:
        return ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        return ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        return ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.get_device() != dev:
        return ValueError(f"{name} is on {t.device}, expected cuda:{dev}")
    return ValueError(f"{name} must be contiguous")


def _ptr(name, t, dtype, shape, dev) -> int:
    """``t``'s address after its checks. A decode loop makes these calls by the thousand: the
    checks are the cheapest that see everything, and the reason is looked for only on refusal."""
    try:
        if t.dtype is dtype and t.shape == shape and t.get_device() == dev and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    raise _bad(name, t, dtype, shape, dev)


def _shape(name, t, dims):
    """Shape of a tensor that gives a call some of its sizes (its other checks are _ptr's)."""
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} is {'None' if t is None else type(t).__name__}, expected a tensor")
    shape = t.shape
    if len(shape) != dims:
        raise ValueError(f"{name} must have {dims} dimensions, got shape {tuple(shape)}")
    if shape[0] > _MAX_DIM or shape[-1] > _MAX_DIM:
        raise ValueError(f"{name} has shape {tuple(shape)}: a dimension is beyond the library's 32-bit sizes")
    return shape


def _first(name, t, dims):
    """(device index, shape) of the tensor that decides a call's device."""
    shape = _shape(name, t, dims)
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    return dev, shape


def _dtype_code(name, t) -> int:
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} is {'None' if t is None else type(t).__name__}, expected a tensor")
    code = DTYPES.get(t.dtype)
    if code is None:
        raise ValueError(f"{name} must be bfloat16, float16 or float32, got {t.dtype}")
    return code


def _call(name, fn, dev, stream, *args) -> None:
    """Run entry point ``fn`` on device ``dev``; ``stream``: None, a torch stream or a handle."""
    if stream is None:
        stream = _raw_stream(dev)
    elif hasattr(stream, "cuda_stream"):
        stream = stream.cuda_stream
    if _get_device() == dev:
        rc = fn(*args, stream)
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, stream)
    if rc != 0:
        raise MlaError(rc, name)


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
    dev, tk = _first("topk_idx", topk_idx, 2)
    T, K = tk
    E, i32 = _shape("expert_offsets", expert_offsets, 1)[0] - 1, torch.int32
    aff = w = ws = None
    total = ws_bytes = 0
    if (affinities is None) != (weights is None):
        raise ValueError("affinities and weights come together")
    if affinities is not None:
        total = _shape("affinities", affinities, 2)[1]
        aff = _ptr("affinities", affinities, torch.bfloat16, (T, total), dev)
        w = _ptr("weights", weights, torch.float32, tk, dev)
    if workspace is not None:
        ws_bytes = _shape("workspace", workspace, 1)[0]
        ws = _ptr("workspace", workspace, torch.uint8, (ws_bytes,), dev)
    _call("mla_moe_sort", _lib_of().mla_moe_sort, dev, stream, _ptr("topk_idx", topk_idx, i32, tk, dev), aff, T, K, total,
          int(first_expert), E, 1 if normalize else 0, float(scale),
          _ptr("expert_offsets", expert_offsets, i32, (E + 1,), dev), _ptr("row_of", row_of, i32, tk, dev),
          _ptr("source_of", source_of, i32, (T * K,), dev), w, ws, ws_bytes)


def mla_moe_gather(x, row_of, rows, scales: Optional[torch.Tensor] = None, stream=None) -> None:
    """``rows``[row_of[t, k]] = ``x``[t]; with ``scales`` [ceil(H / 128), R] fp32, ``rows`` [R, H]
    is e4m3. Its gradient is ``mla_moe_combine`` without weights."""
    dev, th = _first("x", x, 2)
    (T, H), code = th, _dtype_code("x", x)
    K, R = _shape("row_of", row_of, 2)[1], _shape("rows", rows, 2)[0]
    sc = None if scales is None else _ptr("scales", scales, torch.float32, (scale_blocks(H), R), dev)
    _call("mla_moe_gather", _lib_of().mla_moe_gather, dev, stream, _ptr("x", x, x.dtype, th, dev), code,
          _ptr("row_of", row_of, torch.int32, (T, K), dev), T, K, H, R,
          _ptr("rows", rows, x.dtype if scales is None else E4M3, (R, H), dev), sc)


def mla_moe_combine(rows, row_of, weights: Optional[torch.Tensor], out, stream=None) -> None:
    """``out``[t] = sum over k of ``weights``[t, k] * ``rows``[row_of[t, k]] (weights None: ones),
    choices without a row left out."""
    dev, rh = _first("rows", rows, 2)
    (R, H), code = rh, _dtype_code("rows", rows)
    tk = _shape("row_of", row_of, 2)
    T, K = tk
    w = None if weights is None else _ptr("weights", weights, torch.float32, tk, dev)
    _call("mla_moe_combine", _lib_of().mla_moe_combine, dev, stream, _ptr("rows", rows, rows.dtype, rh, dev), code,
          _ptr("row_of", row_of, torch.int32, tk, dev), w, T, K, H, R,
          _ptr("out", out, rows.dtype, (T, H), dev))


def mla_moe_combine_backward(grad_out, rows, row_of, weights: Optional[torch.Tensor],
                             grad_rows: Optional[torch.Tensor], grad_weights: Optional[torch.Tensor],
                             stream=None) -> None:
    """Gradients of ``mla_moe_combine``: ``grad_rows`` [R, H] (rows of no choice are left as they
    were) and ``grad_weights`` [T, K] fp32; either may be None. ``rows`` may be None without
    ``grad_weights``."""
    dev, th = _first("grad_out", grad_out, 2)
    (T, H), code = th, _dtype_code("grad_out", grad_out)
    if grad_rows is None and grad_weights is None:
        raise ValueError("grad_rows and grad_weights are both None")
    if rows is None and grad_weights is not None:
        raise ValueError("grad_weights needs rows")
    held = rows if rows is not None else grad_rows
    K, R = _shape("row_of", row_of, 2)[1], _shape("rows" if rows is not None else "grad_rows", held, 2)[0]
    opt = lambda name, t, dtype, shape: None if t is None else _ptr(name, t, dtype, shape, dev)
    _call("mla_moe_combine_backward", _lib_of().mla_moe_combine_backward, dev, stream,
          _ptr("grad_out", grad_out, grad_out.dtype, th, dev), opt("rows", rows, grad_out.dtype, (R, H)), code,
          _ptr("row_of", row_of, torch.int32, (T, K), dev),
          opt("weights", weights, torch.float32, (T, K)), T, K, H, R,
          opt("grad_rows", grad_rows, grad_out.dtype, (R, H)), opt("grad_weights", grad_weights, torch.float32, (T, K)))


def mla_fp8_quantize(x, q, scales, gated: bool = False, valid_rows: Optional[torch.Tensor] = None,
                     stream=None) -> None:
    """Rows of ``x`` [R, C] to e4m3 ``q`` [R, C] with ``scales`` [ceil(C / 128), R] fp32; ``gated``:
    ``x`` is [R, 2 C] = [g | u] and silu(g) * u is quantised. ``valid_rows`` (int32, one element on
    the device): only that many rows, the others are left as they were."""
    code = _dtype_code("x", x)
    dev, rc = _first("q", q, 2)
    R, C = rc
    valid = None if valid_rows is None else _ptr("valid_rows", valid_rows, torch.int32, (1,), dev)
    _call("mla_fp8_quantize", _lib_of().mla_fp8_quantize, dev, stream,
          _ptr("x", x, x.dtype, (R, 2 * C) if gated else rc, dev), code, R, C, 1 if gated else 0, valid,
          _ptr("q", q, E4M3, rc, dev), _ptr("scales", scales, torch.float32, (-(-C // SCALE_BLOCK), R), dev))


def mla_fp8_matmul(x, x_scales, w, w_scales, out, status: Optional[torch.Tensor] = None, stream=None) -> None:
    """``out`` [M, N] (bf16, fp16 or fp32) = x w^T of e4m3 ``x`` [M, K] with ``x_scales``
    [ceil(K / 128), M] and e4m3 ``w`` [N, K] with ``w_scales`` [ceil(N / 128), ceil(K / 128)].
    ``status``: int32, one element, into which a wait that gave up is recorded."""
    dev, mk = _first("x", x, 2)
    (M, K), N, code = mk, _shape("w", w, 2)[0], _dtype_code("out", out)
    kb = -(-K // SCALE_BLOCK)
    st = None if status is None else _ptr("status", status, torch.int32, (1,), dev)
    _call("mla_fp8_matmul", _lib_of().mla_fp8_matmul, dev, stream, _ptr("x", x, E4M3, mk, dev),
          _ptr("x_scales", x_scales, torch.float32, (kb, M), dev), _ptr("w", w, E4M3, (N, K), dev),
          _ptr("w_scales", w_scales, torch.float32, (-(-N // SCALE_BLOCK), kb), dev), M, N, K,
          _ptr("out", out, out.dtype, (M, N), dev), code, st)


def mla_fp8_grouped_matmul(x, x_scales, w, w_scales, expert_offsets, out, status: Optional[torch.Tensor] = None,
                           stream=None) -> None:
    """``mla_fp8_matmul`` with a weight for each expert: rows [expert_offsets[e], expert_offsets[e + 1])
    of ``x`` [R, K] with ``w``[e] ([E, N, K]; ``w_scales`` [E, ceil(N / 128), ceil(K / 128)]); rows
    of no expert are left as they were."""
    dev, mk = _first("x", x, 2)
    (M, K), (E, N, _), code = mk, _shape("w", w, 3), _dtype_code("out", out)
    kb = -(-K // SCALE_BLOCK)
    st = None if status is None else _ptr("status", status, torch.int32, (1,), dev)
    _call("mla_fp8_grouped_matmul", _lib_of().mla_fp8_grouped_matmul, dev, stream, _ptr("x", x, E4M3, mk, dev),
          _ptr("x_scales", x_scales, torch.float32, (kb, M), dev), _ptr("w", w, E4M3, (E, N, K), dev),
          _ptr("w_scales", w_scales, torch.float32, (E, -(-N // SCALE_BLOCK), kb), dev),
          _ptr("expert_offsets", expert_offsets, torch.int32, (E + 1,), dev), M, E, N, K,
          _ptr("out", out, out.dtype, (M, N), dev), code, st)
