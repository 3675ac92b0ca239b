"""CPU fp64 oracle of the routed experts of a MoE decoder layer (include/moe_experts.h).

TEST INFRASTRUCTURE ONLY. Nothing in the product path may import, call or
execute this module; only ``tests/`` uses it. It shares no code, tables or
constants with the CUDA path.

Every function restates the operator's definition in the header, in numpy and
fp64; 8-bit values are handled as the numbers they stand for, and the e4m3 grid
is built here from the format (1 sign bit, 4 exponent bits of bias 7, 3 mantissa
bits, no infinities). Loops over choices and experts are written out where that
is the plainest reading.
"""
from __future__ import annotations

from typing import Dict, Optional

import numpy as np

BLOCK = 128
AMAX_FLOOR = 2.0 ** -100


def e4m3_grid() -> np.ndarray:
    """The 127 non-negative finite e4m3 values, by bit pattern 0 .. 0x7e."""
    v = []
    for bits in range(0x7F):
        e, m = bits >> 3, bits & 7
        v.append(m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
    return np.array(v)


def round_e4m3(x: np.ndarray) -> np.ndarray:
    """To the nearest e4m3 value, ties to the even bit pattern, beyond the largest to it; NaN stays."""
    grid = e4m3_grid()
    a = np.minimum(np.abs(x), grid[-1])
    hi = np.clip(np.searchsorted(grid, a), 1, len(grid) - 1)
    lo = hi - 1
    up = np.where(a - grid[lo] == grid[hi] - a, hi % 2 == 0, a - grid[lo] > grid[hi] - a)
    return np.where(np.isnan(x), np.nan, np.copysign(np.where(up, grid[hi], grid[lo]), x))


def sort(idx: np.ndarray, first: int, n_experts: int) -> Dict[str, np.ndarray]:
    """expert_offsets, row_of and source_of of the choices idx [T, K]."""
    T, K = idx.shape
    lists = [[] for _ in range(n_experts)]
    for i, e in enumerate(idx.reshape(-1).tolist()):
        if 0 <= e - first < n_experts:
            lists[e - first].append(i)
    source = np.full(T * K, -1, np.int32)
    order = np.array([i for l in lists for i in l], np.int64)
    source[:len(order)] = order
    row_of = np.full(T * K, -1, np.int32)
    row_of[order] = np.arange(len(order), dtype=np.int32)
    offsets = np.concatenate([[0], np.cumsum([len(l) for l in lists])]).astype(np.int32)
    return dict(expert_offsets=offsets, row_of=row_of.reshape(T, K), source_of=source)


def routing_weights(idx: np.ndarray, affinities: np.ndarray, normalize: bool, scale: float) -> np.ndarray:
    T, K = idx.shape
    E = affinities.shape[1]
    a = np.zeros((T, K))
    for t in range(T):
        for k in range(K):
            if 0 <= idx[t, k] < E:
                a[t, k] = affinities[t, idx[t, k]]
    if normalize:
        s = a.sum(1, keepdims=True)
        a = np.where(s == 0, 0.0, a / np.where(s == 0, 1.0, s))
    return scale * a


def quantize(v: np.ndarray):
    """(values before the rounding v * 448 / amax [R, C], scales [blocks, R]); a block with a NaN
    or an infinity is NaN as a whole."""
    R, C = v.shape
    nb = -(-C // BLOCK)
    q, scales = np.empty((R, C)), np.empty((nb, R))
    for b in range(nb):
        part = v[:, b * BLOCK:(b + 1) * BLOCK]
        amax = np.maximum(np.abs(part).max(1), AMAX_FLOOR)
        scales[b] = amax / 448.0
        with np.errstate(invalid="ignore"):
            q[:, b * BLOCK:(b + 1) * BLOCK] = part * (448.0 / amax)[:, None]
    return q, scales


def gated(x: np.ndarray) -> np.ndarray:
    g, u = np.split(x, 2, axis=1)
    with np.errstate(over="ignore"):
        return g / (1.0 + np.exp(-g)) * u


def combine(rows: np.ndarray, row_of: np.ndarray, weights: Optional[np.ndarray]) -> np.ndarray:
    T, K = row_of.shape
    out = np.zeros((T, rows.shape[1]))
    for t in range(T):
        for k in range(K):
            r = row_of[t, k]
            if 0 <= r < rows.shape[0]:
                out[t] += (1.0 if weights is None else weights[t, k]) * rows[r]
    return out


def combine_backward(grad_out, rows, row_of, weights):
    """(grad_rows, NaN for a row of no choice; grad_weights)."""
    T, K = row_of.shape
    grad_rows = np.full(rows.shape, np.nan)
    grad_weights = np.zeros((T, K))
    for t in range(T):
        for k in range(K):
            r = row_of[t, k]
            if 0 <= r < rows.shape[0]:
                grad_rows[r] = (1.0 if weights is None else weights[t, k]) * grad_out[t]
                grad_weights[t, k] = grad_out[t] @ rows[r]
    return grad_rows, grad_weights


def product(x: np.ndarray, x_scales: np.ndarray, w: np.ndarray, w_scales: np.ndarray):
    """(out [M, N], the sum of the terms' magnitudes) of 8-bit values x [M, K], w [N, K]."""
    M, K = x.shape
    N = w.shape[0]
    out, mag = np.zeros((M, N)), np.zeros((M, N))
    for b in range(-(-K // BLOCK)):
        part = slice(b * BLOCK, (b + 1) * BLOCK)
        s = x_scales[b][:, None] * np.repeat(w_scales[:, b], BLOCK)[None, :N]
        out += s * (x[:, part] @ w[:, part].T)
        mag += np.abs(s) * (np.abs(x[:, part]) @ np.abs(w[:, part]).T)
    return out, mag
