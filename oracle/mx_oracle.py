"""CPU oracle of the narrow-format (MX) operators: quantisation, its inverse,
the norm with a residual, grouped products and the experts on MX operands.

The formats are those of the OCP Microscaling specification (MXFP8 with E4M3
elements, MXFP4 with E2M1 elements, 32-element blocks, UE8M0 scales); the
choice of a block's power (no element saturates) and the treatment of
non-finite blocks are the library's own (include/routed_moe.h).  Plain NumPy,
float64; every value is looked up on the format's grid, written out from its
definition.
"""

from __future__ import annotations

import numpy as np

from .moe_oracle import bf16_round, fp8_e4m3_decode, rmsnorm, ue8m0_decode, _silu

MX_BLOCK = 32

# magnitudes of the codes without a sign, in order
_E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def mx_grid(fmt: str) -> np.ndarray:
    """The nonnegative elements by code."""
    return fp8_e4m3_decode(np.arange(127)) if fmt == "mxfp8" else _E2M1


def mx_round(v: np.ndarray, fmt: str) -> np.ndarray:
    """Codes (sign and magnitude) of values within the format's range: the
    nearest element, the even code on a tie."""
    grid = mx_grid(fmt)
    a = np.abs(v)
    hi = np.clip(np.searchsorted(grid, a), 1, len(grid) - 1)
    down, up = a - grid[hi - 1], grid[hi] - a
    low = (down < up) | ((down == up) & (hi % 2 == 1))
    mag = np.where(low, hi - 1, hi)
    return (mag + np.where(np.signbit(v), 128 if fmt == "mxfp8" else 8, 0)).astype(np.uint8)


def mx_power(amax: float, fmt: str) -> int:
    """Smallest p >= -127 with amax <= largest * 2^p."""
    top = mx_grid(fmt)[-1]
    p = -127 if amax == 0 else max(-127, int(np.floor(np.log2(amax / top))) - 1)
    while top * 2.0 ** p < amax:
        p += 1
    return p


def mx_quantize(x: np.ndarray, fmt: str):
    """x [rows, K] -> (elements' codes uint8 [rows, K], scale bytes uint8 [rows, K/32])."""
    rows, K = x.shape
    codes = np.zeros((rows, K), np.uint8)
    scales = np.zeros((rows, K // MX_BLOCK), np.uint8)
    for r in range(rows):
        for b in range(K // MX_BLOCK):
            blk = x[r, b * MX_BLOCK:(b + 1) * MX_BLOCK].astype(np.float64)
            if not np.all(np.isfinite(blk)):
                scales[r, b] = 255
                continue
            p = mx_power(np.max(np.abs(blk)), fmt)
            scales[r, b] = p + 127
            codes[r, b * MX_BLOCK:(b + 1) * MX_BLOCK] = mx_round(blk / 2.0 ** p, fmt)
    return codes, scales


def mx_values(codes: np.ndarray, scales: np.ndarray, fmt: str) -> np.ndarray:
    """float64 values of element codes [..., K] and scale bytes [..., K/32]."""
    if fmt == "mxfp8":
        v = fp8_e4m3_decode(codes)
    else:
        c = codes.astype(np.int64)
        v = np.where(c >= 8, -_E2M1[c & 7], _E2M1[c & 7])
    return v * np.repeat(ue8m0_decode(scales), MX_BLOCK, axis=-1)


def mx_store(codes: np.ndarray, scales: np.ndarray, fmt: str):
    """The library's arrays: codes (two E2M1 to a byte, the even element low) and
    scales [ceil(K/128), rows, 4] of one matrix."""
    if fmt == "mxfp4":
        codes = (codes[:, 0::2] | (codes[:, 1::2] << 4)).astype(np.uint8)
    rows, blocks = scales.shape
    words = -(-blocks // 4)
    out = np.zeros((words, rows, 4), np.uint8)
    for b in range(blocks):
        out[b // 4, :, b % 4] = scales[:, b]
    return codes, out


def mx_load(codes: np.ndarray, stored: np.ndarray, K: int, fmt: str):
    """The inverse of mx_store: element codes [rows, K] and scale bytes [rows, K/32]."""
    if fmt == "mxfp4":
        wide = np.zeros((codes.shape[0], K), np.uint8)
        wide[:, 0::2], wide[:, 1::2] = codes & 15, codes >> 4
        codes = wide
    scales = np.stack([stored[b // 4, :, b % 4] for b in range(K // MX_BLOCK)], axis=1)
    return codes, scales


def add_rmsnorm(x: np.ndarray, residual, eps: float = 1e-6, gamma=None):
    """(sum, xn): the bf16 sum, and its RMSNorm in float64 (not rounded)."""
    s = x if residual is None else bf16_round(x.astype(np.float64) + residual.astype(np.float64))
    return s, rmsnorm(s, eps, gamma)


def grouped_mm(x: np.ndarray, w, offsets) -> np.ndarray:
    """x [R,K], w [E,N,K], offsets [E+1] -> float64 [R,N]; NaN outside the groups."""
    out = np.full((x.shape[0], w.shape[1]), np.nan)
    for e in range(len(offsets) - 1):
        lo, hi = offsets[e], offsets[e + 1]
        out[lo:hi] = x[lo:hi].astype(np.float64) @ w[e].astype(np.float64).T
    return out


def swiglu(gate_up: np.ndarray) -> np.ndarray:
    """silu(gate) * up of [R, 2I]: gate columns, then up columns."""
    I = gate_up.shape[1] // 2
    return _silu(gate_up[:, :I]) * gate_up[:, I:]
