"""MXFP4 blocks and products with MXFP4 weights (oracle; test use only).

Blocks of 32 values along a row share a power of two 2^(byte - 127) (E8M0, 255
stands for NaN); a value is an E2M1 code s|ee|m. The block exponent is the
layer's UE8M0 rule with E2M1's largest value: the smallest e with
2^e >= fp32(amax / 6), clamped to [-127, 127], amax = 0 giving -127. Codes are
the nearest representable value, ties to the even code. A block that holds an
infinity or a NaN has byte 255 and codes 0.
"""
from __future__ import annotations

import numpy as np

E2M1_VALUES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def blocks(K: int) -> int:
    return -(-K // 32)


def quantize(x: np.ndarray):
    """float32-representable data [rows, K] -> (codes uint8 [rows, 16 B], scales uint8 [rows, B])."""
    x = np.asarray(x, dtype=np.float64)
    rows, K = x.shape
    B = blocks(K)
    b = np.zeros((rows, B * 32))
    b[:, :K] = x
    b = b.reshape(rows, B, 32)
    amax = np.max(np.abs(b), axis=-1)
    bad = ~np.isfinite(amax)
    with np.errstate(over="ignore", under="ignore"):
        q = (np.where(bad, 0.0, amax).astype(np.float32) / np.float32(6)).astype(np.float64)
    frac, ex = np.frexp(q)
    e = np.where(frac == 0.5, ex - 1, ex)
    e = np.clip(np.where(q == 0.0, -127, e), -127, 127).astype(np.int64)
    a = np.abs(np.where(bad[..., None], 0.0, b)) * np.exp2(-e.astype(np.float64))[..., None]
    code = np.zeros(a.shape, dtype=np.uint8)
    for i in range(1, 8):                       # the boundary between two codes goes to the even one
        mid = 0.5 * (E2M1_VALUES[i - 1] + E2M1_VALUES[i])
        code += ((a > mid) | ((a == mid) & (i % 2 == 0))).astype(np.uint8)
    code |= (np.signbit(b) & ~bad[..., None]).astype(np.uint8) << 3
    code = np.where(bad[..., None], 0, code).astype(np.uint8).reshape(rows, -1, 2)
    return code[..., 0] | (code[..., 1] << 4), np.where(bad, 255, e + 127).astype(np.uint8)


def dequantize(codes: np.ndarray, scales: np.ndarray, K: int) -> np.ndarray:
    """float64 values [..., K]."""
    c = np.stack([codes & 15, codes >> 4], axis=-1).reshape(*codes.shape[:-1], -1)
    v = E2M1_VALUES[c & 7] * np.where(c & 8, -1.0, 1.0)
    s = np.where(scales == 255, np.nan, np.exp2(scales.astype(np.float64) - 127))
    return (v * np.repeat(s, 32, axis=-1))[..., :K]


def product(xq, W, gated: bool):
    """Rows xq [R, K] times W [N or 2N, K]; returns y and the sum of the products' magnitudes [R, rows of W]."""
    y = xq @ W.T
    mag = np.abs(xq) @ np.abs(W).T
    if gated:
        n = W.shape[0] // 2
        g = y[:, :n]
        return g / (1 + np.exp(-g)) * y[:, n:], mag
    return y, mag


def expert_rows(xq, W, ids, topk: int, per_route: bool, gated: bool):
    """Rows [T * topk, N] in route order for xq (a row a token or a route), W [E, R, K]."""
    flat = np.asarray(ids).reshape(-1)
    E, R = W.shape[0], W.shape[1]
    N = R // 2 if gated else R
    out = np.zeros((flat.size, N))
    mag = np.zeros((flat.size, R))
    for r, e in enumerate(flat):
        if 0 <= e < E:
            row = xq[r if per_route else r // topk][None]
            y, m = product(row, W[e], gated)
            out[r], mag[r] = y[0], m[0]
    return out, mag
