"""fp64 CPU oracle of the e4m3 layers with block scales and of the expert layout of tokens.

TEST INFRASTRUCTURE ONLY -- see ``oracle/__init__.py``.  Written from the definitions:

* e4m3: value = +-(1 + f / 8) 2^(e - 7) for e = 1..15 (e = 15, f = 7 is NaN), +-(f / 8) 2^-6 for
  e = 0; largest finite value 448; rounding to nearest, ties to even, saturating.
* a block's scale is fp32(a / 448) for its absolute maximum a, a code the e4m3 value next to
  fp32(x fp32(448 / a)); each of the three is formed in fp64 and rounded once (a quotient or a
  product of fp32 numbers rounded through fp64 equals the one rounded directly: fp64 has more than
  2 * 24 + 2 bits).  a == 0: scale 0, codes 0; 0 < a < 2^-100 counts as 2^-100.
* the product, the sort, the weighted sum and its gradient as their formulas say, in loops.
"""

from __future__ import annotations

import numpy as np

__all__ = ["e4m3_decode", "e4m3_round", "fp8_quantize", "fp8_dequantize", "fp8_product", "fp8_expert_product",
           "expert_sort", "expert_combine", "expert_combine_backward"]


def _f32(x) -> np.ndarray:
    with np.errstate(over="ignore", invalid="ignore"):
        return np.asarray(x, np.float64).astype(np.float32).astype(np.float64)


def e4m3_decode(byte) -> np.ndarray:
    """Values of e4m3 bytes."""
    b = np.asarray(byte, np.uint8).astype(np.int64)
    e, f = (b >> 3) & 15, b & 7
    mag = np.where(e == 0, f / 8.0 * 2.0 ** -6, (1 + f / 8.0) * 2.0 ** (e - 7.0))
    mag = np.where((e == 15) & (f == 7), np.nan, mag)
    return np.where(b & 128, -mag, mag)


def e4m3_round(v) -> np.ndarray:
    """The e4m3 value next to v (ties to even), saturating at 448; NaN stays."""
    v = np.asarray(v, np.float64)
    m = np.abs(v)
    with np.errstate(divide="ignore", invalid="ignore"):
        e = np.floor(np.log2(np.where(np.isfinite(m) & (m > 0), m, 1.0)))
    e = np.maximum(e, -6.0)
    step = 2.0 ** (e - 3)
    r = np.where(np.isinf(m), 448.0, np.minimum(np.rint(np.where(np.isfinite(m), m, 0.0) / step) * step, 448.0))
    return np.where(np.isnan(v), np.nan, np.copysign(r, v))


def fp8_quantize(x, block_rows: int):
    """(code values [n, k], scales [ceil(n / block_rows), ceil(k / 128)]) of x [n, k]."""
    x = np.asarray(x, np.float64)
    n, k = x.shape
    codes = np.zeros((n, k))
    scales = np.zeros((-(-n // block_rows), -(-k // 128)))
    with np.errstate(invalid="ignore", divide="ignore", over="ignore"):
        for i in range(scales.shape[0]):
            for j in range(scales.shape[1]):
                at = np.s_[i * block_rows:(i + 1) * block_rows, j * 128:(j + 1) * 128]
                a = np.max(np.abs(x[at]))  # NaN if the block holds one
                if a == 0:
                    continue
                if a < 2.0 ** -100:
                    a = 2.0 ** -100
                scales[i, j] = _f32(a / 448.0)
                codes[at] = e4m3_round(_f32(x[at] * _f32(448.0 / a)))
    return codes, scales


def fp8_dequantize(codes, scales, block_rows: int) -> np.ndarray:
    n, k = codes.shape
    with np.errstate(invalid="ignore"):
        return codes * np.asarray(scales, np.float64)[np.arange(n) // block_rows][:, np.arange(k) // 128]


def fp8_product(a_codes, a_scales, w_codes, w_scales):
    """(Y, S): the product [M, N] in fp64, and the sum of its terms' magnitudes."""
    A, W = fp8_dequantize(a_codes, a_scales, 1), fp8_dequantize(w_codes, w_scales, 128)
    with np.errstate(invalid="ignore"):
        return A @ W.T, np.abs(A) @ np.abs(W).T


def fp8_expert_product(a_codes, a_scales, offsets, w_codes, w_scales, out, size):
    """Rows offsets[e] .. offsets[e + 1] - 1 of `out` and `size` (see fp8_product) for every expert."""
    for e in range(len(offsets) - 1):
        r = np.s_[offsets[e]:offsets[e + 1]]
        if offsets[e] < offsets[e + 1]:
            out[r], size[r] = fp8_product(a_codes[r], a_scales[r], w_codes[e], w_scales[e])
    return out, size


def expert_sort(ids, E: int):
    """(offsets, order of the rows in use, position) of choices ids [T, top]."""
    ids = np.asarray(ids)
    order, offsets = [], [0]
    for e in range(E):
        order += [i for i, x in enumerate(ids.reshape(-1)) if x == e]
        offsets.append(len(order))
    position = np.full(ids.size, -1, np.int64)
    position[order] = np.arange(len(order))
    return np.array(offsets), np.array(order, np.int64), position.reshape(ids.shape)


def expert_combine(rows, position, weights):
    """Y [T, K]: each token's rows, weighted (all ones for None) and summed."""
    T, top = position.shape
    Y = np.zeros((T, rows.shape[1]))
    for t in range(T):
        for j in range(top):
            if position[t, j] >= 0:
                Y[t] += (1.0 if weights is None else float(weights[t, j])) * rows[position[t, j]]
    return Y


def expert_combine_backward(dY, rows, position, weights, d_rows):
    """(d_rows, d_weights): `d_rows` with the named rows' gradients put in, and the weights'."""
    T, top = position.shape
    d_weights = np.zeros((T, top))
    for t in range(T):
        for j in range(top):
            if position[t, j] >= 0:
                d_rows[position[t, j]] = float(weights[t, j]) * dY[t]
                d_weights[t, j] = np.dot(dY[t], rows[position[t, j]])
    return d_rows, d_weights
