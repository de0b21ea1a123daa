"""CPU oracle of the 8-bit and windowed single operations, in numpy fp64.

TEST INFRASTRUCTURE, as lens_oracle.py: the plain restatement of what
lens_op_quantize_f8, lens_op_gemm_f8, lens_op_sandwich_norm and
lens_op_attention_window compute, sharing no code with the library.
"""
from __future__ import annotations

from typing import Optional, Sequence

import numpy as np

GROUP = 128
F64 = np.float64
F32 = np.float32
AMAX_FLOOR = F32(2.0 ** -116)


def e4m3_table() -> np.ndarray:
    """The value of each of the 256 codes: sign, 4 exponent bits (bias 7), 3 mantissa bits;
    exponent 0 is subnormal, 0x7F and 0xFF are NaN, there is no infinity."""
    c = np.arange(256)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    v[(c & 127) == 127] = np.nan
    return np.where(c & 128, -v, v)


def e4m3_encode(x) -> np.ndarray:
    """Code of the nearest e4m3 value, ties to the even code, saturating at 448."""
    x = np.asarray(x, F64)
    pos = e4m3_table()[:127]
    mid = (pos[:-1] + pos[1:]) / 2
    a = np.where(np.isnan(x), 0.0, np.abs(x))
    i = np.searchsorted(mid, a, side="left")           # a tie stays at the lower code
    tie = (i < 126) & (a == mid[np.minimum(i, 125)])
    i = i + (tie & (i % 2 == 1))
    return np.where(np.isnan(x), 127, i + 128 * np.signbit(x)).astype(np.uint8)


def e4m3_decode(codes) -> np.ndarray:
    return e4m3_table()[np.asarray(codes, np.uint8)]


def quantize_f8(x: np.ndarray, block_rows: int):
    """(codes [rows, k], fp32 scales [k blocks, row blocks]); the three fp32 roundings of the
    definition (scale, inverse, product) are taken as it states them."""
    x = np.asarray(x, F32)
    rows, k = x.shape
    kb, rb = -(-k // GROUP), -(-rows // block_rows)
    codes, scales = np.zeros((rows, k), np.uint8), np.zeros((kb, rb), F32)
    for g in range(kb):
        for r in range(rb):
            blk = x[r * block_rows:(r + 1) * block_rows, g * GROUP:(g + 1) * GROUP]
            amax = np.maximum(np.max(np.abs(blk)), AMAX_FLOOR)       # keeps NaN
            with np.errstate(invalid="ignore", over="ignore"):
                scales[g, r] = F32(amax) / F32(448)
                codes[r * block_rows:(r + 1) * block_rows, g * GROUP:(g + 1) * GROUP] = \
                    e4m3_encode(blk * (F32(448) / F32(amax)))
    return codes, scales


def widen_f8(codes: np.ndarray, scales: np.ndarray, block_rows: int) -> np.ndarray:
    """The values that codes and scales stand for."""
    s = np.repeat(np.repeat(np.asarray(scales, F64).T, block_rows, 0), GROUP, 1)
    return e4m3_decode(codes) * s[:codes.shape[0], :codes.shape[1]]


def sandwich_norm(h, y, residual_scale: float, eps: float, post_gain=None, gate=None, pre_gain=None, shift=None,
                  scale=None):
    """(h_out, out): h_out = residual_scale h + gate post_gain y / rms(y), out = (1 + scale)
    pre_gain h_out / rms(h_out) + shift; the vectors broadcast against the rows."""
    def rms(x):
        return np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps)

    def opt(v, other):
        return other if v is None else np.asarray(v, F64)

    h, y = np.asarray(h, F64), np.asarray(y, F64)
    h = residual_scale * h + opt(gate, 1.0) * opt(post_gain, 1.0) * y / rms(y)
    return h, (1 + opt(scale, 0.0)) * opt(pre_gain, 1.0) * h / rms(h) + opt(shift, 0.0)


def window_mask(n_q: int, n_kv: int, start: int, length: int, left: int, right: int, sinks: int) -> np.ndarray:
    """[n_q, n_kv]: query i at position start + i attends key j."""
    m = np.zeros((n_q, n_kv), bool)
    for i in range(n_q):
        p = start + i
        for j in range(min(length, n_kv)):
            m[i, j] = (right < 0 or j <= p + right) and (left < 0 or j >= p - left or j < sinks)
    return m


def window_attention(q, k, v, scale: float, mask: np.ndarray):
    """(out, weight of |v|) of one head: softmax over the attended keys, zeros where there are
    none; the second result is sum_j p_j |v_j|, which bounds the effect of rounding p."""
    q, k, v = (np.asarray(a, F64) for a in (q, k, v))
    out, mag = np.zeros((q.shape[0], v.shape[1])), np.zeros((q.shape[0], v.shape[1]))
    for i in range(q.shape[0]):
        j = np.nonzero(mask[i])[0]
        if j.size == 0:
            continue
        s = k[j] @ q[i] * scale
        e = np.exp(s - s.max())
        e /= e.sum()
        out[i], mag[i] = e @ v[j], e @ np.abs(v[j])
    return out, mag
