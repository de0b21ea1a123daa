"""Pins of oracle/ops_oracle.py: e4m3 against torch's conversion and hand-worked values,
block scales, the norms' closed forms, and the window mask against its two key ranges."""
import numpy as np
import pytest
import torch

from oracle import ops_oracle as oo


def test_e4m3_values_and_rounding():
    t = oo.e4m3_table()
    assert t[0x38] == 1.0 and t[0x7E] == 448.0 and t[1] == 2.0 ** -9 and t[0xB8] == -1.0 and np.isnan(t[0x7F])
    # halfway cases go to the even code; 448 saturates
    assert list(oo.e4m3_encode([1.0625, 1.1875, 1e9, -1e9, 2.0 ** -10, 3 * 2.0 ** -10])) == [0x38, 0x3A, 0x7E, 0xFE, 0, 2]
    rng = np.random.default_rng(0)
    x = np.concatenate([rng.standard_normal(20000) * 10.0 ** rng.uniform(-4, 2.5, 20000), oo.e4m3_table()[:127]])
    x = np.clip(x, -448, 448).astype(np.float32)
    ref = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(oo.e4m3_encode(x), ref)


@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantize_uses_the_whole_range_of_each_block(block_rows):
    rng = np.random.default_rng(1)
    x = (rng.standard_normal((130, 272)) * np.exp(rng.standard_normal(272))).astype(np.float32)
    x[0, :128] = 0
    codes, scales = oo.quantize_f8(x, block_rows)
    assert scales.shape == (3, 130 if block_rows == 1 else 2)
    w = oo.widen_f8(codes, scales, block_rows)
    # half a step of a 3-bit mantissa, or half the subnormal step, of the block's scale
    s = np.repeat(np.repeat(scales.T.astype(np.float64), block_rows, 0), 128, 1)[:130, :272]
    assert np.all(np.abs(w - x) <= np.maximum(np.abs(x) * 2.0 ** -4, s * 2.0 ** -10) * (1 + 1e-6))
    assert np.all(oo.e4m3_decode(codes[2:]).max() == 448.0)
    if block_rows == 1:
        assert not codes[0, :128].any() and scales[0, 0] == oo.AMAX_FLOOR / np.float32(448)


def test_sandwich_norm_closed_forms():
    y = np.array([[3.0, 4.0, 0.0, 0.0]])                    # rms 2.5
    h = np.array([[1.0, 1.0, 1.0, 1.0]])
    ho, o = oo.sandwich_norm(h, y, 2.0, 0.0)
    assert np.allclose(ho, [[3.2, 3.6, 2.0, 2.0]])
    assert np.allclose(o, ho / np.sqrt(np.mean(ho ** 2)))
    ho2, o2 = oo.sandwich_norm(h, y, 0.0, 0.0, post_gain=[1, 2, 3, 4], gate=[[2.0] * 4], pre_gain=[5.0] * 4,
                               shift=[[7.0] * 4], scale=[[1.0] * 4])
    assert np.allclose(ho2, [[2.4, 6.4, 0, 0]])
    assert np.allclose(o2, 10 * ho2 / np.sqrt(np.mean(ho2 ** 2)) + 7)


def test_window_mask_is_two_ranges():
    rng = np.random.default_rng(2)
    for _ in range(200):
        n_q, n_kv, start = int(rng.integers(1, 9)), int(rng.integers(1, 14)), int(rng.integers(0, 9))
        length, left, right = int(rng.integers(0, n_kv + 1)), int(rng.integers(-1, 9)), int(rng.integers(-1, 9))
        sinks = int(rng.integers(0, 6))
        m = oo.window_mask(n_q, n_kv, start, length, left, right, sinks)
        for i in range(n_q):
            hi = length if right < 0 else min(start + i + right + 1, length)
            lo = 0 if left < 0 else max(start + i - left, 0)
            want = np.zeros(n_kv, bool)
            want[:min(sinks, lo, hi)] = True
            want[lo:max(hi, lo)] = True
            assert np.array_equal(m[i], want)


def test_window_attention_reduces_to_plain_attention():
    from oracle import lens_oracle as o
    rng = np.random.default_rng(3)
    q, k, v = (rng.standard_normal((7, 64)) for _ in range(3))
    full = oo.window_mask(7, 7, 0, 7, -1, -1, 0)
    assert full.all()
    got, _ = oo.window_attention(q, k, v, 0.125, full)
    assert np.allclose(got, o.attention(q[None, None], k[None, None], v[None, None])[0, 0])
    none, _ = oo.window_attention(q, k, v, 0.125, np.zeros((7, 7), bool))
    assert not none.any()
