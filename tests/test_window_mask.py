"""The mask that the GPU tests of windowed attention build, against the oracle's.  CPU only."""
import numpy as np

from oracle import ops_oracle as oo
from tests.test_gpu_window import mask_of


def test_the_gpu_tests_mask_is_the_oracles():
    rng = np.random.default_rng(5)
    for _ in range(500):
        n_q, n_kv, start = int(rng.integers(1, 9)), int(rng.integers(1, 14)), int(rng.integers(0, 12))
        length, left, right = int(rng.integers(0, n_kv + 1)), int(rng.integers(-1, 9)), int(rng.integers(-1, 9))
        sinks = int(rng.integers(0, 16))
        assert np.array_equal(mask_of(n_q, n_kv, start, length, left, right, sinks, device="cpu").numpy(),
                              oo.window_mask(n_q, n_kv, start, length, left, right, sinks))
