"""GPU tests of windowed attention beside test_gpu_window.py: caches longer than what they hold."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import flow_matching_mmdit_b200 as L  # noqa: E402
from tests.test_gpu_window import check, make, run  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    L.load_library()


@pytest.mark.parametrize("n_q", [1, 4])
def test_a_row_does_not_depend_on_the_capacity_of_the_cache(n_q):
    """The same keys in a cache sixteen times as long: their split goes by the lengths in use."""
    B, H, Hk, held, capacity = 32, 8, 8, 1028, 16448
    q, k, v = make(B, H, Hk, n_q, held, 21)
    length = [held - 7 * (b % 5) for b in range(B)]
    start = [n - n_q for n in length]
    want = run(q, k, v, start, length, -1, 0, 0)
    check(want, q, k, v, start, length, -1, 0, 0, heads=[0, 7])
    big = torch.full((2, B, Hk, capacity, 64), float("nan"), dtype=torch.bfloat16, device="cuda")
    big[0, :, :, :held], big[1, :, :, :held] = k, v
    assert torch.equal(run(q, big[0], big[1], start, length, -1, 0, 0), want)
