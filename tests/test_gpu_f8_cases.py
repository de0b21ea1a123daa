"""GPU tests of the 8-bit product beside test_gpu_f8.py: every kernel that a size selects (which one,
test_f8_choice.py checks) at its edges, with every code, scales at the ends of their range, zero and
non-finite ones, on streams and in graphs."""
import numpy as np
import pytest

from tests import f8_sizes
from tests.helpers import dev

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import flow_matching_mmdit_b200 as L  # noqa: E402
from tests.test_gpu_f8 import _operands, _widen, check_gemm, gemm, guarded, quantize  # noqa: E402

KERNELS = list(f8_sizes.KERNELS.values())


@pytest.fixture(scope="module", autouse=True)
def cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    L.load_library()


@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("M,N,K", f8_sizes.SIZES)
def test_every_kernel_at_its_edges(M, N, K, bf16, bias):
    a, w, b = _operands(M, N, K, M + N + K)
    (ca, sa), (cw, sw) = quantize(a, 1), quantize(w, 128)
    b = dev(b) if bias else None
    check_gemm(gemm(ca, sa, cw, sw, b, M, N, K, bf16), ca, sa, cw, sw, b, K, bf16)


@pytest.mark.parametrize("M,N,K", KERNELS)
def test_every_code_and_wide_scales(M, N, K):
    rng = np.random.default_rng(M)
    groups = -(-K // 128)
    finite = np.array([c for c in range(256) if c & 127 != 127], np.uint8)
    ca, cw = dev(rng.choice(finite, (M, K))), dev(rng.choice(finite, (N, K)))
    sa, sw = dev(scales(rng, (groups, M), -15, 15)), dev(scales(rng, (groups, -(-N // 128)), -15, 15))
    check_gemm(gemm(ca, sa, cw, sw, None, M, N, K, False), ca, sa, cw, sw, None, K, False)


@pytest.mark.parametrize("M,N,K", KERNELS)
def test_non_finite_codes_stay_in_their_row_or_column(M, N, K):
    a, w, _ = _operands(M, N, K, 7)
    (ca, sa), (cw, sw) = quantize(a, 1), quantize(w, 128)
    want = gemm(ca, sa, cw, sw, None, M, N, K, False).clone()
    row, col = M - 2, N - 3
    ca[row, K - 1], cw[col, 5] = 0x7F, 0xFF
    c = gemm(ca, sa, cw, sw, None, M, N, K, False)
    assert bool(torch.isnan(c[row]).all()) and bool(torch.isnan(c[:, col]).all())
    keep_m, keep_n = [i for i in range(M) if i != row], [i for i in range(N) if i != col]
    assert torch.equal(c[keep_m][:, keep_n], want[keep_m][:, keep_n])


@pytest.mark.parametrize("M,N,K", KERNELS)
def test_the_same_bits_from_streams_and_graphs(M, N, K):
    a, w, bias = _operands(M, N, K, 3)
    (ca, sa), (cw, sw), b = quantize(a, 1), quantize(w, 128), dev(bias)
    want = gemm(ca, sa, cw, sw, b, M, N, K, False).clone()
    outs = [guarded((M, N), torch.float32, -7.0) for _ in range(5)]
    torch.cuda.synchronize()                        # the fills come before the streams' work
    streams = [torch.cuda.Stream() for _ in range(2)]
    for i, (o, _) in enumerate(outs[:4]):
        L.lens_op_gemm_f8(ca, sa, cw, sw, b, o, L.LENS_F32, M, N, K, stream=streams[i % 2])
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        L.lens_op_gemm_f8(ca, sa, cw, sw, b, outs[4][0], L.LENS_F32, M, N, K)
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    for o, intact in outs:
        assert torch.equal(o, want)
        intact()


def scales(rng, shape, lo, hi):
    return np.exp2(rng.uniform(lo, hi, shape)).astype(np.float32)


def check(c, ca, sa, cw, sw, K):
    """As test_gpu_f8.check_gemm: (128 + K / 128 + 4) roundings of 2^-23 of the magnitudes, and one of
    2^-149 for each block, the scales' product and the output where they are subnormal."""
    A, W = _widen(ca, sa, 1), _widen(cw, sw, 128)
    ref, mag = A @ W.t(), A.abs() @ W.abs().t()
    assert bool((mag < 2.0 ** 128).all())
    tol = (128 + K / 128 + 4) * 2.0 ** -23 * mag + (K // 128 + 2) * 2.0 ** -149
    err = (c.double() - ref).abs()
    assert bool((err <= tol).all()), float((err / tol).max())


@pytest.mark.parametrize("M,N,K", KERNELS)
def test_products_of_scales_down_to_the_smallest_normal_number(M, N, K):
    """Scales of 2^-63 to 2^-55 on both sides, beside rows with larger ones."""
    rng = np.random.default_rng(M)
    groups = -(-K // 128)
    finite = np.array([c for c in range(256) if c & 127 != 127], np.uint8)
    ca, cw = dev(rng.choice(finite, (M, K))), dev(rng.choice(finite, (N, K)))
    a = scales(rng, (groups, M), -63, -55)
    a[:, ::3] = scales(rng, a[:, ::3].shape, -30, 20)
    sa, sw = dev(a), dev(scales(rng, (groups, -(-N // 128)), -63, -55))
    c = gemm(ca, sa, cw, sw, None, M, N, K, False)
    check(c, ca, sa, cw, sw, K)
    assert bool((c != 0).any(1).all())


@pytest.mark.parametrize("M,N,K", KERNELS)
def test_products_of_scales_up_to_the_largest_number(M, N, K):
    """Scales whose product comes near 2^128 on blocks that sum to little, or to zero."""
    rng = np.random.default_rng(M + 1)
    groups = -(-K // 128)
    small = np.array([0, 1, 2, 3, 0x81, 0x82, 0x83], np.uint8)         # up to 3 * 2^-9: sums below 2^-7
    a, w = rng.choice(small, (M, K)), rng.choice(small, (N, K))
    a[1], w[5] = 0, 0                                                   # a row and a column of zeros
    ca, cw = dev(a), dev(w)
    s = scales(rng, (groups, M), 58, 63.9)
    s[:, ::3] = scales(rng, s[:, ::3].shape, -20, 20)
    sa, sw = dev(s), dev(scales(rng, (groups, -(-N // 128)), 58, 63.9))
    c = gemm(ca, sa, cw, sw, None, M, N, K, False)
    check(c, ca, sa, cw, sw, K)
    assert not bool(c[1].any()) and not bool(c[:, 5].any())


@pytest.mark.parametrize("M,N,K", KERNELS)
def test_zero_and_non_finite_scales_act_as_written(M, N, K):
    """A zero scale takes its block out, an infinite or NaN one makes its row non-finite."""
    rng = np.random.default_rng(M + 2)
    groups = -(-K // 128)
    ca = dev(rng.choice(np.array([0x30, 0x38, 0x40], np.uint8), (M, K)))
    cw = dev(rng.choice(np.array([0x30, 0x38, 0x40], np.uint8), (N, K)))
    s = scales(rng, (groups, M), -5, 5)
    s[0, ::2] = 0
    sa, sw = dev(s), dev(scales(rng, (groups, -(-N // 128)), -5, 5))
    check(gemm(ca, sa, cw, sw, None, M, N, K, False), ca, sa, cw, sw, K)
    sa[groups - 1, 1], sa[0, 2 % M] = float("inf"), float("nan")
    c = gemm(ca, sa, cw, sw, None, M, N, K, False)
    assert bool((c[1] == float("inf")).all()) and bool(torch.isnan(c[2 % M]).all())
    keep = [i for i in range(M) if i not in (1, 2 % M)]
    assert bool(torch.isfinite(c[keep]).all())
