"""GPU parity of the 8-bit operations against the fp64 oracle: quantization bit for bit,
the product within the rounding of its accumulation, and the two run together."""
import numpy as np
import pytest

from lens_inputs import f32_to_bf16_bits
from oracle import ops_oracle as oo
from tests.helpers import bf16_to_f64, dev, host

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import flow_matching_mmdit_b200 as L  # noqa: E402

GUARD = 64


@pytest.fixture(scope="module", autouse=True)
def cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    L.load_library()


def guarded(shape, dtype, fill):
    """A tensor of `shape` inside a larger buffer filled with `fill`, and the check that the
    elements around it were left alone."""
    n = int(np.prod(shape))
    buf = torch.full((n + 2 * GUARD,), fill, dtype=dtype, device="cuda")

    def intact():
        assert bool((buf[:GUARD] == fill).all()) and bool((buf[GUARD + n:] == fill).all())

    return buf[GUARD:GUARD + n].view(shape), intact


def quantize(x, block_rows, bf16=False):
    rows, k = x.shape
    codes, ok1 = guarded((rows, k), torch.uint8, 0x55)
    scales, ok2 = guarded((-(-k // 128), -(-rows // block_rows)), torch.float32, -7.0)
    xd = dev(f32_to_bf16_bits(x)) if bf16 else dev(x)
    L.lens_op_quantize_f8(xd, L.LENS_BF16 if bf16 else L.LENS_F32, rows, k, block_rows, codes, scales)
    torch.cuda.synchronize()
    ok1(), ok2()
    return codes, scales


def _values(rows, k, seed):
    rng = np.random.default_rng(seed)
    x = (rng.standard_normal((rows, k)) * np.exp(rng.standard_normal(k))).astype(np.float32)
    x[rows // 2, :16] = 0
    x[-1, -16:] = 1e-30
    return x


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("rows,k,block_rows", [(1, 16, 1), (1, 16, 128), (33, 272, 1), (129, 272, 128), (77, 4096, 1),
                                               (256, 1536, 128), (5, 11520, 1)])
def test_quantize_is_the_definition_bit_for_bit(rows, k, block_rows, bf16):
    x = _values(rows, k, rows + k)
    if bf16:
        x = bf16_to_f64(f32_to_bf16_bits(x)).astype(np.float32)
    codes, scales = quantize(x, block_rows, bf16)
    want_c, want_s = oo.quantize_f8(x, block_rows)
    assert np.array_equal(host(scales), want_s)
    assert np.array_equal(host(codes), want_c)


@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantize_zeros_extremes_and_non_finite_values(block_rows):
    x = np.zeros((130, 400), np.float32)
    x[1, 3], x[2, 200] = 3e38, -1e-38           # the largest scale; far below the floor
    x[129, 390] = np.nan                        # the last, partial block
    x[0, 300] = np.inf
    codes, scales = quantize(x, block_rows)
    want_c, want_s = oo.quantize_f8(x, block_rows)
    assert np.array_equal(host(scales), want_s, equal_nan=True)
    assert np.array_equal(host(codes) & 0x7F, want_c & 0x7F)       # the sign of a NaN or zero is free
    w = oo.widen_f8(host(codes), host(scales), block_rows)
    assert np.isnan(w[129, 390]) and np.isnan(w[0, 300])


def _operands(M, N, K, seed):
    rng = np.random.default_rng(seed)
    a = (rng.standard_normal((M, K)) * np.exp(0.5 * rng.standard_normal(K))).astype(np.float32)
    w = (rng.standard_normal((N, K)) * 0.02).astype(np.float32)
    return a, w, rng.standard_normal(N).astype(np.float32)


def gemm(a, sa, w, sw, bias, M, N, K, bf16):
    c, ok = guarded((M, N), torch.bfloat16 if bf16 else torch.float32, -7.0)
    L.lens_op_gemm_f8(a, sa, w, sw, bias, c, L.LENS_BF16 if bf16 else L.LENS_F32, M, N, K)
    torch.cuda.synchronize()
    ok()
    return c


def _widen(codes, scales, block_rows):
    s = scales.double().t().repeat_interleave(block_rows, 0).repeat_interleave(128, 1)
    return codes.view(torch.float8_e4m3fn).double() * s[:codes.shape[0], :codes.shape[1]]


def check_gemm(c, codes_a, sa, codes_w, sw, bias, K, bf16):
    """Against fp64 on the same codes and scales.  The products of two e4m3 values are exact
    in fp32; a sum of n terms in any order, each addition off by at most 2^-23 of the sum of
    magnitudes (truncation counted), is off by n 2^-23: 128 terms a block, one per block,
    the scale product, the bias."""
    A, W = _widen(codes_a, sa, 1), _widen(codes_w, sw, 128)
    ref, mag = A @ W.t(), A.abs() @ W.abs().t()
    if bias is not None:
        ref, mag = ref + bias.double(), mag + bias.double().abs()
    tol = (128 + K / 128 + 4) * 2.0 ** -23 * mag
    if bf16:
        tol = tol + 2.0 ** -8 * ref.abs()
    err = (c.double() - ref).abs()
    assert bool((err <= tol).all()), float((err / tol).max())


SIZES = [(1, 16, 16), (1, 4608, 1536), (2, 144, 400), (8, 1536, 4096), (9, 272, 1552), (16, 8192, 1536), (17, 128, 128),
         (33, 2000, 2880), (77, 1536, 4096), (128, 256, 384), (129, 400, 144), (255, 512, 1536), (333, 4608, 1536),
         (513, 1040, 2896), (1152, 1536, 1536), (4352, 1536, 4096),
         (40, 16, 16), (300, 16, 272), (64, 1536, 2576), (200, 400, 11520), (1500, 8192, 400), (2100, 4624, 144),
         (24, 8192, 1536), (50, 24576, 144), (64, 4096, 8192), (65, 144, 11520), (100, 19200, 144), (129, 2320, 1040),
         (300, 768, 4096), (640, 1536, 1536)]


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_gemm_f8(M, N, K, bf16):
    a, w, bias = _operands(M, N, K, M + N + K)
    (ca, sa), (cw, sw) = quantize(a, 1), quantize(w, 128)
    b = dev(bias) if (M + N) % 2 == 0 else None
    check_gemm(gemm(ca, sa, cw, sw, b, M, N, K, bf16), ca, sa, cw, sw, b, K, bf16)


@pytest.mark.parametrize("M", [3, 40, 300])
def test_gemm_f8_every_code_and_wide_scales(M):
    """Every finite e4m3 code on both sides, scales over thirty binary orders."""
    N, K = 272, 400
    rng = np.random.default_rng(M)
    finite = np.array([c for c in range(256) if c & 127 != 127], np.uint8)
    ca, cw = dev(rng.choice(finite, (M, K))), dev(rng.choice(finite, (N, K)))
    sa = dev(np.exp2(rng.uniform(-15, 15, (4, M))).astype(np.float32))
    sw = dev(np.exp2(rng.uniform(-15, 15, (4, 3))).astype(np.float32))
    check_gemm(gemm(ca, sa, cw, sw, None, M, N, K, False), ca, sa, cw, sw, None, K, False)


@pytest.mark.parametrize("M", [2, 100, 300])
def test_gemm_f8_non_finite_values_stay_in_their_row_or_column(M):
    N, K = 256, 272
    a, w, _ = _operands(M, N, K, 7)
    (ca, sa), (cw, sw) = quantize(a, 1), quantize(w, 128)
    ca[1, K - 1] = 0x7F                         # a NaN code in row 1
    sa[0, 0] = float("inf")                     # an infinite scale in row 0
    cw[200, 5] = 0xFF                           # a NaN code in column 200
    c = host(gemm(ca, sa, cw, sw, None, M, N, K, False))
    assert np.isnan(c[1]).all() and np.isnan(c[:, 200]).all() and not np.isfinite(c[0]).any()
    rest = np.delete(np.delete(c, [0, 1], 0), 200, 1)
    assert np.isfinite(rest).all()


@pytest.mark.parametrize("M,N,K", [(1, 1536, 1536), (40, 1536, 400), (600, 768, 1536)])
def test_gemm_f8_is_repeatable_on_streams_and_in_graphs(M, N, K):
    """The same bits from call to call, from two streams at once and from a replayed graph."""
    a, w, bias = _operands(M, N, K, 3)
    (ca, sa), (cw, sw), b = quantize(a, 1), quantize(w, 128), dev(bias)
    want = gemm(ca, sa, cw, sw, b, M, N, K, False).clone()
    outs = [torch.zeros((M, N), device="cuda") for _ in range(4)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    for i, o in enumerate(outs[:3]):
        with torch.cuda.stream(streams[i % 2]):
            L.lens_op_gemm_f8(ca, sa, cw, sw, b, o, L.LENS_F32, M, N, K)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        L.lens_op_gemm_f8(ca, sa, cw, sw, b, outs[3], L.LENS_F32, M, N, K)
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o, want)


def test_gemm_f8_large_outputs_pass_32_bit_offsets():
    """C beyond 2^31 elements: rows at the end are where they belong."""
    M, N, K = 40000, 65536, 16
    ca = torch.zeros((M, K), dtype=torch.uint8, device="cuda")
    cw = torch.full((N, K), 0x38, dtype=torch.uint8, device="cuda")          # ones
    ca[-1] = 0x38
    ca[-2, 0] = 0x40                                                          # 2
    sa, sw = torch.ones((1, M), device="cuda"), torch.ones((1, N // 128), device="cuda")
    c = torch.full((M, N), -7.0, dtype=torch.bfloat16, device="cuda")
    L.lens_op_gemm_f8(ca, sa, cw, sw, None, c, L.LENS_BF16, M, N, K)
    torch.cuda.synchronize()
    assert bool((c[-1] == 16).all()) and bool((c[-2] == 2).all()) and not bool(c[:-2].any())


def test_refuses_views_that_are_not_contiguous():
    x = torch.zeros((64, 256), device="cuda")
    codes, scales = torch.zeros((64, 128), dtype=torch.uint8, device="cuda"), torch.zeros((1, 64), device="cuda")
    with pytest.raises(L.LensError) as ei:
        L.lens_op_quantize_f8(x[:, :128], L.LENS_F32, 64, 128, 1, codes, scales)
    assert ei.value.status == 1
