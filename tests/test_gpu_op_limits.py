"""The 8-bit and windowed operations at the ends of their documented ranges, and captured together."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import flow_matching_mmdit_b200 as L  # noqa: E402
from tests.test_gpu_window import check as check_window  # noqa: E402
from tests.test_gpu_window import make, run as window  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    L.load_library()


def ones(rows, k):
    return torch.full((rows, k), 0x38, dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("M,N,K", [(2 ** 22, 16, 16), (1, 2 ** 22, 16), (40, 2 ** 22, 16), (2, 16, 2 ** 22),
                                   (60, 32, 2 ** 22), (200, 16, 2 ** 20)])
def test_products_of_the_largest_sizes(M, N, K):
    """Rows and columns of ones times small integers: every sum is exact in fp32."""
    ca, cw = ones(M, K), ones(N, K)
    groups = -(-K // 128)
    g = torch.Generator(device="cuda")
    g.manual_seed(M + N)
    # powers of two that keep each sum a multiple of 2^-2 below 2^24
    sa = torch.where(torch.rand((groups, M), generator=g, device="cuda") < 0.5, 0.25, 0.5)
    sw = torch.ones((groups, -(-N // 128)), device="cuda")
    c = torch.empty((M, N), device="cuda")
    L.lens_op_gemm_f8(ca, sa, cw, sw, None, c, L.LENS_F32, M, N, K)
    last = K - 128 * (groups - 1)
    want = sa[:-1].double().sum(0) * 128 + sa[-1].double() * last
    assert bool((c.double() == want[:, None]).all())


@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("rows,k", [(2, 2 ** 22), (2 ** 21 + 5, 16), (130, 2 ** 20)])
def test_quantization_of_the_largest_sizes(rows, k, block_rows):
    x = torch.full((rows, k), 3.0, dtype=torch.bfloat16, device="cuda")
    x[-1, -16:], x[0, :16] = 7.0, -14.0
    codes = torch.empty((rows, k), dtype=torch.uint8, device="cuda")
    scales = torch.empty((-(-k // 128), -(-rows // block_rows)), device="cuda")
    L.lens_op_quantize_f8(x, L.LENS_BF16, rows, k, block_rows, codes, scales)
    amax = torch.full_like(scales, 3.0)
    amax[-1, -1] = 7.0
    amax[0, 0] = 14.0
    want = amax / torch.full_like(amax, 448.0)       # (by a number torch multiplies by 1 / 448)
    assert torch.equal(scales, want)
    # 448 / amax is 149.33, 64 or 32: 3 becomes 448, 192 or 96, all e4m3 values
    at = amax.t().repeat_interleave(block_rows, 0)[:rows].repeat_interleave(128, 1)[:, :k]
    value = torch.where(at == 3.0, 448.0, torch.where(at == 7.0, 192.0, 96.0))
    value[-1, -16:], value[0, :16] = 448.0, -448.0
    got = codes.view(torch.float8_e4m3fn)
    assert all(torch.equal(got[i:i + 2 ** 18].float(), value[i:i + 2 ** 18]) for i in range(0, rows, 2 ** 18))


@pytest.mark.parametrize("H,Hk,n_q,n_kv", [(1024, 1, 1, 50), (1024, 1024, 2, 9), (1023, 1, 3, 70), (1000, 8, 40, 200),
                                           (1024, 1, 300, 300), (1024, 1024, 130, 130)])
def test_windows_of_the_most_heads(H, Hk, n_q, n_kv):
    q, k, v = make(1, H, Hk, n_q, n_kv, H + n_q)
    start = [n_kv - n_q]
    check_window(window(q, k, v, start, None, 40, 0, 2), q, k, v, start, None, 40, 0, 2, heads=[0, 1, H // 2, H - 1])


@pytest.mark.parametrize("n_q", [1, 200])
def test_windows_of_the_most_sequences(n_q):
    B, n_kv = 64, 260
    q, k, v = make(B, 2, 1, n_q, n_kv, n_q)
    length = [(i * 13) % (n_kv + 1) for i in range(B)]
    start = [max(0, n - n_q) for n in length]
    check_window(window(q, k, v, start, length, 50, 3, 4), q, k, v, start, length, 50, 3, 4)


@pytest.mark.parametrize("n_q", [1, 50, 200])
def test_windows_of_the_largest_numbers(n_q):
    """Starts at the end of the position range, widths and sinks of the largest int."""
    n_kv, big, end = 150, 2 ** 31 - 1, 2 ** 29 - n_q
    q, k, v = make(1, 2, 2, n_q, n_kv, 3)
    for start, left, right, sinks in ((end, big, big, 0), (end, -1, big, big), (0, big, big, big), (0, 0, 0, big),
                                      (end, 5, 0, big), (end, 0, 0, 0), (end, 2 ** 29 - n_q, 0, 0)):
        check_window(window(q, k, v, [start], None, left, right, sinks), q, k, v, [start], None, left, right, sinks)


@pytest.mark.parametrize("n_q,n_kv", [(500, 20), (40, 1), (129, 128), (1, 1)])
def test_more_queries_than_keys(n_q, n_kv):
    q, k, v = make(2, 4, 2, n_q, n_kv, 4)
    for length in (None, [n_kv, n_kv // 2], [0, 0]):
        check_window(window(q, k, v, None, length, 30, 5, 1), q, k, v, None, length, 30, 5, 1)


@pytest.mark.parametrize("rows", [3, 90, 700])
def test_a_captured_branch_replays_over_new_inputs(rows):
    """Quantize, project, attend, quantize, project back, norms to 8 bits: one graph, replayed over
    inputs that change between replays, against the same calls made one by one."""
    D, heads = 256, 4
    g = torch.Generator(device="cuda")
    g.manual_seed(rows)

    def normal(*s, std=1.0):
        return torch.randn(s, generator=g, device="cuda") * std

    def codes(*shape):
        return torch.empty(shape, dtype=torch.uint8, device="cuda")

    def weight(n, k):
        c, s = codes(n, k), torch.empty((k // 128, n // 128), device="cuda")
        L.lens_op_quantize_f8(normal(n, k, std=0.1), L.LENS_F32, n, k, 128, c, s)
        return c, s

    def bf16(*shape):
        return torch.empty(shape, dtype=torch.bfloat16, device="cuda")

    wq, wo = weight(D, D), weight(D, D)
    x, h, mod = normal(rows, D).to(torch.bfloat16), normal(rows, D), normal(1, 3, D, std=0.3)
    k, v = (normal(1, heads, rows, 64).to(torch.bfloat16) for _ in range(2))
    xc, xs, q, att, ac, as_, y = (codes(rows, D), torch.empty((2, rows), device="cuda"), bf16(rows, D),
                                  bf16(1, rows, D), codes(rows, D), torch.empty((2, rows), device="cuda"), bf16(rows, D))
    qh = bf16(1, heads, rows, 64)
    h_out, out, out_s = torch.empty((rows, D), device="cuda"), codes(rows, D), torch.empty((2, rows), device="cuda")

    def branch():
        L.lens_op_quantize_f8(x, L.LENS_BF16, rows, D, 1, xc, xs)
        L.lens_op_gemm_f8(xc, xs, *wq, None, q, L.LENS_BF16, rows, D, D)
        qh.copy_(q.view(1, rows, heads, 64).transpose(1, 2))
        L.lens_op_attention_window(qh, k, v, 1, heads, heads, rows, rows, None, None, 40, 0, 2, 0.125, att)
        L.lens_op_quantize_f8(att.view(rows, D), L.LENS_BF16, rows, D, 1, ac, as_)
        L.lens_op_gemm_f8(ac, as_, *wo, None, y, L.LENS_BF16, rows, D, D)
        L.lens_op_sandwich_norm(h, y, L.LENS_BF16, rows, D, rows, None, mod[:, 0], None, mod[:, 1], mod[:, 2], 3 * D,
                                0.5, 1e-6, h_out, out, L.LENS_F8E4M3, out_s)

    branch()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(2):                        # the second over the first's buffers
            branch()
    for seed in range(3):
        x.copy_(normal(rows, D))
        h.copy_(normal(rows, D))
        k.copy_(normal(1, heads, rows, 64))
        branch()
        torch.cuda.synchronize()
        want = [t.clone() for t in (h_out, out, out_s)]
        for t in (h_out, out, out_s, att, y, q):
            t.zero_()
        graph.replay()
        L.lens_op_sync()
        assert all(torch.equal(a, b) for a, b in zip((h_out, out, out_s), want))
