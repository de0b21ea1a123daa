"""The 8-bit and windowed operations run together, as the attention half of a block uses
them: quantize the rows, project, attend a window with the text visible, project back,
then both norms with the gate and the next branch's 8-bit operand."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import flow_matching_mmdit_b200 as L  # noqa: E402
from tests.test_gpu_f8 import _widen  # noqa: E402
from tests.test_gpu_window import mask_of  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    L.load_library()


def rel(a, b):
    return float((a.double() - b).norm() / b.norm())


def test_attention_half_of_a_block():
    B, n_txt, n_img, heads, D = 2, 40, 360, 4, 256
    n, M = n_txt + n_img, 2 * 400
    g = torch.Generator(device="cuda")
    g.manual_seed(0)

    def normal(*s, std=1.0):
        return torch.randn(s, generator=g, device="cuda") * std

    def quantized(x, block_rows, kind):
        codes = torch.empty(x.shape, dtype=torch.uint8, device="cuda")
        scales = torch.empty((-(-x.shape[1] // 128), -(-x.shape[0] // block_rows)), device="cuda")
        L.lens_op_quantize_f8(x, kind, x.shape[0], x.shape[1], block_rows, codes, scales)
        return codes, scales

    x, h = normal(M, D).to(torch.bfloat16), normal(M, D)
    wqkv, wo = quantized(normal(3 * D, D, std=0.1), 128, L.LENS_F32), quantized(normal(D, D, std=0.1), 128, L.LENS_F32)
    bias = normal(3 * D)
    gain, mod = 1 + normal(D, std=0.1), normal(B, 3, D, std=0.3)

    # ---- the library, on one stream without a wait in between
    xa = quantized(x, 1, L.LENS_BF16)
    qkv = torch.empty((M, 3 * D), dtype=torch.bfloat16, device="cuda")
    L.lens_op_gemm_f8(*xa, *wqkv, bias, qkv, L.LENS_BF16, M, 3 * D, D)
    q, k, v = (t.contiguous() for t in qkv.view(B, n, 3, heads, 64).permute(2, 0, 3, 1, 4))
    att = torch.empty((B, n, D), dtype=torch.bfloat16, device="cuda")
    L.lens_op_attention_window(q, k, v, B, heads, heads, n, n, None, [n, n - 30], 50, 50, n_txt, 0.125, att)
    aa = quantized(att.view(M, D), 1, L.LENS_BF16)
    y = torch.empty((M, D), dtype=torch.bfloat16, device="cuda")
    L.lens_op_gemm_f8(*aa, *wo, None, y, L.LENS_BF16, M, D, D)
    h_out = torch.empty_like(h)
    codes = torch.empty((M, D), dtype=torch.uint8, device="cuda")
    scales = torch.empty((D // 128, M), device="cuda")
    L.lens_op_sandwich_norm(h, y, L.LENS_BF16, M, D, n, gain, mod[:, 0], None, mod[:, 1], mod[:, 2], 3 * D, 0.75, 1e-6,
                            h_out, codes, L.LENS_F8E4M3, scales)
    out = torch.empty((M, 3 * D), device="cuda")
    L.lens_op_gemm_f8(codes, scales, *wqkv, bias, out, L.LENS_F32, M, 3 * D, D)
    torch.cuda.synchronize()

    # ---- the same steps in fp64, unrounded between them except for the 8-bit weights
    W, Wo = _widen(*wqkv, 128), _widen(*wo, 128)
    r = (x.double() @ W.t() + bias.double()).view(B, n, 3, heads, 64).permute(2, 0, 3, 1, 4)
    o = torch.zeros((B, n, heads, 64), dtype=torch.float64, device="cuda")
    for b in range(B):
        m = mask_of(n, n, 0, [n, n - 30][b], 50, 50, n_txt)
        for i in range(heads):
            s = torch.where(m, r[0, b, i] @ r[1, b, i].t() * 0.125, -torch.inf)
            o[b, :, i] = torch.softmax(s, 1) @ r[2, b, i]
    yr = o.view(M, D) @ Wo.t()
    of = torch.arange(M, device="cuda") // n
    hr = 0.75 * h.double() + mod[of, 0].double() * gain.double() * yr / (yr.square().mean(1, keepdim=True) + 1e-6).sqrt()
    xr = (1 + mod[of, 2].double()) * hr / (hr.square().mean(1, keepdim=True) + 1e-6).sqrt() + mod[of, 1].double()
    # e4m3 rounds a value by up to 2^-4 of it, 0.026 rms over a 3-bit mantissa: each product
    # of rounded rows is held to 0.04.  Scores here have a deviation of 3.4, so theirs are off
    # by 0.026 * 3.4 * 2^(1/2) = 0.13, and so are the attention weights, whose errors average
    # out over the keys: the whole chain is held to 0.2 (a cosine of 0.98)
    cos = float((y.double() * yr).sum() / (y.double().norm() * yr.norm()))
    assert cos > 0.98, cos
    assert rel(qkv, (x.double() @ W.t() + bias.double())) < 0.04
    step_y = att.view(M, D).double() @ Wo.t()
    assert rel(y, step_y) < 0.04
    yd = y.double()
    hs = 0.75 * h.double() + mod[of, 0].double() * gain.double() * yd / (yd.square().mean(1, keepdim=True) + 1e-6).sqrt()
    assert rel(h_out, hs) < 1e-6
    xs = (1 + mod[of, 2].double()) * hs / (hs.square().mean(1, keepdim=True) + 1e-6).sqrt() + mod[of, 1].double()
    assert rel(_widen(codes, scales, 1), xs) < 0.04
    assert rel(out, xs @ W.t() + bias.double()) < 0.04
    assert rel(out, xr @ W.t() + bias.double()) < 0.2
    assert np.isfinite(float(out.sum()))


def test_operations_on_several_streams_at_once():
    """Products of each kernel and both attention kernels, shuffled over four streams: the same bits as alone."""
    rng = np.random.default_rng(3)
    jobs = []
    for M, N, K in ((8, 768, 1536), (77, 768, 2576), (300, 400, 1536), (1100, 2320, 272)):
        x = torch.from_numpy(rng.standard_normal((M + N, K)).astype(np.float32)).cuda()
        groups = -(-K // 128)
        ca, sa = torch.empty((M, K), dtype=torch.uint8, device="cuda"), torch.empty((groups, M), device="cuda")
        cw, sw = torch.empty((N, K), dtype=torch.uint8, device="cuda"), torch.empty((groups, -(-N // 128)), device="cuda")
        L.lens_op_quantize_f8(x[:M], L.LENS_F32, M, K, 1, ca, sa)
        L.lens_op_quantize_f8(x[M:], L.LENS_F32, N, K, 128, cw, sw)
        c = torch.empty((M, N), device="cuda")
        jobs.append((lambda st, a=(ca, sa, cw, sw, None, c, L.LENS_F32, M, N, K): L.lens_op_gemm_f8(*a, stream=st), c))
    for n_q, n_kv in ((1, 1500), (40, 700), (300, 1500)):
        q = torch.from_numpy(rng.standard_normal((2, 6, n_q, 64)).astype(np.float32)).cuda().to(torch.bfloat16)
        k, v = (torch.from_numpy(rng.standard_normal((2, 3, n_kv, 64)).astype(np.float32)).cuda().to(torch.bfloat16)
                for _ in range(2))
        o = torch.empty((2, n_q, 384), dtype=torch.bfloat16, device="cuda")
        a = (q, k, v, 2, 6, 3, n_q, n_kv, [n_kv - n_q] * 2, None, 400, 0, 4, 0.125, o)
        jobs.append((lambda st, a=a: L.lens_op_attention_window(*a, stream=st), o))
    want = []
    for call, out in jobs:
        call(None)
        torch.cuda.synchronize()
        want.append(out.clone())
    streams = [torch.cuda.Stream() for _ in range(4)]
    for _ in range(10):
        for _, out in jobs:
            out.zero_()
        torch.cuda.synchronize()
        for i, job in enumerate(rng.permutation(len(jobs))):
            jobs[job][0](streams[i % 4])
        torch.cuda.synchronize()
        for (_, out), w in zip(jobs, want):
            assert torch.equal(out, w)


def test_the_forms_with_single_arguments_give_the_same_bits():
    lib, M, D = L.load_library(), 40, 400
    rng = np.random.default_rng(4)
    x, h = (torch.from_numpy(rng.standard_normal((M, D)).astype(np.float32)).cuda() for _ in range(2))
    st = torch.cuda.current_stream().cuda_stream

    def outputs():
        return (torch.empty((M, D), dtype=torch.uint8, device="cuda"), torch.empty((4, M), device="cuda"),
                torch.empty((M, D), device="cuda"), torch.empty((M, D), dtype=torch.bfloat16, device="cuda"),
                torch.empty((M, 48), device="cuda"), torch.empty((1, M, 320), dtype=torch.bfloat16, device="cuda"))

    a, b = outputs(), outputs()
    w, ws = torch.empty((48, D), dtype=torch.uint8, device="cuda"), torch.empty((4, 1), device="cuda")
    q = x[:, :320].reshape(M, 5, 64).transpose(0, 1).contiguous().to(torch.bfloat16)
    L.lens_op_quantize_f8(h[:, :48].t().contiguous().repeat(1, 10), L.LENS_F32, 48, D, 128, w, ws)
    L.lens_op_quantize_f8(x, L.LENS_F32, M, D, 1, a[0], a[1])
    L.lens_op_sandwich_norm(h, x, L.LENS_F32, M, D, M, None, None, h[0], x[1], x[2], 0, 0.5, 1e-6, a[2], a[3], L.LENS_BF16)
    L.lens_op_gemm_f8(a[0], a[1], w, ws, None, a[4], L.LENS_F32, M, 48, D)
    L.lens_op_attention_window(q, q, q, 1, 5, 5, M, M, None, None, 7, 3, 2, 0.125, a[5])
    assert lib.lens_op_quantize_f8(x.data_ptr(), 0, M, D, 1, b[0].data_ptr(), b[1].data_ptr(), st) == 0
    assert lib.lens_op_sandwich_norm(h.data_ptr(), x.data_ptr(), 0, M, D, M, None, None, h[0].data_ptr(),
                                     x[1].data_ptr(), x[2].data_ptr(), 0, 0.5, 1e-6, b[2].data_ptr(), b[3].data_ptr(),
                                     1, None, st) == 0
    assert lib.lens_op_gemm_f8(b[0].data_ptr(), b[1].data_ptr(), w.data_ptr(), ws.data_ptr(), None, b[4].data_ptr(), 0,
                               M, 48, D, st) == 0
    assert lib.lens_op_attention_window(q.data_ptr(), q.data_ptr(), q.data_ptr(), 1, 5, 5, M, M, None, None, 7, 3, 2,
                                        0.125, b[5].data_ptr(), st) == 0
    torch.cuda.synchronize()
    for one, other in zip(a, b):
        assert torch.equal(one, other)
