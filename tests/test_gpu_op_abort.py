"""The abort flag that the handle-free operations share: a call after one of them gave up
reports it, lens_op_sync clears it, and the operations are right again.  The flag is raised
by its test hook; nothing waits out, faults or hangs."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import flow_matching_mmdit_b200 as L  # noqa: E402

TIMEOUT = 5


@pytest.fixture(autouse=True)
def cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    L.load_library()
    yield
    torch.cuda.synchronize()
    try:
        L.lens_op_sync()
    except L.LensError:
        pass


def normal(*shape, dtype=torch.bfloat16, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + sum(shape))
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def gemm_f8(M, N, K):
    groups = -(-K // 128)
    x = normal(M + N, K, dtype=torch.float32)
    ca, sa = torch.empty((M, K), dtype=torch.uint8, device="cuda"), torch.empty((groups, M), device="cuda")
    cw, sw = torch.empty((N, K), dtype=torch.uint8, device="cuda"), torch.empty((groups, -(-N // 128)), device="cuda")
    L.lens_op_quantize_f8(x[:M], L.LENS_F32, M, K, 1, ca, sa)
    L.lens_op_quantize_f8(x[M:], L.LENS_F32, N, K, 128, cw, sw)
    c = torch.zeros((M, N), device="cuda")
    return lambda: L.lens_op_gemm_f8(ca, sa, cw, sw, None, c, L.LENS_F32, M, N, K), c


def window(n_q, n_kv):
    q, k, v = normal(1, 6, n_q, 64), normal(1, 3, n_kv, 64), normal(1, 3, n_kv, 64, seed=1)
    o = torch.zeros((1, n_q, 384), dtype=torch.bfloat16, device="cuda")
    return lambda: L.lens_op_attention_window(q, k, v, 1, 6, 3, n_q, n_kv, None, None, 300, 300, 4, 0.125, o), o


def gemm_bf16(M, N, K):
    a, b = normal(M, K), normal(N, K, seed=1)
    c = torch.zeros((M, N), device="cuda")
    return lambda: L.lens_op_gemm_bf16(a, b, None, c, M, N, K), c


def joint(n_txt, n_img):
    q, k, v = (normal(1, 24, n_txt + n_img, 64, seed=i) for i in range(3))
    ot, oi = (torch.zeros((1, n, 1536), dtype=torch.bfloat16, device="cuda") for n in (n_txt, n_img))
    return lambda: L.lens_op_attention(q, k, v, 1, n_txt, n_img, ot, oi), oi


# the 8-bit product's split 64- and 128-column kernels and both pair kernels, the many-row
# window kernel, a bf16 product and joint attention
FLAGGED = [(gemm_f8, (60, 768, 2576)), (gemm_f8, (100, 768, 2576)), (gemm_f8, (1280, 1040, 1040)),
           (gemm_f8, (1100, 2320, 2320)), (window, (700, 700)), (gemm_bf16, (300, 512, 512)), (joint, (40, 300))]


@pytest.mark.parametrize("make,size", FLAGGED)
def test_a_call_after_an_abort_reports_it(make, size):
    call, out = make(*size)
    call()
    L.lens_op_sync()
    want = out.clone()
    out.zero_()
    L.lens_op_debug_raise_abort()
    torch.cuda.synchronize()
    for _ in range(2):                              # until it has been reported by lens_op_sync
        with pytest.raises(L.LensError) as e:
            call()
        assert e.value.status == TIMEOUT
    torch.cuda.synchronize()
    assert not bool(out.any())
    with pytest.raises(L.LensError) as e:
        L.lens_op_sync()
    assert e.value.status == TIMEOUT
    L.lens_op_sync()                                # reported once
    call()
    L.lens_op_sync()
    assert torch.equal(out, want)


@pytest.mark.parametrize("make,size", FLAGGED)
def test_kernels_launched_behind_an_abort_leave_and_the_next_are_right(make, size):
    """Launched before the host sees the flag (or refused, if it already has): each leaves in
    order, draining what it started, and nothing of it reaches the calls after the report."""
    call, out = make(*size)
    call()
    L.lens_op_sync()
    want = out.clone()
    for _ in range(3):
        L.lens_op_debug_raise_abort()
        for _ in range(4):
            try:
                call()
            except L.LensError as e:
                assert e.status == TIMEOUT
        with pytest.raises(L.LensError) as e:
            L.lens_op_sync()
        assert e.value.status == TIMEOUT
        out.zero_()
        call()
        L.lens_op_sync()
        assert torch.equal(out, want)


def test_sync_on_another_stream_reports_it_too():
    side = torch.cuda.Stream()
    L.lens_op_debug_raise_abort(stream=side)
    side.synchronize()
    with pytest.raises(L.LensError) as e:
        L.lens_op_sync()
    assert e.value.status == TIMEOUT
    L.lens_op_sync(stream=side)


FIRST_CALL_CAPTURED = """
import torch
import flow_matching_mmdit_b200 as L
a, c = torch.ones((64, 64), dtype=torch.bfloat16, device="cuda"), torch.zeros((64, 64), device="cuda")
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    L.lens_op_gemm_bf16(a, a, None, c, 64, 64, 64)
assert not bool(c.any())
g.replay()
L.lens_op_sync()
assert bool((c == 64).all())
"""


def test_the_first_call_of_a_process_may_come_inside_a_capture():
    """The flag's host word is set up aside from the capture."""
    subprocess.run([sys.executable, "-c", FIRST_CALL_CAPTURED], cwd=ROOT, check=True, timeout=300)
