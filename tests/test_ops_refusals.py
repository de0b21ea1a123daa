"""Argument errors of the 8-bit and windowed operations: refused before any device call."""
import ctypes
import os

import pytest

from flow_matching_mmdit_b200 import binding

P = ctypes.c_void_p
BAD, SHAPE = 1, 2


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(binding.LIB_PATH):
        from flow_matching_mmdit_b200 import build
        build.build()
    return binding.load_library()


def test_quantize_f8_refusals(lib):
    def call(x=16, t=0, rows=4, k=128, br=1, codes=16, scales=16):
        return lib.lens_op_quantize_f8(P(x), t, rows, k, br, P(codes), P(scales), None)
    for kw in (dict(x=0), dict(codes=0), dict(scales=0), dict(t=2), dict(t=7), dict(br=2), dict(br=0), dict(x=8),
               dict(codes=4), dict(scales=2)):
        assert call(**kw) == BAD, kw
    for kw in (dict(rows=0), dict(rows=-1), dict(rows=2 ** 30 + 1), dict(k=0), dict(k=24), dict(k=2 ** 22 + 16)):
        assert call(**kw) == SHAPE, kw


def test_gemm_f8_refusals(lib):
    def call(a=16, sa=16, w=16, sw=16, bias=0, c=16, t=0, m=4, n=32, k=128):
        return lib.lens_op_gemm_f8(P(a), P(sa), P(w), P(sw), P(bias), P(c), t, m, n, k, None)
    for kw in (dict(a=0), dict(sa=0), dict(w=0), dict(sw=0), dict(c=0), dict(t=2), dict(a=8), dict(w=8), dict(c=8),
               dict(sa=2), dict(sw=1), dict(bias=3)):
        assert call(**kw) == BAD, kw
    for kw in (dict(m=0), dict(n=0), dict(n=24), dict(k=0), dict(k=8), dict(k=136), dict(m=-3),
               dict(n=2 ** 22 + 16), dict(m=2 ** 22 + 1), dict(k=2 ** 22 + 16)):
        assert call(**kw) == SHAPE, kw


def test_sandwich_norm_refusals(lib):
    def call(h=16, y=16, yt=1, m=4, d=128, rpb=4, post=0, gate=0, pre=0, shift=0, scale=0, stride=128, a=1.0, eps=1e-6,
             ho=16, out=16, ot=1, os_=0):
        return lib.lens_op_sandwich_norm(P(h), P(y), yt, m, d, rpb, P(post), P(gate), P(pre), P(shift), P(scale), stride,
                                         a, eps, P(ho), P(out), ot, P(os_), None)
    nan, inf = float("nan"), float("inf")
    for kw in (dict(h=0), dict(y=0), dict(ho=0), dict(out=0), dict(yt=2), dict(ot=0), dict(ot=2), dict(ot=2, os_=2),
               dict(eps=0.0), dict(eps=nan), dict(eps=inf), dict(a=nan), dict(a=inf), dict(h=8), dict(y=4), dict(ho=24),
               dict(out=8), dict(gate=4), dict(shift=8), dict(scale=8), dict(post=8), dict(pre=8)):
        assert call(**kw) == BAD, kw
    for kw in (dict(m=0), dict(d=0), dict(d=24), dict(d=8208), dict(rpb=0), dict(stride=-4), dict(stride=6)):
        assert call(**kw) == SHAPE, kw


def test_attention_window_refusals(lib):
    def ints(v):
        return (ctypes.c_int * len(v))(*v) if v is not None else None

    def call(q=16, k=16, v=16, b=2, h=4, hk=2, nq=5, nkv=9, start=None, length=None, left=3, right=0, sinks=1,
             scale=0.125, out=16):
        return lib.lens_op_attention_window(P(q), P(k), P(v), b, h, hk, nq, nkv, ints(start), ints(length), left, right,
                                            sinks, scale, P(out), None)
    for kw in (dict(q=0), dict(k=0), dict(v=0), dict(out=0), dict(q=8), dict(k=8), dict(v=8), dict(out=8),
               dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")), dict(scale=3e38), dict(left=-2),
               dict(right=-2), dict(sinks=-1)):
        assert call(**kw) == BAD, kw
    for kw in (dict(b=0), dict(b=65), dict(h=0), dict(h=1025, hk=1025), dict(hk=0), dict(h=4, hk=3), dict(nq=0),
               dict(nkv=0), dict(nkv=2 ** 29 + 1), dict(nq=2 ** 29 + 1), dict(start=[0, -1]),
               dict(start=[2 ** 29 - 4, 0]), dict(length=[10, 1]), dict(length=[-1, 1])):
        assert call(**kw) == SHAPE, kw


def test_binding_refuses_lengths_for_another_batch():
    with pytest.raises(binding.LensError) as ei:
        binding.lens_op_attention_window(None, None, None, 2, 4, 4, 1, 8, [0], [8, 8], 1, 0, 0, 0.125, None, stream=0)
    assert ei.value.status == SHAPE


def test_binding_refuses_host_tensors():
    """Tensors that are not on the current device (here: on the host) never reach the library."""
    import torch
    f, b = torch.zeros(128, 128), torch.zeros(128, 128, dtype=torch.uint8)
    for call in (lambda: binding.lens_op_quantize_f8(f, 0, 128, 128, 1, b, f, stream=0),
                 lambda: binding.lens_op_gemm_f8(b, f, b, f, None, f, 0, 128, 128, 128, stream=0),
                 lambda: binding.lens_op_sandwich_norm(f, f, 0, 128, 128, 1, None, None, None, None, None, 0, 1.0, 1e-6,
                                                       f, f, 1, stream=0),
                 lambda: binding.lens_op_attention_window(f, f, f, 1, 1, 1, 1, 1, None, None, 0, 0, 0, 0.125, f,
                                                          stream=0)):
        with pytest.raises(binding.LensError) as ei:
            call()
        assert ei.value.status == BAD


def test_binding_refuses_modulation_rows_of_another_device_or_not_dense():
    import torch
    x = torch.zeros(4, 6, 128)
    host = x.get_device()
    assert binding._rows("norm", host, None) is None
    assert binding._rows("norm", host, x[:, 2]) == x.data_ptr() + 2 * 128 * 4
    for dev, bad in ((0, x[:, 0]), (host, x[:, 0].t()), (host, x[:, 0, ::2])):
        with pytest.raises(binding.LensError) as ei:
            binding._rows("norm", dev, bad)
        assert ei.value.status == BAD


# valid arguments of each operation (never called as they are: the pointers are made up)
VALID = {
    "lens_op_quantize_f8": [16, 0, 4, 128, 1, 16, 16, 0],
    "lens_op_gemm_f8": [16, 16, 16, 16, 16, 16, 0, 4, 32, 128, 0],
    "lens_op_sandwich_norm": [16, 16, 1, 4, 128, 4, 16, 16, 16, 16, 16, 128, 1.0, 1e-6, 16, 16, 2, 16, 0],
    "lens_op_attention_window": [16, 16, 16, 2, 4, 2, 5, 9, 0, 0, 3, 0, 1, 0.125, 16, 0],
}
# (argument, value, status): one wrong value for every argument that is looked at
WRONG = {
    "lens_op_quantize_f8": [(0, 8, BAD), (1, 2, BAD), (2, 2 ** 40, SHAPE), (3, 2 ** 40, SHAPE), (4, 3, BAD), (5, 8, BAD),
                            (6, 2, BAD)],
    "lens_op_gemm_f8": [(0, 8, BAD), (1, 2, BAD), (2, 8, BAD), (3, 2, BAD), (4, 2, BAD), (5, 8, BAD), (6, 2, BAD),
                        (7, 0, SHAPE), (8, 24, SHAPE), (9, 24, SHAPE)],
    "lens_op_sandwich_norm": [(0, 8, BAD), (1, 8, BAD), (2, 2, BAD), (3, 0, SHAPE), (4, 24, SHAPE), (5, 0, SHAPE),
                              (6, 8, BAD), (7, 8, BAD), (8, 8, BAD), (9, 8, BAD), (10, 8, BAD), (11, 6, SHAPE),
                              (12, float("inf"), BAD), (13, 0.0, BAD), (14, 8, BAD), (15, 8, BAD), (16, 0, BAD),
                              (17, 2, BAD)],
    "lens_op_attention_window": [(0, 8, BAD), (1, 8, BAD), (2, 8, BAD), (3, 65, SHAPE), (4, 5, SHAPE), (5, 3, SHAPE),
                                 (6, 0, SHAPE), (7, 0, SHAPE), (10, -2, BAD), (11, -2, BAD), (12, -1, BAD),
                                 (13, 0.0, BAD), (14, 8, BAD)],
}


@pytest.mark.parametrize("name", sorted(VALID))
def test_argument_blocks_hold_the_arguments_in_order(lib, name):
    """Each wrong argument alone is refused with its status by both forms, and no block by a NULL."""
    for at, value, status in WRONG[name]:
        args = list(VALID[name])
        args[at] = value
        assert getattr(lib, name)(*args) == status, (at, value)
        assert lib.f8_blocks[name](binding._BLOCKS[name].pack(*args)) == status, (at, value)
    assert lib.f8_blocks[name](None) == BAD


def test_argument_blocks_hold_the_lengths(lib):
    for at in (8, 9):
        args, bad = list(VALID["lens_op_attention_window"]), (ctypes.c_int * 2)(0, -1)
        args[at] = ctypes.addressof(bad)
        assert lib.f8_blocks["lens_op_attention_window"](
            binding._BLOCKS["lens_op_attention_window"].pack(*args)) == SHAPE


def test_binding_refuses_numbers_that_do_not_fit():
    for args in ([16, 0, 4, 128, 2 ** 40, 16, 16, 0], [16, 0, 2 ** 70, 128, 1, 16, 16, 0], [16, 0.5, 4, 128, 1, 16, 16, 0]):
        with pytest.raises(binding.LensError) as ei:
            binding._run_block("lens_op_quantize_f8", *args)
        assert ei.value.status == BAD
