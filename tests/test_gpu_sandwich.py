"""GPU parity of the fused norms against the fp64 oracle."""
import numpy as np
import pytest

from oracle import ops_oracle as oo
from tests.helpers import dev, host
from tests.test_gpu_f8 import guarded

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import flow_matching_mmdit_b200 as L  # noqa: E402

EPS, RS = 1e-6, 0.75


@pytest.fixture(scope="module", autouse=True)
def cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    L.load_library()


def make(M, D, rpb, seed, y_bf16=True):
    rng = np.random.default_rng(seed)
    nb = -(-M // rpb)
    t = {"h": 3 * rng.standard_normal((M, D)), "y": rng.standard_normal((M, D)),
         "post_gain": 1 + 0.1 * rng.standard_normal(D), "pre_gain": 1 + 0.1 * rng.standard_normal(D),
         "mod": 0.3 * rng.standard_normal((nb, 3, D))}
    t = {k: dev(v.astype(np.float32)) for k, v in t.items()}
    if y_bf16:
        t["y"] = t["y"].to(torch.bfloat16)
    return t


def run(t, M, D, rpb, use, f8, in_place=False, residual_scale=RS, stream=None):
    opt = {"post_gain": t["post_gain"], "pre_gain": t["pre_gain"], "gate": t["mod"][:, 0], "shift": t["mod"][:, 1],
           "scale": t["mod"][:, 2]}
    opt = {k: (v if k in use else None) for k, v in opt.items()}
    h_out, ok1 = guarded((M, D), torch.float32, -7.0)
    h = t["h"]
    if in_place:
        h_out.copy_(h)
        h = h_out
    out, ok2 = guarded((M, D), torch.uint8 if f8 else torch.bfloat16, 3)
    scales, ok3 = guarded((-(-D // 128), M), torch.float32, -7.0)
    L.lens_op_sandwich_norm(h, t["y"], L.LENS_BF16 if t["y"].dtype == torch.bfloat16 else L.LENS_F32, M, D, rpb,
                            opt["post_gain"], opt["gate"], opt["pre_gain"], opt["shift"], opt["scale"], 3 * D,
                            residual_scale, EPS, h_out, out, L.LENS_F8E4M3 if f8 else L.LENS_BF16,
                            scales if f8 else None, stream=stream)
    torch.cuda.synchronize()
    ok1(), ok2(), ok3()
    return h_out, out, scales


def reference(t, M, rpb, use, residual_scale=RS):
    of = np.arange(M) // rpb
    mod = host(t["mod"]).astype(np.float64)[of]
    opt = {"post_gain": host(t["post_gain"]), "pre_gain": host(t["pre_gain"]), "gate": mod[:, 0], "shift": mod[:, 1],
           "scale": mod[:, 2]}
    opt = {k: (v if k in use else None) for k, v in opt.items()}
    y = t["y"].double().cpu().numpy()
    h, out = oo.sandwich_norm(host(t["h"]), y, residual_scale, EPS, **opt)
    return h, out, np.abs(h - residual_scale * host(t["h"]).astype(np.float64)), opt


ALL = ("post_gain", "pre_gain", "gate", "shift", "scale")
U = 2.0 ** -24


def tolerances(t, h, out, branch, opt, residual_scale=RS):
    """A sum of D squares by eight terms a thread and a tree of at most 5 + 32 additions is
    off by at most 46 U, the mean, root and reciprocal by 4 U more (U = 2^-24): 50 U on each
    norm, half of it under the root.  h_out: that and five products on the branch, three
    roundings on the residual.  out: the error of h_out carried through, the second norm (its
    rms is off by at most the largest error of a row), five more roundings."""
    e_h = U * (30 * branch + 3 * np.abs(residual_scale * host(t["h"]).astype(np.float64)) + 2 * np.abs(h))
    rms = np.sqrt(np.mean(h * h, axis=1, keepdims=True) + EPS)
    mul = np.abs((1 + (0 if opt["scale"] is None else opt["scale"])) * (1 if opt["pre_gain"] is None else opt["pre_gain"]))
    e_o = mul / rms * (e_h + np.abs(h) * (30 * U + e_h.max(axis=1, keepdims=True) / rms)) + 5 * U * np.abs(out) \
        + U * (0 if opt["shift"] is None else np.abs(opt["shift"])) + 5 * U * mul * np.abs(h) / rms
    return e_h, e_o


@pytest.mark.parametrize("M,D,rpb,use,y_bf16", [
    (1, 16, 1, (), True), (3, 144, 2, ALL, True), (77, 1536, 77, ("post_gain", "gate"), True),
    (130, 1536, 65, ALL, False), (9, 2896, 4, ("pre_gain", "shift"), True), (5, 4096, 100, ("scale",), False),
    (33, 4112, 11, ALL, True), (3001, 128, 7, ALL, True), (700, 2048, 699, ALL, False), (7, 8192, 3, ALL, True), (2, 8192, 1, ("gate",), False), (1000, 272, 333, ALL, True)])
def test_sandwich_norm(M, D, rpb, use, y_bf16):
    t = make(M, D, rpb, M + D, y_bf16)
    h, out, branch, opt = reference(t, M, rpb, use)
    e_h, e_o = tolerances(t, h, out, branch, opt)
    gh, go, _ = run(t, M, D, rpb, use, False)
    assert np.all(np.abs(host(gh) - h) <= e_h)
    assert np.all(np.abs(go.double().cpu().numpy() - out) <= 2.0 ** -8 * np.abs(out) + e_o)
    # quantized: scale from the largest magnitude of each block, codes within half a step
    gh8, codes, scales = run(t, M, D, rpb, use, True)
    assert torch.equal(gh8, gh)
    w = oo.widen_f8(host(codes), host(scales), 1)
    for g in range(scales.shape[0]):
        c = slice(128 * g, 128 * (g + 1))
        top, e = np.abs(out[:, c]).max(1), e_o[:, c].max(1)
        assert np.all(np.abs(host(scales)[g] * 448.0 - top) <= e + 2 * U * top)
        half = np.maximum(np.abs(out[:, c]) * 2.0 ** -4, host(scales)[g][:, None] * 2.0 ** -10)
        assert np.all(np.abs(w[:, c] - out[:, c]) <= half * (1 + 1e-5) + 2 * e_o[:, c])


def test_sandwich_norm_in_place_and_zero_rows():
    M, D = 65, 1536
    t = make(M, D, 13, 5)
    t["y"][3] = 0
    t["h"][4], t["y"][4] = 0, 0
    a, out_a, _ = run(t, M, D, 13, ALL, False)
    b, out_b, _ = run(t, M, D, 13, ALL, False, in_place=True)
    assert torch.equal(a, b) and torch.equal(out_a, out_b)
    assert torch.equal(a[3], RS * t["h"][3]) and not bool(a[4].any())
    assert torch.equal(out_a[4], t["mod"][4 // 13, 1].to(torch.bfloat16))
    _, codes, scales = run(t, M, D, 13, ("gate",), True)
    assert not bool(codes[4].any()) and bool((scales[:, 4] == float(oo.AMAX_FLOOR) / 448).all())


def test_sandwich_norm_non_finite_rows_stay_alone():
    M, D = 20, 400
    t = make(M, D, 20, 6)
    want, want_o, _ = run(t, M, D, 20, ALL, False)
    t["y"][2, 7], t["h"][11, 300] = float("nan"), float("inf")
    got, got_o, _ = run(t, M, D, 20, ALL, False)
    keep = [i for i in range(M) if i not in (2, 11)]
    assert torch.equal(got[keep], want[keep]) and torch.equal(got_o[keep], want_o[keep])
    assert bool(torch.isnan(got[2]).all()) and bool(torch.isinf(got[11, 300])) and bool(torch.isnan(got_o[2]).all())


def test_sandwich_norm_on_a_side_stream_and_in_a_graph():
    M, D = 300, 1536
    t = make(M, D, 100, 8)
    want, want_o, _ = run(t, M, D, 100, ALL, False)
    side = torch.cuda.Stream()
    got, got_o, _ = run(t, M, D, 100, ALL, False, stream=side)
    assert torch.equal(got, want) and torch.equal(got_o, want_o)
    h_out, out = torch.zeros_like(want), torch.zeros_like(want_o)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        L.lens_op_sandwich_norm(t["h"], t["y"], L.LENS_BF16, M, D, 100, t["post_gain"], t["mod"][:, 0], t["pre_gain"],
                                t["mod"][:, 1], t["mod"][:, 2], 3 * D, RS, EPS, h_out, out, L.LENS_BF16)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(h_out, want) and torch.equal(out, want_o)


@pytest.mark.parametrize("which", ["gate", "shift", "scale"])
def test_sandwich_norm_refuses_modulation_that_is_not_on_the_device_or_not_dense(which):
    M, D = 8, 128
    t = make(M, D, 8, 9)
    h_out, out = torch.empty_like(t["h"]), torch.empty((M, D), dtype=torch.bfloat16, device="cuda")
    for bad in (torch.zeros((1, D)), torch.zeros((1, 2 * D), device="cuda")[:, ::2]):
        mod = dict(gate=None, shift=None, scale=None)
        mod[which] = bad
        with pytest.raises(L.LensError) as ei:
            L.lens_op_sandwich_norm(t["h"], t["y"], L.LENS_BF16, M, D, 8, None, mod["gate"], None, mod["shift"],
                                    mod["scale"], D, RS, EPS, h_out, out, L.LENS_BF16)
        assert ei.value.status == 1
