"""GPU tests of windowed attention beside test_gpu_window.py: caches longer than what they hold,
and non-finite values in attended places."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import flow_matching_mmdit_b200 as L  # noqa: E402
from tests.test_gpu_window import check, make, mask_of, run  # noqa: E402


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


@pytest.mark.parametrize("sinks", [16, 17, 40, 100, 127, 128, 129])
@pytest.mark.parametrize("B,H,Hk,n_q,n_kv,left,right", [(1, 2, 1, 600, 600, 60, 0), (2, 3, 3, 300, 700, 130, 40),
                                                        (1, 4, 2, 20, 900, 100, 0), (1, 2, 2, 260, 260, 0, 0)])
def test_sinks_around_a_key_tile(B, H, Hk, n_q, n_kv, left, right, sinks):
    """Up to 16 sinks are a tile of their own size, more of them a masked tile of 128, or two."""
    q, k, v = make(B, H, Hk, n_q, n_kv, sinks)
    length = [n_kv - 37 * b for b in range(B)]
    start = [n - n_q for n in length]
    check(run(q, k, v, start, length, left, right, sinks), q, k, v, start, length, left, right, sinks)


@pytest.mark.parametrize("n_q,n_kv", [(1, 2000), (40, 900), (300, 300)])
def test_the_same_bits_from_a_side_stream_and_beside_other_work(n_q, n_kv):
    q, k, v = make(2, 6, 2, n_q, n_kv, 14)
    start = [n_kv - n_q, n_kv - n_q]
    want = run(q, k, v, start, None, 70, 0, 4).clone()
    outs = [torch.full_like(want, -7.0) for _ in range(6)]
    torch.cuda.synchronize()                        # the fills come before the streams' work
    streams = [torch.cuda.Stream() for _ in range(3)]
    for i, o in enumerate(outs):
        L.lens_op_attention_window(q, k, v, 2, 6, 2, n_q, n_kv, start, None, 70, 0, 4, 0.125, o, stream=streams[i % 3])
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)


def expected(q, k, v, start, length, left, right, sinks, b, h):
    """(fp64 output, sum p |v|) of one head with every non-finite value of V taken as 0, and the
    output's infinities and NaNs: what the attended values of a column sum to, where it is not
    finite (their weights are positive: scores here are small)."""
    kv = h * k.shape[1] // q.shape[1]
    m = mask_of(q.shape[2], k.shape[2], start[b], length[b], left, right, sinks)
    some = m.any(1, keepdim=True)
    # (masked before the exponential: K may hold anything at keys that are not attended)
    s = torch.where(m, q[b, h].double() @ k[b, kv].double().t() * 0.125, -torch.inf)
    p = torch.where(some, torch.softmax(torch.where(some, s, 0.0), 1), 0.0)
    vv = v[b, kv].double()
    finite = torch.where(torch.isfinite(vv), vv, 0.0)
    md = m.double()
    nan = (md @ torch.isnan(vv).double() > 0) | torch.isnan(p).any(1, keepdim=True)
    plus, minus = md @ (vv == torch.inf).double() > 0, md @ (vv == -torch.inf).double() > 0
    special = torch.where(plus, torch.inf, 0.0) + torch.where(minus, -torch.inf, 0.0)
    return p @ finite, p @ finite.abs(), torch.where(nan, torch.nan, special)


def check_special(out, q, k, v, start, length, left, right, sinks):
    """Non-finite exactly where, and as, the attended values make it; the rest within the bound of
    test_gpu_window.check."""
    n_special = n_finite = 0
    for b in range(q.shape[0]):
        for h in range(q.shape[1]):
            ref, mag, special = expected(q, k, v, start, length, left, right, sinks, b, h)
            got = out[b, :, h * 64:(h + 1) * 64].double()
            is_special = special != 0
            assert torch.equal(torch.nan_to_num(got[is_special], 5.0, 6.0, 7.0),
                               torch.nan_to_num(special[is_special], 5.0, 6.0, 7.0)), (b, h)
            err = (got - ref).abs()[~is_special]
            tol = (2.0 ** -8 * (mag + ref.abs()) + 2.0 ** -13 * mag)[~is_special]
            assert bool((err <= tol).all()), (b, h, float((err - tol).max()))
            n_special, n_finite = n_special + int(is_special.sum()), n_finite + int((~is_special).sum())
    return n_special, n_finite


SPECIALS = [(1, 4, 2, 300, 300, 40, 0, 3), (2, 3, 1, 500, 500, 60, 60, 20), (1, 2, 2, 130, 900, 100, 30, 130),
            (2, 8, 2, 1, 700, 300, 0, 4), (1, 6, 2, 9, 400, 5, 3, 1), (1, 4, 4, 48, 1500, -1, 0, 0),
            (1, 2, 1, 200, 333, -1, -1, 0), (1, 3, 3, 17, 64, 0, 0, 16)]


@pytest.mark.parametrize("B,H,Hk,n_q,n_kv,left,right,sinks", SPECIALS)
@pytest.mark.parametrize("density", ["one", "few", "many"])
def test_non_finite_values_that_are_attended(B, H, Hk, n_q, n_kv, left, right, sinks, density):
    """Infinities of both signs and NaNs in V, in sinks, windows and places that nobody attends."""
    q, k, v = make(B, H, Hk, n_q, n_kv, 31 + n_q)
    length = [n_kv - 11 * b for b in range(B)]
    start = [max(0, n - n_q) for n in length]
    g = torch.Generator(device="cuda")
    g.manual_seed(n_kv)
    if density == "one":
        v[0, 0, start[0] + n_q // 2, 5] = float("inf")
    else:
        share = 0.001 if density == "few" else 0.02
        hit = torch.rand(v.shape, generator=g, device="cuda") < share
        hit[:, :, :, 7] = False                                # a column that stays finite
        what = torch.tensor([float("inf"), -float("inf"), float("nan")], device="cuda").to(torch.bfloat16)
        v = torch.where(hit, what[torch.randint(0, 3, v.shape, generator=g, device="cuda")], v)
    out = run(q, k, v, start, length, left, right, sinks)
    n_special, n_finite = check_special(out, q, k, v, start, length, left, right, sinks)
    assert n_special > 0 and n_finite > 0


@pytest.mark.parametrize("n_q", [2, 200])
def test_a_nan_score_makes_its_rows_nan_and_no_others(n_q):
    n_kv, left = 400, 30
    q, k, v = make(1, 2, 1, n_q, n_kv, 33)
    start = [n_kv - n_q]
    j = start[0] + n_q // 2
    k[0, 0, j, 9] = float("nan")
    v[0, 0, j + 1 if n_q > 2 else j, 3] = float("inf")
    out = run(q, k, v, start, [n_kv], left, 0, 2).view(n_q, 2, 64)
    seen = mask_of(n_q, n_kv, start[0], n_kv, left, 0, 2)[:, j]
    assert bool(torch.isnan(out[seen]).all()) and not bool(torch.isnan(out[~seen]).any())
    check_special(out.view(1, n_q, 128), q, k, v, start, [n_kv], left, 0, 2)


def test_a_row_that_attends_nothing_is_zero_beside_non_finite_values():
    q, k, v = make(1, 2, 2, 300, 300, 34)
    v[0, :, 140:, :] = float("nan")
    out = run(q, k, v, [0], [150], 20, 0, 0).view(300, 128)
    assert not bool(out[170:].any()) and bool(torch.isfinite(out[:140]).all()) and bool(torch.isnan(out[140:170]).all())


def _time_us(call):
    for _ in range(3):
        call()
    best = []
    for _ in range(5):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        call()
        b.record()
        torch.cuda.synchronize()
        best.append(a.elapsed_time(b) * 1e3)
    return min(best)


@pytest.mark.parametrize("n_q,n_kv,left,right,sinks", [(4096, 4096, 1024, 1024, 256), (4096, 4096, 300, 0, 4),
                                                       (1, 100000, -1, 0, 0)])
def test_a_non_finite_value_that_all_rows_attend_costs_a_few_calls(n_q, n_kv, left, right, sinks):
    """One infinity in a key that every row attends.  Rows are done again sixteen at a time from
    their own keys: a few times the call, where one key of one row at a time takes hundreds.  The
    bound leaves room for a busy host."""
    q, k, v = make(1, 24, 24, n_q, n_kv, 35)
    out = torch.empty((1, n_q, 24 * 64), dtype=torch.bfloat16, device="cuda")

    def call():
        L.lens_op_attention_window(q, k, v, 1, 24, 24, n_q, n_kv, [n_kv - n_q], None, left, right, sinks, 0.125, out)

    clean = _time_us(call)
    v[:, :, 0 if sinks else n_kv - 1, 5] = float("inf")
    slow = _time_us(call)
    print(f"clean {clean:.0f} us, with an infinity {slow:.0f} us")
    assert bool((out.view(n_q, 24, 64)[-1, :, 5] == float("inf")).all())
    assert slow <= 15 * clean + 50, (clean, slow)
