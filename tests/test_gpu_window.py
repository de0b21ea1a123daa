"""GPU parity of windowed attention against the fp64 oracle: masks, lengths, shared key
heads, few queries against a long cache, and values in places that are not attended."""
import numpy as np
import pytest

from oracle import ops_oracle as oo
from tests.test_gpu_f8 import guarded

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import flow_matching_mmdit_b200 as L  # noqa: E402

SCALE = 0.125


@pytest.fixture(scope="module", autouse=True)
def cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    L.load_library()


def make(B, H, Hk, nq, nkv, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*s, std=1.0):
        return (torch.randn(s, generator=g, device="cuda") * std).to(torch.bfloat16)

    return normal(B, H, nq, 64, std=1.5), normal(B, Hk, nkv, 64, std=1.5), normal(B, Hk, nkv, 64)


def run(q, k, v, start, length, left, right, sinks, scale=SCALE, stream=None):
    B, H, nq, _ = q.shape
    out, ok = guarded((B, nq, H * 64), torch.bfloat16, -7.0)
    L.lens_op_attention_window(q, k, v, B, H, k.shape[1], nq, k.shape[2], start, length, left, right, sinks, scale, out,
                               stream=stream)
    torch.cuda.synchronize()
    ok()
    return out


def mask_of(nq, nkv, start, length, left, right, sinks, device="cuda"):
    p = start + torch.arange(nq, device=device)[:, None]
    j = torch.arange(nkv, device=device)[None]
    m = (j < length).expand(nq, nkv).clone()
    if right >= 0:
        m &= j <= p + right
    if left >= 0:
        m &= (j >= p - left) | (j < sinks)
    return m


def check(out, q, k, v, start, length, left, right, sinks, scale=SCALE, heads=None):
    """Against fp64.  The weights are rounded to bf16 before they meet the values (2^-8 of
    sum p |v|) and so is the output (2^-8 of it); the exponentials are good to 2^-21 and their
    arguments to 2^-23 of a score of at most 64, the sums to 2^-14 with room."""
    B, H, nq, _ = q.shape
    for b in range(B):
        m = mask_of(nq, k.shape[2], start[b] if start else 0, length[b] if length else k.shape[2], left, right, sinks)
        some = m.any(1, keepdim=True)
        for h in heads or range(H):
            kv = h * k.shape[1] // H
            s = torch.where(m, q[b, h].double() @ k[b, kv].double().t() * scale, -torch.inf)
            p = torch.where(some, torch.softmax(torch.where(some, s, 0.0), 1), 0.0)
            vv = v[b, kv].double()
            ref, mag = p @ vv, p @ vv.abs()
            got = out[b, :, h * 64:(h + 1) * 64].double()
            err, tol = (got - ref).abs(), 2.0 ** -8 * (mag + ref.abs()) + 2.0 ** -13 * mag
            assert bool((err <= tol).all()), (b, h, float((err - tol).max()))
            assert not bool(got[~some[:, 0]].any())


@pytest.mark.parametrize("B,H,Hk,nq,nkv,start,length,left,right,sinks", [
    (1, 1, 1, 1, 1, None, None, 0, 0, 0),
    (2, 3, 3, 5, 5, None, [5, 2], -1, -1, 0),                     # no window, padding
    (1, 24, 24, 64, 64, None, None, 7, 7, 4),
    (2, 4, 2, 130, 130, None, [130, 77], 31, 0, 4),               # causal, padded
    (1, 2, 1, 257, 257, None, None, 64, 64, 16),
    (1, 3, 1, 300, 300, None, None, 1000, 1000, 0),               # the window covers all
    (2, 2, 2, 256, 384, [128, 0], [384, 256], 100, 20, 130),      # sinks past the first key tile
    (1, 2, 2, 700, 700, None, None, 0, 0, 0),                     # every token sees itself alone
    (1, 2, 2, 513, 1100, [587], None, 200, 0, 1),
    (1, 1, 1, 900, 900, None, [450], 50, 10, 3),                  # rows far past the end see the sinks only
    (1, 1, 1, 900, 900, None, [450], 50, 10, 0),                  # and without sinks nothing
    (2, 2, 1, 300, 300, None, [0, 1], 50, 0, 4),                  # no key, one key
    (1, 2, 2, 128, 5000, [100000], None, 200000, 0, 0),           # positions behind the cache's end
    (1, 2, 2, 128, 5000, [100000], None, 20, 0, 7),
    (1, 8, 1, 1500, 1500, None, None, 255, 255, 256),
    (1, 2, 2, 2100, 2100, None, None, 128, 512, 0),
    (1, 2, 2, 600, 600, None, None, -1, 0, 3),                    # causal without a window
    (1, 2, 2, 600, 600, None, None, 5, -1, 3),                    # everything after
])
def test_window_attention(B, H, Hk, nq, nkv, start, length, left, right, sinks):
    q, k, v = make(B, H, Hk, nq, nkv, nq + nkv)
    check(run(q, k, v, start, length, left, right, sinks), q, k, v, start, length, left, right, sinks)


@pytest.mark.parametrize("H,Hk", [(1, 1), (6, 2), (8, 1), (24, 8), (32, 1), (33, 3)])
@pytest.mark.parametrize("nq,nkv,left,sinks", [(1, 1, 0, 0), (1, 17, 5, 1), (1, 1000, 255, 4), (2, 4100, 1023, 4),
                                               (5, 4100, -1, 0), (16, 777, 100, 130), (17, 777, 100, 130)])
def test_few_queries_against_a_cache(H, Hk, nq, nkv, left, sinks):
    """The newest tokens of sequences of different lengths, causal."""
    B = 3
    length = [nkv, max(1, nkv // 2), max(1, nkv - 1)]
    start = [max(0, n - nq) for n in length]
    q, k, v = make(B, H, Hk, nq, nkv, H + nq + nkv)
    check(run(q, k, v, start, length, left, 0, sinks), q, k, v, start, length, left, 0, sinks)


@pytest.mark.parametrize("H,Hk", [(1, 1), (16, 4), (32, 8), (9, 9), (12, 12)])
@pytest.mark.parametrize("nq,nkv", [(1, 2500), (3, 9001), (1, 20000)])
def test_few_queries_against_all_of_a_long_cache(H, Hk, nq, nkv):
    q, k, v = make(1, H, Hk, nq, nkv, H + nkv)
    check(run(q, k, v, [nkv - nq], None, -1, 0, 0), q, k, v, [nkv - nq], None, -1, 0, 0)
    check(run(q, k, v, [nkv - nq], [nkv - 70], -1, 0, 5), q, k, v, [nkv - nq], [nkv - 70], -1, 0, 5)


@pytest.mark.parametrize("B,H,Hk,nkv", [(40, 24, 24, 700), (64, 8, 8, 1100), (20, 16, 4, 2300)])
def test_one_query_in_large_batches(B, H, Hk, nkv):
    """Enough tiles for the keys to be split over fewer CTAs, down to one."""
    g = np.random.default_rng(B)
    length = [int(g.integers(0, nkv + 1)) for _ in range(B)]
    start = [max(0, n - 1) for n in length]
    q, k, v = make(B, H, Hk, 1, nkv, B)
    for left in (-1, 500, 100):
        check(run(q, k, v, start, length, left, 0, 4), q, k, v, start, length, left, 0, 4, heads=[0, H - 1])


@pytest.mark.parametrize("nq", [1, 7, 300])
@pytest.mark.parametrize("what", [float("nan"), float("inf"), -3e38])
def test_values_in_places_that_are_not_attended_have_no_effect(nq, what):
    """Padding behind a sequence and evicted tokens between the sinks and the window may hold
    anything, inside the tiles that are read."""
    B, H, Hk, nkv, left, sinks = 2, 4, 2, 500, 40, 3
    length, start = [500, 321], [500 - nq, 321 - nq if nq < 321 else 0]
    q, k, v = make(B, H, Hk, nq, nkv, 9)
    want = run(q, k, v, start, length, left, 0, sinks)
    k2, v2 = k.clone(), v.clone()
    for b in range(B):
        seen = mask_of(nq, nkv, start[b], length[b], left, 0, sinks).any(0)
        k2[b][:, ~seen], v2[b][:, ~seen] = what, what
    assert torch.equal(run(q, k2, v2, start, length, left, 0, sinks), want)


@pytest.mark.parametrize("nq", [6, 300])
def test_a_non_finite_value_reaches_only_the_rows_that_attend_it(nq):
    nkv, left = 400, 30
    q, k, v = make(1, 2, 1, nq, nkv, 10)
    start = [nkv - nq]
    want = run(q, k, v, start, None, left, 0, 2)
    j = start[0] + nq // 2
    v2 = v.clone()
    v2[0, 0, j, 5] = float("inf")
    got = run(q, k, v2, start, None, left, 0, 2)
    seen = mask_of(nq, nkv, start[0], nkv, left, 0, 2)[:, j]
    assert bool(seen.any()) and not bool(seen.all())
    # the other rows' values may come from another order of summation: held to the bound
    finite = got[:, ~seen]
    assert bool(torch.isfinite(finite.float()).all())
    err = (finite.double() - want[:, ~seen].double()).abs()
    assert bool((err <= 2.0 ** -6 * (1 + want[:, ~seen].double().abs())).all())
    col = got.view(1, nq, 2, 64)[0, seen]
    assert bool((col[:, :, 5] == float("inf")).all())


@pytest.mark.parametrize("nq", [1, 200])
def test_large_scores(nq):
    """Scores of several hundred: the running maximum carries the softmax."""
    q, k, v = make(1, 2, 2, nq, 600, 12)
    q, k = q * 8, k * 4
    # fp32 scores of up to 2000 are off by 2^-13 at most: exponentials by 1.2e-4
    out = run(q, k, v, [600 - nq], None, 300, 0, 4)
    m = mask_of(nq, 600, 600 - nq, 600, 300, 0, 4)
    for h in range(2):
        s = torch.where(m, q[0, h].double() @ k[0, h].double().t() * SCALE, -torch.inf)
        p = torch.softmax(s, 1)
        ref, mag = p @ v[0, h].double(), p @ v[0, h].double().abs()
        err = (out[0, :, h * 64:(h + 1) * 64].double() - ref).abs()
        assert bool((err <= 2.0 ** -8 * (mag + ref.abs()) + 2.0 ** -11 * mag).all())


@pytest.mark.parametrize("nq,nkv", [(1, 2000), (300, 300)])
def test_rows_do_not_depend_on_the_batch_streams_or_graphs(nq, nkv):
    # (for few queries: while the batch leaves the split of the keys as it is)
    B, left, sinks = 3, 70, 4
    q, k, v = make(B, 6, 2, nq, nkv, 14)
    length = [nkv, nkv - 3, nkv // 2]
    start = [0] * B if nq == nkv else [n - nq for n in length]
    want = run(q, k, v, start, length, left, 0, sinks).clone()
    for b in range(B):
        one = run(q[b:b + 1], k[b:b + 1], v[b:b + 1], start[b:b + 1], length[b:b + 1], left, 0, sinks)
        assert torch.equal(one[0], want[b])
    side = torch.cuda.Stream()
    assert torch.equal(run(q, k, v, start, length, left, 0, sinks, stream=side), want)
    out = torch.zeros_like(want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        L.lens_op_attention_window(q, k, v, B, 6, 2, nq, nkv, start, length, left, 0, sinks, SCALE, out)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_a_long_cache_passes_32_bit_offsets():
    """The last key head of a cache of more than 2^31 values."""
    Hk, nkv = 9, 4_000_000
    k = torch.zeros((1, Hk, nkv, 64), dtype=torch.bfloat16, device="cuda")
    v = torch.zeros((1, Hk, nkv, 64), dtype=torch.bfloat16, device="cuda")
    q, ks, vs = make(1, Hk, Hk, 1, 300, 15)
    k[:, :, -300:], v[:, :, -300:] = ks, vs
    out = run(q, k, v, [nkv - 1], None, 299, 0, 0)
    assert torch.equal(out, run(q, ks, vs, [299], None, 299, 0, 0))
    q2 = make(1, Hk, Hk, 100, 300, 16)[0]
    out = run(q2, k, v, [nkv - 100], None, 199, 0, 0)
    check(out, q2, ks, vs, [200], None, 199, 0, 0)


def test_joint_tokens_with_an_unbounded_window_are_joint_attention():
    """Beside lens_op_attention: text first, every token attends every token."""
    B, nt, ni = 2, 77, 200
    q, k, v = make(B, 24, 24, nt + ni, nt + ni, 17)
    ot = torch.zeros((B, nt, 1536), dtype=torch.bfloat16, device="cuda")
    oi = torch.zeros((B, ni, 1536), dtype=torch.bfloat16, device="cuda")
    L.lens_op_attention(q, k, v, B, nt, ni, ot, oi)
    got = run(q, k, v, None, None, -1, -1, 0)
    both = torch.cat([ot, oi], 1).double()
    # two kernels, each within 2^-8 of sum p |v| and of its value (at most 4.5 here)
    assert bool(((got.double() - both).abs() <= 2 * 2.0 ** -8 * (1.3 + both.abs())).all())
