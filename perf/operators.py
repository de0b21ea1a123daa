"""Workloads of the 8-bit and windowed single operations, for timing and comparison.

Four operators of one transformer block: quantization to e4m3 with a scale per block of
128 (`lens_op_quantize_f8`), the matrix product on such operands (`lens_op_gemm_f8`), the
norms after one branch and before the next fused with the gate and the residual scale
(`lens_op_sandwich_norm`), and attention over a window of keys with first tokens that stay
visible (`lens_op_attention_window`).

With `own` false, `run` evaluates an operator in elementary torch operations in fp32,
rounded once at the end; with `own` true it makes the library call.  `exact` evaluates
the definitions in fp64.
"""
import torch

own = False

GROUP = 128                 # values that share a scale along k (and rows of a weight block)
E4M3_MAX = 448.0
AMAX_FLOOR = 2.0 ** -116    # smallest amax a scale is made of
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f8": torch.float8_e4m3fn}


# ------------------------------------------------------------------ cases
def _quantize(rows, k, block_rows, x):
    return {"op": "quantize", "rows": rows, "k": k, "block_rows": block_rows, "x": x}


def _gemm(m, n, k, c, bias):
    return {"op": "gemm", "m": m, "n": n, "k": k, "c": c, "bias": bias}


def _norm(m, d, per_batch, y, out, post_gain, pre_gain, gate, mod):
    return {"op": "norm", "m": m, "d": d, "per_batch": per_batch, "y": y, "out": out, "post_gain": post_gain,
            "pre_gain": pre_gain, "gate": gate, "mod": mod}


def _attn(b, heads, kv_heads, n_q, n_kv, left, right, sinks, ragged):
    return {"op": "attn", "b": b, "heads": heads, "kv_heads": kv_heads, "n_q": n_q, "n_kv": n_kv, "left": left,
            "right": right, "sinks": sinks, "ragged": ragged}


def listed():
    return [
        # one row through the QKV projection: a conditioning vector or one decoded token
        dict(_gemm(1, 4608, 1536, "bf16", True), name="gemm 1x4608x1536"),
        # the text rows of a short prompt through the second MLP matrix, residual kept in fp32
        dict(_gemm(77, 1536, 4096, "f32", False), name="gemm 77x1536x4096 f32"),
        # a ragged batch with an inner size that ends inside a scale block
        dict(_gemm(1021, 2000, 2880, "bf16", True), name="gemm 1021x2000x2880"),
        # w1|w3 of a 1024^2 image with guidance (2 x 4352 tokens)
        dict(_gemm(8704, 8192, 1536, "bf16", False), name="gemm 8704x8192x1536"),
        # activations of an MLP, one scale per row and 128 columns
        dict(_quantize(4352, 4096, 1, "bf16"), name="quantize 4352x4096 rows"),
        # a weight matrix from fp32 masters, one scale per 128 x 128, ragged in both directions
        dict(_quantize(1000, 2896, 128, "f32"), name="quantize 1000x2896 blocks"),
        # text rows of one sample between two branches
        dict(_norm(77, 1536, 77, "bf16", "bf16", True, False, True, True), name="norm 77x1536"),
        # image and text rows of a guided 1024^2 sample, quantized for the next product
        dict(_norm(8704, 1536, 4352, "bf16", "f8", True, True, True, True), name="norm 8704x1536 f8"),
        # a wide model with an fp32 branch, no modulation
        dict(_norm(1021, 4096, 1021, "f32", "bf16", True, True, False, False), name="norm 1021x4096 f32"),
        # one new token per sequence against caches of different lengths, shared key heads
        dict(_attn(4, 24, 8, 1, 4352, 1023, 0, 4, True), name="attn 1 of 4352"),
        # causal prefill of padded sequences, shared key heads
        dict(_attn(3, 24, 8, 1999, 1999, 511, 0, 4, True), name="attn 1999 causal"),
        # a 1440^2 image: every token sees the 256 text tokens and a window on both sides
        dict(_attn(1, 24, 24, 8356, 8356, 1024, 1024, 256, False), name="attn 8356 window"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["quantize", "gemm", "gemm", "norm", "attn", "attn"])
    while True:
        if op == "quantize":
            c = _quantize(_log(rng, 1, 9000), 16 * _log(rng, 1, 720), rng.choice([1, 1, 128]), rng.choice(["f32", "bf16"]))
            if c["rows"] * c["k"] <= 4352 * 8192:
                return c
        elif op == "gemm":
            c = _gemm(_log(rng, 1, 9000), 16 * _log(rng, 1, 576), 16 * _log(rng, 4, 720), rng.choice(["f32", "bf16"]),
                      rng.random() < 0.5)
            if c["m"] * c["n"] * c["k"] <= 8704 * 8192 * 1536:
                return c
        elif op == "norm":
            m = _log(rng, 1, 9000)
            c = _norm(m, 16 * _log(rng, 4, 512), rng.choice([m, -(-m // 2), -(-m // 3)]), rng.choice(["f32", "bf16"]),
                      rng.choice(["bf16", "f8"]), rng.random() < 0.8, rng.random() < 0.5, rng.random() < 0.8,
                      rng.random() < 0.8)
            if c["m"] * c["d"] <= 8704 * 2048:
                return c
        else:
            kv_heads, group = rng.choice([1, 2, 4, 8, 24]), rng.choice([1, 1, 2, 3, 4, 8])
            n_kv = _log(rng, 1, 8400)
            n_q = rng.choice([1, _log(rng, 1, min(16, n_kv)), _log(rng, 1, n_kv), n_kv])
            c = _attn(rng.choice([1, 2, 3, 4]), kv_heads * group, kv_heads, n_q, n_kv, _log(rng, 1, 2048),
                      rng.choice([0, 0, _log(rng, 1, 2048)]), rng.choice([0, 1, 4, 128, 256]), rng.random() < 0.5)
            if c["heads"] <= 32 and c["b"] * c["heads"] * n_q * n_kv <= 24 * 8356 * 8356:
                return c


def _lengths(case):
    """Valid keys of each batch row and the position of its first query."""
    n_q, n_kv = case["n_q"], case["n_kv"]
    if not case["ragged"]:
        return [n_kv] * case["b"], [n_kv - n_q] * case["b"]
    lens = [max(1, n_kv - (i * n_kv) // (2 * case["b"])) for i in range(case["b"])]
    # whole sequences start at 0 with padding behind them; fewer queries than keys end at the cache's end
    return lens, [0 if n_q == n_kv else max(0, n - n_q) for n in lens]


def _visible(case):
    """Per batch row, the number of (query, key) pairs attended and of keys any query attends."""
    lens, starts = _lengths(case)
    pairs, keys = 0, 0
    for n, s in zip(lens, starts):
        p = torch.arange(s, s + case["n_q"])
        lo = (p - case["left"]).clamp(min=0)
        hi = (p + case["right"] + 1).clamp(max=n)
        window = (hi - lo).clamp(min=0)
        before = torch.minimum(lo, hi.clamp(min=0)).clamp(max=case["sinks"])     # sinks in front of the window
        pairs += int((window + before).sum())
        keys += int(min(n, case["sinks"] + max(0, int(hi.max()) - max(int(lo.min()), case["sinks"]))))
    return pairs, keys


def work(case):
    op = case["op"]
    size = {"f32": 4, "bf16": 2, "f8": 1}
    if op == "quantize":
        n = case["rows"] * case["k"]
        scales = -(-case["rows"] // case["block_rows"]) * -(-case["k"] // GROUP)
        return {"bytes": n * (size[case["x"]] + 1) + 4 * scales, "flops": 3 * n}
    if op == "gemm":
        m, n, k = case["m"], case["n"], case["k"]
        kb = -(-k // GROUP)
        return {"bytes": m * k + n * k + 4 * kb * (m + -(-n // GROUP)) + m * n * size[case["c"]] + 4 * n * case["bias"],
                "flops": 2 * m * n * k}
    if op == "norm":
        m, d = case["m"], case["d"]
        batches = -(-m // case["per_batch"])
        vectors = case["post_gain"] + case["pre_gain"] + batches * (case["gate"] + 2 * case["mod"])
        out = size[case["out"]] * d + (4 * -(-d // GROUP) if case["out"] == "f8" else 0)
        return {"bytes": m * (d * (8 + size[case["y"]]) + out) + 4 * vectors * d, "flops": 12 * m * d}
    pairs, keys = _visible(case)
    rows = case["b"] * case["n_q"] * case["heads"]
    return {"bytes": 2 * 64 * (2 * rows + 2 * keys * case["kv_heads"]), "flops": 4 * 64 * pairs * case["heads"]}


# ------------------------------------------------------------------ inputs
def _padded(x, block_rows):
    """x zero-padded to whole blocks, as [row blocks, block_rows, k blocks, 128]."""
    r, k = x.shape
    x = torch.nn.functional.pad(x, (0, -k % GROUP, 0, -r % block_rows))
    return x.reshape(x.shape[0] // block_rows, block_rows, x.shape[1] // GROUP, GROUP)


def _quantized(x, block_rows):
    """(e4m3 codes [rows, k], fp32 scales [k blocks, row blocks]) of fp32 x."""
    b = _padded(x, block_rows)
    amax = b.abs().amax(dim=(1, 3), keepdim=True).clamp(min=AMAX_FLOOR)
    codes = (b * (E4M3_MAX / amax)).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    codes = codes.reshape(b.shape[0] * block_rows, -1)[:x.shape[0], :x.shape[1]].contiguous()
    return codes, (amax / E4M3_MAX)[:, 0, :, 0].t().contiguous()


def _widened(codes, scales, block_rows, dtype):
    """The values that codes and scales stand for."""
    s = scales.to(dtype).t().repeat_interleave(block_rows, 0).repeat_interleave(GROUP, 1)
    return codes.to(dtype) * s[:codes.shape[0], :codes.shape[1]]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))

    def normal(*shape, std=1.0, dtype=torch.float32):
        return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)

    def empty(*shape, dtype=torch.float32):
        return torch.empty(shape, dtype=dtype, device="cuda")

    op, s = case["op"], {"case": case}
    if op == "quantize":
        rows, k = case["rows"], case["k"]
        # activations have columns of very different size, weights have not
        spread = torch.exp(normal(k)) if case["block_rows"] == 1 else 0.02
        s["x"] = (normal(rows, k) * spread).to(DTYPES[case["x"]])
        s["codes"] = empty(rows, k, dtype=torch.uint8)
        s["scales"] = empty(-(-k // GROUP), -(-rows // case["block_rows"]))
    elif op == "gemm":
        m, n, k = case["m"], case["n"], case["k"]
        s["a"], s["a_scales"] = _quantized(normal(m, k) * torch.exp(0.5 * normal(k)), 1)
        s["w"], s["w_scales"] = _quantized(normal(n, k, std=0.02), GROUP)
        s["bias"] = normal(n) if case["bias"] else None
        s["c"] = empty(m, n, dtype=DTYPES[case["c"]])
    elif op == "norm":
        m, d = case["m"], case["d"]
        batches = -(-m // case["per_batch"])
        s["h"], s["y"] = normal(m, d, std=3.0), normal(m, d, dtype=DTYPES[case["y"]])
        s["post_gain"] = 1 + normal(d, std=0.1) if case["post_gain"] else None
        s["pre_gain"] = 1 + normal(d, std=0.1) if case["pre_gain"] else None
        mod = normal(batches, 3, d, std=0.3)      # gate, shift, scale of each sample
        s["gate"] = mod[:, 0] if case["gate"] else None
        s["shift"], s["scale"] = (mod[:, 1], mod[:, 2]) if case["mod"] else (None, None)
        s["h_out"] = empty(m, d)
        s["out"] = empty(m, d, dtype=DTYPES[case["out"]])
        s["out_scales"] = empty(-(-d // GROUP), m) if case["out"] == "f8" else None
    else:
        b, h, hk = case["b"], case["heads"], case["kv_heads"]
        s["q"] = normal(b, h, case["n_q"], 64, std=1.5, dtype=torch.bfloat16)
        s["k"] = normal(b, hk, case["n_kv"], 64, std=1.5, dtype=torch.bfloat16)
        s["v"] = normal(b, hk, case["n_kv"], 64, dtype=torch.bfloat16)
        s["kv_len"], s["q_start"] = _lengths(case)
        s["out"] = empty(b, case["n_q"], h * 64, dtype=torch.bfloat16)
    return s


RESIDUAL_SCALE, EPS, SOFTMAX_SCALE = 0.75, 1e-6, 0.125


# ------------------------------------------------------------------ one pass
def run(s):
    case = s["case"]
    if own:
        return _run_own(case, s)
    return {"quantize": _plain_quantize, "gemm": _plain_gemm, "norm": _plain_norm, "attn": _plain_attn}[case["op"]](case, s)


def _run_own(case, s):
    import flow_matching_mmdit_b200 as L
    kind = {"f32": L.LENS_F32, "bf16": L.LENS_BF16, "f8": L.LENS_F8E4M3}
    if case["op"] == "quantize":
        L.lens_op_quantize_f8(s["x"], kind[case["x"]], case["rows"], case["k"], case["block_rows"], s["codes"], s["scales"])
        return s["codes"].view(torch.float8_e4m3fn), s["scales"]
    if case["op"] == "gemm":
        L.lens_op_gemm_f8(s["a"], s["a_scales"], s["w"], s["w_scales"], s["bias"], s["c"], kind[case["c"]], case["m"],
                          case["n"], case["k"])
        return s["c"]
    if case["op"] == "norm":
        L.lens_op_sandwich_norm(s["h"], s["y"], kind[case["y"]], case["m"], case["d"], case["per_batch"], s["post_gain"],
                                s["gate"], s["pre_gain"], s["shift"], s["scale"], 3 * case["d"], RESIDUAL_SCALE, EPS,
                                s["h_out"], s["out"], kind[case["out"]], s["out_scales"])
        return s["h_out"], s["out"], s["out_scales"]
    L.lens_op_attention_window(s["q"], s["k"], s["v"], case["b"], case["heads"], case["kv_heads"], case["n_q"],
                               case["n_kv"], s["q_start"], s["kv_len"], case["left"], case["right"], case["sinks"],
                               SOFTMAX_SCALE, s["out"])
    return s["out"]


def _plain_quantize(case, s):
    return _quantized(s["x"].float(), case["block_rows"])


def _plain_gemm(case, s):
    c = _widened(s["a"], s["a_scales"], 1, torch.float32) @ _widened(s["w"], s["w_scales"], GROUP, torch.float32).t()
    if s["bias"] is not None:
        c = c + s["bias"]
    return c.to(DTYPES[case["c"]])


def _rows(v, case):
    """A per-sample [batches, d] vector as one row per row of the call."""
    return v.repeat_interleave(case["per_batch"], 0)[:case["m"]]


def _plain_norm(case, s):
    y = s["y"].float()
    y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + EPS)
    if s["post_gain"] is not None:
        y = y * s["post_gain"]
    if s["gate"] is not None:
        y = y * _rows(s["gate"], case)
    h = RESIDUAL_SCALE * s["h"] + y
    x = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + EPS)
    if s["pre_gain"] is not None:
        x = x * s["pre_gain"]
    if s["scale"] is not None:
        x = (1 + _rows(s["scale"], case)) * x + _rows(s["shift"], case)
    if case["out"] == "f8":
        codes, scales = _quantized(x, 1)
        return h, codes, scales
    return h, x.to(torch.bfloat16), None


def _mask(case, s, device):
    """[b, n_q, n_kv]: whether a query attends a key."""
    start = torch.tensor(s["q_start"], device=device)[:, None, None]
    length = torch.tensor(s["kv_len"], device=device)[:, None, None]
    p = start + torch.arange(case["n_q"], device=device)[None, :, None]
    j = torch.arange(case["n_kv"], device=device)[None, None, :]
    return (j < length) & (j <= p + case["right"]) & ((j >= p - case["left"]) | (j < case["sinks"]))


def _plain_attn(case, s):
    b, h, hk, n = case["b"], case["heads"], case["kv_heads"], case["n_q"]
    q = s["q"].float().reshape(b, hk, h // hk, n, 64)
    scores = q @ s["k"].float()[:, :, None].transpose(-1, -2) * SOFTMAX_SCALE
    scores = scores.masked_fill(~_mask(case, s, scores.device)[:, None, None], float("-inf"))
    top = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - torch.where(torch.isinf(top), torch.zeros_like(top), top))
    total = p.sum(-1, keepdim=True)
    o = p @ s["v"].float()[:, :, None] / torch.where(total > 0, total, torch.ones_like(total))
    return o.permute(0, 3, 1, 2, 4).reshape(b, n, h * 64).to(torch.bfloat16)


# ------------------------------------------------------------------ the definitions in fp64
def _e4m3_nearest(v):
    """The e4m3 value nearest to fp64 v (ties to even), saturating at 448."""
    _, e = torch.frexp(v.abs())                       # |v| in [2^(e-1), 2^e)
    step = torch.exp2((e - 1).clamp(min=-6).double() - 3)
    return (torch.round(v / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def _exact_codes(x, block_rows):
    r, k = x.shape
    codes = torch.empty_like(x)
    scales = torch.empty(-(-k // GROUP), -(-r // block_rows), dtype=torch.float64, device=x.device)
    for kb in range(scales.shape[0]):
        cols = x[:, kb * GROUP:(kb + 1) * GROUP]
        top = cols.abs().amax(1)
        top = torch.stack([t.amax() for t in top.split(block_rows)]) if block_rows > 1 else top
        scales[kb] = top.clamp(min=AMAX_FLOOR) / E4M3_MAX
        codes[:, kb * GROUP:(kb + 1) * GROUP] = _e4m3_nearest(cols / scales[kb].repeat_interleave(block_rows)[:r, None])
    return codes, scales


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "quantize":
        return _exact_codes(s["x"].double(), case["block_rows"])
    if case["op"] == "gemm":
        c = torch.zeros(case["m"], case["n"], dtype=torch.float64, device="cuda")
        for kb in range(s["a_scales"].shape[0]):
            cols = slice(kb * GROUP, (kb + 1) * GROUP)
            a = s["a"][:, cols].double() * s["a_scales"][kb].double()[:, None]
            w = s["w"][:, cols].double() * s["w_scales"][kb].double().repeat_interleave(GROUP)[:case["n"], None]
            c += a @ w.t()
        return c if s["bias"] is None else c + s["bias"].double()
    if case["op"] == "norm":
        d = case["d"]
        of = torch.arange(case["m"], device="cuda") // case["per_batch"]
        one, none = torch.ones(d, dtype=torch.float64, device="cuda"), torch.zeros(d, dtype=torch.float64, device="cuda")
        post = one if s["post_gain"] is None else s["post_gain"].double()
        pre = one if s["pre_gain"] is None else s["pre_gain"].double()
        gate = one if s["gate"] is None else s["gate"].double()[of]
        scale, shift = (none, none) if s["scale"] is None else (s["scale"].double()[of], s["shift"].double()[of])
        y = s["y"].double()
        h = RESIDUAL_SCALE * s["h"].double() + gate * post * y / torch.sqrt((y * y).sum(1, keepdim=True) / d + EPS)
        x = (1 + scale) * pre * h / torch.sqrt((h * h).sum(1, keepdim=True) / d + EPS) + shift
        if case["out"] == "f8":
            return (h,) + _exact_codes(x, 1)
        return h, x, None
    b, h, hk, n = case["b"], case["heads"], case["kv_heads"], case["n_q"]
    o = torch.zeros(b, n, h, 64, dtype=torch.float64, device="cuda")
    j = torch.arange(case["n_kv"], device="cuda")
    for i in range(b):
        p = torch.arange(n, device="cuda")[:, None] + s["q_start"][i]
        seen = (j >= p - case["left"]) | (j < case["sinks"])
        seen = seen & (j <= p + case["right"]) & (j < s["kv_len"][i])
        some = seen.any(1, keepdim=True)
        for a in range(h):
            key, value = s["k"][i, a * hk // h].double(), s["v"][i, a * hk // h].double()
            z = torch.where(seen, s["q"][i, a].double() @ key.t() * SOFTMAX_SCALE, -torch.inf)
            e = torch.softmax(torch.where(some, z, 0.0), 1)
            o[i, :, a] = torch.where(some, e @ value, 0.0)
    return o.reshape(b, n, h * 64)
