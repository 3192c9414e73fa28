"""The operators around an MoE step's expert side: what is measured of them.

Three operators and the path that they stand on:

  gemm  products grouped by expert with ragged row counts (bf16, or fp8 e4m3
        with one scale per 128 activations and per 128 x 128 weights), plain
        or with the gated activation silu(gate) * up, out in bf16 or in fp8
        with a scale per 128 columns
  w4    the same products with 4-bit weights: groups of 32, 64 or 128 along k
        share a bf16 scale and, if there are any, an 8-bit zero point
  norm  root-mean-square norm of x plus the residual, out in bf16 or in fp8
        with a scale per 128 columns, and the new residual

Rows stand as the dispatch's expert side leaves them: expert e owns rows
[e * max_tokens, (e + 1) * max_tokens) and fills the first counts[e]. Rows
behind are poisoned with NaN on the way in and keep their zeros on the way
out.
"""
import numpy as np
import torch

own = False

DEV = "cuda:0"
FP8 = torch.float8_e4m3fn
BLOCK = 128
EPS = 1e-6


def listed():
    return [
        # a decode batch of 128 tokens over 256 experts, first product with the
        # activation: about 4 rows an expert, all weights read for them
        dict(name="gemm decode fp8 gated", op="gemm", tokens=128, experts=256, topk=8, routing="uniform",
             n=2048, k=7168, dtype="fp8", gated=True, out="fp8"),
        # one token alone: the latency that a user waits for, 8 of 256 experts
        dict(name="gemm one token bf16 gated", op="gemm", tokens=1, experts=256, topk=8, routing="uniform",
             n=2048, k=7168, dtype="bf16", gated=True, out="bf16"),
        # the smallest layer: 8 small experts, launch latency
        dict(name="gemm tiny bf16 gated", op="gemm", tokens=128, experts=8, topk=2, routing="uniform",
             n=512, k=1024, dtype="bf16", gated=True, out="bf16"),
        # skewed routing, second product: some experts with hundreds of rows, some with few
        dict(name="gemm zipf bf16 down", op="gemm", tokens=512, experts=64, topk=6, routing="zipf",
             n=4096, k=1536, dtype="bf16", gated=False, out="bf16"),
        # a prompt's tokens over few experts: bound by the matrix cores
        dict(name="gemm prompt bf16 gated", op="gemm", tokens=8192, experts=8, topk=2, routing="uniform",
             n=2048, k=4096, dtype="bf16", gated=True, out="bf16"),
        # half of 1024 tokens on 8 hot experts, second product in fp8
        dict(name="gemm hot fp8 down", op="gemm", tokens=1024, experts=256, topk=8, routing="hotset",
             n=7168, k=2048, dtype="fp8", gated=False, out="bf16"),
        # the decode batch with 4-bit weights
        dict(name="w4 decode gated", op="w4", tokens=128, experts=256, topk=8, routing="uniform",
             n=2048, k=7168, group=128, zeros=False, gated=True),
        # one token with 4-bit weights: matrix-vector products of 8 experts
        dict(name="w4 one token gated", op="w4", tokens=1, experts=64, topk=8, routing="uniform",
             n=1536, k=4096, group=32, zeros=True, gated=True),
        # skewed routing with 4-bit weights, second product
        dict(name="w4 zipf down", op="w4", tokens=512, experts=64, topk=6, routing="zipf",
             n=4096, k=1536, group=64, zeros=False, gated=False),
        # the norm in front of a layer for one token: latency
        dict(name="norm one token fp8", op="norm", tokens=1, hidden=7168, x="bf16", residual=True, out="fp8"),
        # a decode batch: the combine's fp32 output joins the residual
        dict(name="norm decode fp32", op="norm", tokens=128, hidden=7168, x="fp32", residual=True, out="bf16"),
        # a prompt's tokens: bound by memory
        dict(name="norm prompt fp8", op="norm", tokens=16384, hidden=7168, x="bf16", residual=True, out="fp8"),
    ]


def _spread(rng, lo, hi, step):
    """A multiple of step in [lo, hi], spread over the logarithm."""
    v = lo * (hi / lo) ** rng.random()
    return max(lo, min(hi, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(["gemm", "gemm", "w4", "norm"])
    if op == "norm":
        out = rng.choice(["bf16", "fp8"])
        return dict(op=op, tokens=_spread(rng, 1, 16384, 1), hidden=_spread(rng, 256, 7168, 128 if out == "fp8" else 8),
                    x=rng.choice(["bf16", "fp32"]), residual=rng.random() < 0.8, out=out)
    while True:
        experts = _spread(rng, 1, 256, 1)
        c = dict(op=op, experts=experts, topk=rng.randint(1, min(8, experts)),
                 routing=rng.choice(["uniform", "zipf", "hotset"]))
        # few experts take long batches, many take short ones
        c["tokens"] = _spread(rng, 1, 8192 if experts <= 16 and op == "gemm" else 1024, 1)
        c["gated"] = rng.random() < 0.5
        if op == "w4":
            c["group"] = rng.choice([32, 64, 128])
            c["zeros"] = rng.random() < 0.5
            c["n"], c["k"] = _spread(rng, 128, 7168, 8), _spread(rng, 256, 7168, c["group"])
        else:
            c["dtype"] = rng.choice(["bf16", "fp8"])
            c["out"] = rng.choice(["bf16", "fp8"]) if c["dtype"] == "fp8" and c["gated"] else "bf16"
            step = {"bf16": 8, "fp8": 16}[c["dtype"]] if c["out"] == "bf16" else 128
            c["n"], c["k"] = _spread(rng, 128, 7168, step), _spread(rng, 256, 7168, 8 if c["dtype"] == "bf16" else 128)
        weights = experts * c["k"] * c["n"] * (2 if c["gated"] else 1)
        if weights <= 256 * 4096 * 7168 and weights / experts * c["tokens"] * c["topk"] <= 8192 * 2 * 4096 * 4096:
            return c


def _counts(case, seed):
    """Rows of each expert: topk distinct experts a token."""
    rng = np.random.default_rng([seed, 17])
    t, e, k = case["tokens"], case["experts"], case["topk"]
    score = rng.random((t, e))
    if case["routing"] == "zipf":  # expert r - 1 has weight r^-1.2; the best of score^(1/weight)
        score = np.log(score) * np.arange(1, e + 1) ** 1.2
    elif case["routing"] == "hotset":  # half the tokens choose among few experts
        hot = rng.permutation(e)[:max(k, min(8, e))]
        score[np.ix_(rng.permutation(t)[:t // 2], hot)] += 1
    picks = np.argpartition(-score, k - 1, axis=1)[:, :k]
    return np.bincount(picks.reshape(-1), minlength=e).tolist()


def _normal(gen, *shape):
    return torch.randn(shape, generator=gen, device=DEV, dtype=torch.bfloat16)


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    s = dict(case=case)
    if case["op"] == "norm":
        t, h = case["tokens"], case["hidden"]
        s["x"] = _normal(gen, t, h).to(torch.float32 if case["x"] == "fp32" else torch.bfloat16)
        if case["x"] == "fp32":  # a weighted sum has all its bits
            s["x"] *= 1 + torch.rand(t, h, generator=gen, device=DEV) / 256
        s["residual"] = 4 * _normal(gen, t, h) if case["residual"] else None
        s["weight"] = 1 + _normal(gen, h) / 8
        s["sum"] = torch.zeros(t, h, dtype=torch.bfloat16, device=DEV) if case["residual"] else None
        s["out"] = torch.zeros(t, h, dtype=FP8 if case["out"] == "fp8" else torch.bfloat16, device=DEV)
        s["out_scales"] = torch.zeros(t, h // BLOCK, device=DEV) if case["out"] == "fp8" else None
        return s
    e, n, k, cap = case["experts"], case["n"], case["k"], case["tokens"]
    rows_w = 2 * n if case["gated"] else n
    counts = _counts(case, seed)
    # `rows` is the plain form's own: a kernel reads the counts on the GPU
    s["rows"] = [(i, i * cap, i * cap + c) for i, c in enumerate(counts) if c]
    s["counts"] = torch.tensor(counts, dtype=torch.int32, device=DEV)
    filled = torch.cat([torch.arange(b, t) for _, b, t in s["rows"]]).to(DEV)
    fp8 = case.get("dtype") == "fp8"
    s["a_scales"] = s["w_scales"] = s["zeros"] = s["out_scales"] = None
    if fp8:
        a = torch.full((e * cap, k), float("nan"), device=DEV).to(FP8).view(torch.uint8)
        codes, scales = _quantized(_normal(gen, len(filled), k).float())
        a[filled] = codes.view(torch.uint8)
        s["a"] = a.view(FP8)
        s["a_scales"] = torch.full((e * cap, k // BLOCK), float("nan"), device=DEV)
        s["a_scales"][filled] = scales
        s["w"] = torch.empty(e, rows_w, k, dtype=FP8, device=DEV)
        for i in range(e):
            s["w"][i] = (_normal(gen, rows_w, k) * 100).clamp(-448, 448).to(FP8)
        s["w_scales"] = (0.5 + torch.rand(e, -(-rows_w // BLOCK), k // BLOCK, generator=gen, device=DEV)) / (100 * k ** 0.5)
    else:
        s["a"] = torch.full((e * cap, k), float("nan"), dtype=torch.bfloat16, device=DEV)
        s["a"][filled] = _normal(gen, len(filled), k)
        if case["op"] == "w4":
            g = k // case["group"]
            s["w"] = torch.randint(0, 256, (e, rows_w, k // 2), generator=gen, device=DEV, dtype=torch.uint8)
            s["w_scales"] = ((0.5 + torch.rand(e, rows_w, g, generator=gen, device=DEV)) / (4.6 * k ** 0.5)).to(torch.bfloat16)
            if case["zeros"]:
                s["zeros"] = torch.randint(6, 10, (e, rows_w, g), generator=gen, device=DEV, dtype=torch.uint8)
        else:
            s["w"] = torch.empty(e, rows_w, k, dtype=torch.bfloat16, device=DEV)
            for i in range(e):
                s["w"][i] = _normal(gen, rows_w, k) / k ** 0.5
    if case.get("out") == "fp8":
        s["out"] = torch.zeros(e * cap, n, dtype=torch.uint8, device=DEV).view(FP8)
        s["out_scales"] = torch.zeros(e * cap, n // BLOCK, device=DEV)
    else:
        s["out"] = torch.zeros(e * cap, n, dtype=torch.bfloat16, device=DEV)
    return s


def _quantized(v):
    """fp32 rows in e4m3, a scale (largest magnitude / 448) per 128 columns."""
    b = v.view(v.shape[0], -1, BLOCK)
    amax = b.abs().amax(-1, keepdim=True)
    inv = torch.where(amax > 0, 448 / amax, torch.zeros_like(amax))
    return (b * inv).clamp(-448, 448).to(FP8).view(v.shape), (amax / 448)[..., 0]


def _blocks(scales, rows, k):
    """A scale per 128 x 128 block as one per element."""
    return scales.repeat_interleave(BLOCK, 0)[:rows].repeat_interleave(BLOCK, 1)[:, :k]


def _weight(s, e):
    """Expert e's weights in 32 bits."""
    case, w = s["case"], s["w"][e]
    if case["op"] == "w4":
        c = torch.stack((w & 15, w >> 4), -1).view(w.shape[0], -1, case["group"]).float()
        zero = s["zeros"][e].float()[..., None] if case["zeros"] else 8.0
        return ((c - zero) * s["w_scales"][e].float()[..., None]).view(w.shape[0], -1)
    if case["dtype"] == "fp8":
        return w.float() * _blocks(s["w_scales"][e], *w.shape)
    return w.float()


def _run_plain(s):
    case = s["case"]
    if case["op"] == "norm":
        h = s["x"].float()
        if case["residual"]:
            h = h + s["residual"].float()
            s["sum"] = h.to(torch.bfloat16)
        y = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + EPS) * s["weight"].float()
        if case["out"] == "fp8":
            s["out"], s["out_scales"] = _quantized(y)
        else:
            s["out"] = y.to(torch.bfloat16)
        return
    n = case["n"]
    for e, b, t in s["rows"]:  # experts have rows of their own number
        a = s["a"][b:t].float()
        if s["a_scales"] is not None:
            a = a * s["a_scales"][b:t].repeat_interleave(BLOCK, 1)
        p = a @ _weight(s, e).t()
        if case["gated"]:
            p = p[:, :n] * torch.sigmoid(p[:, :n]) * p[:, n:]
        if s["out_scales"] is not None:
            codes, s["out_scales"][b:t] = _quantized(p)
            s["out"].view(torch.uint8)[b:t] = codes.view(torch.uint8)
        else:
            s["out"][b:t] = p.to(torch.bfloat16)


def _run_own(s):
    import combine_ll_moe_amd as ll
    case = s["case"]
    if case["op"] == "norm":
        ll.ll_moe_rms_norm(case["tokens"], case["hidden"], ll.FP32 if case["x"] == "fp32" else ll.BF16,
                           ll.FP8_E4M3 if case["out"] == "fp8" else ll.BF16, EPS, s["x"], s["residual"], s["weight"],
                           s["sum"], s["out"], s["out_scales"])
        return
    act = ll.ACT_SILU_MUL if case["gated"] else ll.ACT_NONE
    if case["op"] == "w4":
        ll.ll_moe_expert_gemm_w4(case["tokens"], case["n"], case["k"], case["experts"], case["group"], act, s["a"], s["w"],
                                 s["w_scales"], s["zeros"], s["counts"], s["out"])
        return
    ll.ll_moe_expert_gemm(case["tokens"], case["n"], case["k"], case["experts"],
                          ll.FP8_E4M3 if case["dtype"] == "fp8" else ll.BF16, act,
                          ll.FP8_E4M3 if case["out"] == "fp8" else ll.BF16, s["a"], s["a_scales"], s["w"], s["w_scales"],
                          s["counts"], s["out"], s["out_scales"])


def run(state):
    if own:
        _run_own(state)
    else:
        _run_plain(state)
    return {name: state[name] for name in ("out", "out_scales", "sum") if state.get(name) is not None}


def work(case):
    if case["op"] == "norm":
        values = case["tokens"] * case["hidden"]
        moved = values * ((4 if case["x"] == "fp32" else 2) + (4 if case["residual"] else 0))
        moved += values * (2 if case["out"] == "bf16" else 1 + 4 / BLOCK) + 2 * case["hidden"]
        return dict(bytes=moved, flops=6 * values)
    n, k = case["n"], case["k"]
    rows_w = 2 * n if case["gated"] else n
    counts = _counts(case, 0)  # as any seed's, near enough
    active, rows = sum(c > 0 for c in counts), sum(counts)
    if case["op"] == "w4":
        weight = rows_w * k / 2 + rows_w * k // case["group"] * (3 if case["zeros"] else 2)
        a_row = 2 * k
    elif case["dtype"] == "fp8":
        weight, a_row = rows_w * k + 4 * -(-rows_w // BLOCK) * (k // BLOCK), k + 4 * (k // BLOCK)
    else:
        weight, a_row = 2 * rows_w * k, 2 * k
    out_row = 2 * n if case.get("out", "bf16") == "bf16" else n + 4 * (n // BLOCK)
    return dict(bytes=active * weight + rows * (a_row + out_row) + 4 * case["experts"], flops=2 * rows * rows_w * k)


def exact(case, seed):
    if work(case)["flops"] > 1e12:
        return None
    s = prepare(case, seed)
    block = lambda v: v.reshape(v.shape[0], v.shape[1] // BLOCK, BLOCK)  # noqa: E731
    out, got = s["out"].double(), {}
    scales = s["out_scales"].double() if s["out_scales"] is not None else None
    if case["op"] == "norm":
        v = s["x"].double()
        if case["residual"]:
            v += s["residual"].double()
            got["sum"] = v.clone()
        v = v / ((v * v).sum(1, keepdim=True) / case["hidden"] + EPS).sqrt() * s["weight"].double()
        done = [(slice(None), v)]
    else:
        done = []
        for e, (first, count) in enumerate(zip(range(0, out.shape[0], case["tokens"]), s["counts"].tolist())):
            if not count:
                continue
            rows = slice(first, first + count)
            a, w = s["a"][rows].double(), s["w"][e]
            if case["op"] == "w4":
                codes = torch.empty(w.shape[0], 2 * w.shape[1], dtype=torch.float64, device=DEV)
                codes[:, 0::2] = w.remainder(16).double()
                codes[:, 1::2] = w.div(16, rounding_mode="floor").double()
                at = torch.arange(case["k"], device=DEV) // case["group"]
                codes -= s["zeros"][e].double()[:, at] if case["zeros"] else 8
                w = codes * s["w_scales"][e].double()[:, at]
            elif case["dtype"] == "fp8":
                at = torch.arange(case["k"], device=DEV) // BLOCK
                a = a * s["a_scales"][rows].double()[:, at]
                w = w.double() * s["w_scales"][e].double()[torch.arange(w.shape[0], device=DEV) // BLOCK][:, at]
            v = a @ w.double().t()
            if case["gated"]:
                gate, up = v.split(case["n"], 1)
                v = gate / (1 + (-gate).exp()) * up
            done.append((rows, v))
    for rows, v in done:
        if scales is None:
            out[rows] = v
        else:  # the codes' values before they are rounded
            b = block(v)
            most = b.abs().max(-1, keepdim=True).values
            out[rows] = torch.where(most > 0, b / (most / 448), torch.zeros_like(b)).reshape(v.shape)
            scales[rows] = most[..., 0] / 448
    got["out"] = out
    if scales is not None:
        got["out_scales"] = scales
    return got
