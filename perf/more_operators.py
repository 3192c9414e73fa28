"""The router and the dense products beside an MoE step: what is measured of them.

Three operators, in the order in which a layer calls them:

  gate   the router's logits: bf16 hidden states times bf16 or fp32 weights of
         each expert, summed and kept in 32 bits
  route  logits to picks: softmax or sigmoid scores, a bias that counts for the
         choice alone, the best groups of experts, the best experts of those
         in descending order (ties to the lower index), and their weights,
         renormalised or not, times a scale; rows behind the batch's valid
         ones get no picks (-1, weight 0). The choice is made in 64 bits.
  dense  the product that every token takes (a shared expert's, a dense
         layer's): fp8 e4m3 with one scale per 128 activations and per
         128 x 128 weights; gated (silu(gate) * up, out in fp8 with scales or
         bf16), or plain, out in bf16 or fp32, with an fp32 addend (the
         combine's output) or without
"""
import torch

own = False

DEV = "cuda:0"
FP8 = torch.float8_e4m3fn
BLOCK = 128
WORKSPACE = 64 << 20  # bytes that a dense product may use for partial sums


def listed():
    return [
        # one token's logits: latency
        dict(name="gate one token bf16", op="gate", tokens=1, hidden=7168, experts=256, w="bf16"),
        # a decode batch, router weights kept in fp32 as training left them
        dict(name="gate decode fp32", op="gate", tokens=128, hidden=7168, experts=256, w="fp32"),
        # a prompt's tokens: bound by the matrix cores
        dict(name="gate prompt bf16", op="gate", tokens=16384, hidden=7168, experts=256, w="bf16"),
        # one token's picks: latency
        dict(name="route one token", op="route", tokens=1, experts=256, topk=8, logits="fp32", score="sigmoid", bias=True,
             groups=8, topk_groups=4, best=2, renormalize=True, scale=2.5, valid=1),
        # a padded decode batch over few experts, plain softmax weights
        dict(name="route decode softmax", op="route", tokens=128, experts=64, topk=6, logits="fp32", score="softmax", bias=False,
             groups=1, topk_groups=1, best=1, renormalize=False, scale=1.0, valid=99),
        # a prompt's tokens with the balancing bias and groups: bound by instructions
        dict(name="route prompt groups", op="route", tokens=16384, experts=256, topk=8, logits="fp32", score="sigmoid", bias=True,
             groups=8, topk_groups=4, best=2, renormalize=True, scale=2.5, valid=16384),
        # bf16 logits (many equal ones) of an odd number of experts
        dict(name="route odd bf16", op="route", tokens=5000, experts=161, topk=7, logits="bf16", score="softmax", bias=True,
             groups=1, topk_groups=1, best=1, renormalize=True, scale=1.0, valid=4987),
        # one token through a shared expert's first product: latency, bound by the weights
        dict(name="dense one token gated", op="dense", tokens=1, n=2048, k=7168, gated=True, out="fp8", addend=False),
        # a decode batch through its second product, joined to the combine's output
        dict(name="dense decode down", op="dense", tokens=128, n=7168, k=2048, gated=False, out="fp32", addend=True),
        # a chunk of a prompt of odd length, first product
        dict(name="dense chunk gated", op="dense", tokens=777, n=2048, k=7168, gated=True, out="fp8", addend=False),
        # few tokens, an odd width
        dict(name="dense few odd", op="dense", tokens=17, n=1040, k=4096, gated=False, out="bf16", addend=False),
        # a prompt's tokens, first product: bound by the matrix cores
        dict(name="dense prompt gated", op="dense", tokens=8192, n=2048, k=7168, gated=True, out="bf16", addend=False),
    ]


def _spread(rng, lo, hi, step):
    """A multiple of step in [lo, hi], spread over the logarithm."""
    v = lo * (hi / lo) ** rng.random()
    return max(lo, min(hi, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(["gate", "route", "dense"])
    while True:
        c = dict(op=op, tokens=_spread(rng, 1, 8192 if op == "dense" else 16384, 1))
        if op == "gate":
            c |= dict(hidden=_spread(rng, 256, 7168, 8), experts=_spread(rng, 4, 512, 1), w=rng.choice(["bf16", "fp32"]))
            if c["tokens"] * c["hidden"] * c["experts"] <= 16384 * 7168 * 256 and (c["w"] == "bf16" or c["tokens"] <= 8192):
                return c
        elif op == "route":
            groups = rng.choice([1, 1, 2, 4, 6, 8])
            per = _spread(rng, 4, 512 // groups, 1)
            c |= dict(experts=groups * per, groups=groups, topk_groups=rng.randint(1, groups), best=rng.choice([1, 2]),
                      logits=rng.choice(["fp32", "bf16"]), score=rng.choice(["softmax", "sigmoid"]), bias=rng.random() < 0.5,
                      renormalize=rng.random() < 0.5, scale=rng.choice([1.0, 2.5]))
            c["topk"] = rng.randint(1, min(8, c["topk_groups"] * per))
            c["valid"] = c["tokens"] - rng.randint(0, c["tokens"] // 8)
            if c["tokens"] * c["experts"] <= 16384 * 256:
                return c
        else:
            c["gated"] = rng.random() < 0.5
            c["out"] = rng.choice(["fp8", "bf16"] if c["gated"] else ["fp32", "bf16"])
            c["addend"] = not c["gated"] and rng.random() < 0.5
            c |= dict(n=_spread(rng, 128, 7168, 128 if c["out"] == "fp8" else 16), k=_spread(rng, 256, 7168, 128))
            if c["tokens"] * c["n"] * (2 if c["gated"] else 1) * c["k"] <= 8192 * 4096 * 7168:
                return c


def _normal(gen, *shape):
    return torch.randn(shape, generator=gen, device=DEV)


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    s, t = dict(case=case), case["tokens"]
    if case["op"] == "gate":
        h, e = case["hidden"], case["experts"]
        s["x"] = _normal(gen, t, h).to(torch.bfloat16)  # a norm's output
        s["w"] = _normal(gen, e, h) / h ** 0.5
        if case["w"] == "bf16":
            s["w"] = s["w"].to(torch.bfloat16)
        s["logits"] = torch.zeros(t, e, device=DEV)
    elif case["op"] == "route":
        e, k = case["experts"], case["topk"]
        # some experts are liked by more tokens than others
        s["logits"] = (_normal(gen, t, e) + _normal(gen, e) / 2).to(torch.bfloat16 if case["logits"] == "bf16" else torch.float32)
        # a balancing bias is moved up and down by a fixed step
        size = 0.03 if case["score"] == "sigmoid" else 0.03 / e
        s["bias"] = (_normal(gen, e) * 30).round() * (size / 30) if case["bias"] else None
        s["valid"] = torch.full((1,), case["valid"], dtype=torch.int32, device=DEV)
        s["idx"] = torch.zeros(t, k, dtype=torch.int32, device=DEV)
        s["weights"] = torch.zeros(t, k, device=DEV)
    else:
        n, k = case["n"], case["k"]
        rows_w = 2 * n if case["gated"] else n
        s["a"], s["a_scales"] = _quantized(_normal(gen, t, k))
        s["w"] = (_normal(gen, rows_w, k) * 100).clamp(-448, 448).to(FP8)
        s["w_scales"] = (0.5 + torch.rand(-(-rows_w // BLOCK), k // BLOCK, generator=gen, device=DEV)) / (100 * k ** 0.5)
        s["addend"] = _normal(gen, t, n) if case["addend"] else None
        s["out"] = torch.zeros(t, n, device=DEV).to({"fp8": FP8, "bf16": torch.bfloat16, "fp32": torch.float32}[case["out"]])
        s["out_scales"] = torch.zeros(t, n // BLOCK, device=DEV) if case["out"] == "fp8" else None
        # one for all of a program's calls
        s["workspace"] = torch.empty(WORKSPACE, dtype=torch.uint8, device=DEV)
    return s


def _quantized(v):
    """fp32 rows in e4m3, a scale (largest magnitude / 448) per 128 columns."""
    b = v.view(v.shape[0], -1, BLOCK)
    amax = b.abs().amax(-1, keepdim=True)
    inv = torch.where(amax > 0, 448 / amax, torch.zeros_like(amax))
    return (b * inv).clamp(-448, 448).to(FP8).view(v.shape), (amax / 448)[..., 0]


def _plain_route(s):
    case, most = s["case"], torch.finfo(torch.float32).max
    t, e, k, groups = case["tokens"], case["experts"], case["topk"], case["groups"]
    # in 64 bits: which of two near scores is the larger shows in whole numbers
    l = s["logits"].double().nan_to_num(nan=float("-inf"), posinf=most, neginf=float("-inf"))
    there = l > float("-inf")
    if case["score"] == "sigmoid":
        score = 1 / (1 + torch.exp(-l))
    else:
        p = torch.exp(l - l.amax(1, keepdim=True))
        score = p / p.sum(1, keepdim=True)
    v = score if case["bias"] else l  # scores rise with the logits
    if case["bias"]:
        v = v + s["bias"].double()
    v = torch.where(there, v, float("-inf"))
    if groups > 1:
        by_group = v.view(t, groups, e // groups)
        # a sum of scores is no sum of logits
        of_group = by_group
        if not case["bias"] and case["best"] == 2:
            of_group = torch.where(there, score, float("-inf")).view_as(by_group)
        best = of_group.sort(dim=-1, descending=True).values[..., :case["best"]].sum(-1)
        kept = best.sort(dim=-1, descending=True, stable=True).indices[:, :case["topk_groups"]]
        inside = torch.zeros_like(best, dtype=torch.bool).scatter_(1, kept, True)
        v = torch.where(inside[..., None], by_group, float("-inf")).view(t, e)
    v, idx = v.sort(dim=1, descending=True, stable=True)
    v, idx = v[:, :k], idx[:, :k]
    live = (v > float("-inf")) & (torch.arange(t, device=DEV) < s["valid"])[:, None]
    w = torch.where(live, score.gather(1, idx), 0.0)
    if case["renormalize"]:
        w = w / w.sum(1, keepdim=True).clamp(min=1e-300)
    s["idx"] = torch.where(live, idx, -1).int()
    s["weights"] = (w * case["scale"]).float()


def _plain_dense(s):
    case, n = s["case"], s["case"]["n"]
    a = s["a"].float() * s["a_scales"].repeat_interleave(BLOCK, 1)
    w = s["w"].float() * s["w_scales"].repeat_interleave(BLOCK, 0)[:s["w"].shape[0]].repeat_interleave(BLOCK, 1)
    p = a @ w.t()
    if case["gated"]:
        p = p[:, :n] / (1 + torch.exp(-p[:, :n])) * p[:, n:]
    if case["addend"]:
        p = p + s["addend"]
    if case["out"] == "fp8":
        s["out"], s["out_scales"] = _quantized(p)
    else:
        s["out"] = p.to(s["out"].dtype)


def _run_own(s):
    import combine_ll_moe_amd as ll
    case = s["case"]
    if case["op"] == "gate":
        ll.ll_moe_gate(case["tokens"], case["hidden"], case["experts"], ll.FP32 if case["w"] == "fp32" else ll.BF16, s["x"],
                       s["w"], s["logits"])
    elif case["op"] == "route":
        ll.ll_moe_route(case["tokens"], case["experts"], case["topk"], ll.FP32 if case["logits"] == "fp32" else ll.BF16,
                        ll.SCORE_SIGMOID if case["score"] == "sigmoid" else ll.SCORE_SOFTMAX, case["groups"],
                        case["topk_groups"], case["best"], case["renormalize"], case["scale"], s["logits"], s["bias"],
                        s["valid"], s["idx"], s["weights"])
    else:
        ll.ll_moe_dense_gemm(case["tokens"], case["n"], case["k"], ll.ACT_SILU_MUL if case["gated"] else ll.ACT_NONE,
                             {"fp8": ll.FP8_E4M3, "bf16": ll.BF16, "fp32": ll.FP32}[case["out"]],
                             s["a"], s["a_scales"], s["w"], s["w_scales"], s["addend"], s["out"], s["out_scales"],
                             s["workspace"])


def run(state):
    op = state["case"]["op"]
    if own:
        _run_own(state)
    elif op == "gate":
        state["logits"] = state["x"].float() @ state["w"].float().t()
    elif op == "route":
        _plain_route(state)
    else:
        _plain_dense(state)
    names = {"gate": ("logits",), "route": ("idx", "weights"), "dense": ("out", "out_scales")}[op]
    return {name: state[name] for name in names if state[name] is not None}


def work(case):
    t = case["tokens"]
    if case["op"] == "gate":
        h, e = case["hidden"], case["experts"]
        return dict(bytes=2 * t * h + (4 if case["w"] == "fp32" else 2) * e * h + 4 * t * e, flops=2 * t * h * e)
    if case["op"] == "route":
        e = case["experts"]
        # a score, a comparison and a few operations around them for each logit
        return dict(bytes=case["valid"] * e * (4 if case["logits"] == "fp32" else 2) + 8 * t * case["topk"] + 4 * e,
                    flops=8 * case["valid"] * e)
    n, k = case["n"], case["k"]
    rows_w = 2 * n if case["gated"] else n
    moved = rows_w * k + 4 * -(-rows_w // BLOCK) * (k // BLOCK) + t * (k + 4 * (k // BLOCK))
    moved += t * n * ({"fp8": 1 + 4 / BLOCK, "bf16": 2, "fp32": 4}[case["out"]] + (4 if case["addend"] else 0))
    return dict(bytes=moved, flops=2 * t * rows_w * k)


def _exact_route(case, s):
    """Row blocks; an expert's place is the number of experts before it."""
    e, groups, inf = case["experts"], case["groups"], float("inf")
    number = torch.arange(e, device=DEV)

    def places(v):
        """How many of a row stand before each: larger, or equal with a lower number."""
        i = torch.arange(v.shape[1], device=DEV)
        a, b = v[:, None, :], v[:, :, None]
        return ((a > b) | ((a == b) & (i[None, None, :] < i[None, :, None]))).sum(2)

    all_idx, all_w = [], []
    for first in range(0, case["tokens"], 256):
        l = s["logits"][first:first + 256].double()
        rows = l.shape[0]
        if case["score"] == "softmax":
            score = (l - torch.logsumexp(l, 1, keepdim=True)).exp()
        else:
            score = torch.special.expit(l)
        if case["bias"]:
            order = score + s["bias"].double()
        else:
            order = score if groups > 1 and case["best"] == 2 else l
        if groups > 1:
            two = order.view(rows, groups, -1).topk(case["best"], 2).values
            group_place = places(two.sum(2))
            out = (group_place >= case["topk_groups"]).repeat_interleave(e // groups, 1)
            order = (order if case["bias"] else l).masked_fill(out, -inf)
        place = places(order)
        idx = torch.empty(rows, e, dtype=torch.int64, device=DEV).scatter_(1, place, number.expand(rows, e))[:, :case["topk"]]
        w = torch.take_along_dim(score, idx, 1)
        if case["renormalize"]:
            w = w / w.sum(1, keepdim=True)
        w = w * case["scale"]
        gone = torch.arange(first, first + rows, device=DEV) >= case["valid"]
        idx[gone], w[gone] = -1, 0.0
        all_idx.append(idx.int())
        all_w.append(w)
    return dict(idx=torch.cat(all_idx), weights=torch.cat(all_w))


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "gate":
        return dict(logits=s["x"].double() @ s["w"].double().t())
    if case["op"] == "route":
        return _exact_route(case, s)
    at = torch.arange(case["k"], device=DEV) // BLOCK
    rows = torch.arange(s["w"].shape[0], device=DEV) // BLOCK
    w = s["w"].double() * s["w_scales"].double()[rows][:, at]
    v = s["a"].double() * s["a_scales"].double()[:, at] @ w.t()
    if case["gated"]:
        gate, up = v.split(case["n"], 1)
        v = gate * torch.special.expit(gate) * up
    if case["addend"]:
        v = v + s["addend"].double()
    if case["out"] != "fp8":
        return dict(out=v)
    b = v.reshape(case["tokens"], -1, BLOCK)  # the codes' values before they are rounded
    scales = b.abs().max(-1).values / 448
    return dict(out=torch.where(scales[..., None] > 0, b / scales[..., None], 0.0).reshape(v.shape), out_scales=scales)
