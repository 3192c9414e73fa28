"""A whole layer's expert part on the GPU, as it is used: norm, dispatch, the
dispatch's expert side, both products with the activation between them, the
combine, and the norm that joins its output to the residual; against the same
computed token by token in 64 bits, with the bounds of every rounding carried
through."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - collected on CPU machines too
    pytest.skip("no GPU", allow_module_level=True)

import combine_ll_moe_amd as ll  # noqa: E402
import _experts as X  # noqa: E402
import workloads as W  # noqa: E402
from _gpu import DEV, say, to_dev  # noqa: E402

BF16, F8 = torch.bfloat16, torch.float8_e4m3fn
EPS = 1e-6


@pytest.mark.parametrize("weights", ["bf16", "fp8", "w4"])
@pytest.mark.parametrize("tokens", [1, 37])
def test_layer(weights, tokens):
    h, inter, e, k, cap = 512, 256, 9, 3, 40
    say("layer", weights, "tokens", tokens)
    g = torch.Generator(device=DEV).manual_seed(7)
    rn = lambda *s: torch.randn(s, generator=g, device=DEV)  # noqa: E731
    pay = ll.FP8_E4M3 if weights == "fp8" else ll.BF16
    wk = W.Workload("layer", tokens, h, e, k, pay, "uniform", max_tokens=cap)
    idx_h = W.routing(wk)
    idx_h[0, 1] = -1  # a masked pick
    idx, wt = to_dev(idx_h), to_dev(W.weights(wk))
    expected = int((idx_h >= 0).sum())
    x, res = rn(tokens, h).to(BF16), (4 * rn(tokens, h)).to(BF16)
    gamma = (1 + rn(h) / 8).to(BF16)
    rows = e * cap

    # weights of both products, and what they stand for in 64 bits
    if weights == "bf16":
        w1, w2 = (rn(e, 2 * inter, h) / h ** 0.5).to(BF16), (rn(e, h, inter) / inter ** 0.5).to(BF16)
        d1, d2 = w1.double(), w2.double()
    elif weights == "fp8":
        w1, w2 = (80 * rn(e, 2 * inter, h)).clamp(-448, 448).to(F8), (80 * rn(e, h, inter)).clamp(-448, 448).to(F8)
        s1 = (torch.rand(e, 2 * inter // 128, h // 128, generator=g, device=DEV) + 0.5) / (80 * h ** 0.5)
        s2 = (torch.rand(e, h // 128, inter // 128, generator=g, device=DEV) + 0.5) / (80 * inter ** 0.5)
        d1 = torch.stack([w1[i].double() * X.spread(s1[i], 2 * inter, h) for i in range(e)])
        d2 = torch.stack([w2[i].double() * X.spread(s2[i], h, inter) for i in range(e)])
    else:
        w1 = torch.randint(0, 256, (e, 2 * inter, h // 2), generator=g, device=DEV, dtype=torch.uint8)
        w2 = torch.randint(0, 256, (e, h, inter // 2), generator=g, device=DEV, dtype=torch.uint8)
        s1, s2 = (rn(e, 2 * inter, h // 64) / 90).to(BF16), (rn(e, h, inter // 64) / 70).to(BF16)
        z1 = torch.randint(0, 16, (e, 2 * inter, h // 64), generator=g, device=DEV, dtype=torch.uint8)
        d1 = torch.stack([X.along(s1[i], h, 64) * (X.unpack4(w1[i]) - X.along(z1[i], h, 64)) for i in range(e)])
        d2 = torch.stack([X.along(s2[i], inter, 64) * (X.unpack4(w2[i]) - 8) for i in range(e)])

    lay = torch.zeros(ll.ll_moe_layout_bytes(cap, h, e, pay), dtype=torch.uint8, device=DEV)
    hidden, stream1 = torch.empty_like(x), torch.empty_like(res)
    payload = torch.empty(rows, h, dtype=F8 if weights == "fp8" else BF16, device=DEV)
    scales = torch.empty(rows, h // 128, device=DEV)
    src, counts = (torch.empty(n, dtype=torch.int32, device=DEV) for n in (rows, e))
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    mid = torch.empty(rows, inter, dtype=F8 if weights == "fp8" else BF16, device=DEV)
    mid_scales = torch.empty(rows, inter // 128, device=DEV)
    y = torch.empty(rows, h, dtype=BF16, device=DEV)
    out = torch.empty(tokens, h, device=DEV)
    nxt, stream2 = torch.empty_like(x), torch.empty_like(res)

    def layer(q):
        ll.ll_moe_rms_norm(tokens, h, ll.BF16, ll.BF16, EPS, x, res, gamma, stream1, hidden)
        ll.ll_moe_dispatch(lay, cap, tokens, h, e, k, pay, q, hidden, idx)
        ll.ll_moe_dispatch_recv(lay, cap, h, e, pay, q, expected, payload, scales, src, counts, 1 << 20, status)
        if weights == "w4":
            ll.ll_moe_expert_gemm_w4(cap, inter, h, e, 64, ll.ACT_SILU_MUL, payload, w1, s1, z1, counts, mid)
            ll.ll_moe_expert_gemm_w4(cap, h, inter, e, 64, ll.ACT_NONE, mid, w2, s2, None, counts, y)
        elif weights == "fp8":
            ll.ll_moe_expert_gemm(cap, inter, h, e, ll.FP8_E4M3, ll.ACT_SILU_MUL, ll.FP8_E4M3, payload, scales, w1, s1,
                                  counts, mid, mid_scales)
            ll.ll_moe_expert_gemm(cap, h, inter, e, ll.FP8_E4M3, ll.ACT_NONE, ll.BF16, mid, mid_scales, w2, s2, counts, y)
        else:
            ll.ll_moe_expert_gemm(cap, inter, h, e, ll.BF16, ll.ACT_SILU_MUL, ll.BF16, payload, None, w1, None, counts,
                                  mid)
            ll.ll_moe_expert_gemm(cap, h, inter, e, ll.BF16, ll.ACT_NONE, ll.BF16, mid, None, w2, None, counts, y)
        ll.ll_moe_combine(lay, cap, tokens, h, e, k, pay, q, y, idx, wt, out)
        ll.ll_moe_rms_norm(tokens, h, ll.FP32, ll.BF16, EPS, out, stream1, gamma, stream2, nxt)

    layer(0)
    torch.cuda.synchronize()
    assert int(status.item()) & ~ll.RECV_WAITED == ll.RECV_READY
    assert counts.tolist() == np.bincount(idx_h[idx_h >= 0], minlength=e).tolist()

    hh, dh, v, dv = X.rms_norm(x, res, gamma, EPS)
    X.check_bf16(stream1, hh, dh, "stream")
    X.check_bf16(hidden, v, dv, "hidden")
    # the layer from the rounded hidden states on; an fp8 payload is a half
    # step (2^-4 relative, of values down to 2^-10 of the scale) off
    half = X.HALF_STEP
    a, da = hidden.double(), torch.zeros_like(hidden.double())

    def quantized(val, err):
        amax = val.abs().view(tokens, -1, 128).amax(-1).repeat_interleave(128, 1)
        return err + torch.maximum(half[F8] * (val.abs() + err), amax / 448 * 2.0 ** -10) + (val.abs() + err) * 8 * X.U

    if weights == "fp8":
        da = quantized(a, da)
    want, bound = torch.zeros_like(a), torch.zeros_like(a)
    for j in range(k):
        for t in range(tokens):
            ex = int(idx_h[t, j])
            if ex < 0:
                continue
            wide = 48.0 if weights == "w4" else 1.0  # the 4-bit sums count the codes' magnitudes
            mag = X.along(s1[ex], h, 64).abs() * wide if weights == "w4" else d1[ex].abs()
            at = a[t:t + 1]
            p = at @ d1[ex].t()
            dp = (h + 16) * X.U * (at.abs() + da[t:t + 1]) @ mag.t() + da[t:t + 1] @ d1[ex].abs().t()
            m, dm = X.gated(p, dp, inter)
            if weights == "fp8":
                am = (m.abs() + dm).view(1, -1, 128).amax(-1).repeat_interleave(128, 1)
                dm = dm + torch.maximum(half[F8] * (m.abs() + dm), am / 448 * 2.0 ** -10) + (m.abs() + dm) * 8 * X.U
            else:
                dm = dm + half[BF16] * (m.abs() + dm)
            mag = X.along(s2[ex], inter, 64).abs() * wide if weights == "w4" else d2[ex].abs()
            o = m @ d2[ex].t()
            do = (inter + 16) * X.U * (m.abs() + dm) @ mag.t() + dm @ d2[ex].abs().t()
            do = do + half[BF16] * (o.abs() + do)
            f = float(wt[t, j])
            want[t] += f * o[0]
            bound[t] += abs(f) * do[0] + 8 * X.U * abs(f) * (o.abs() + do)[0]
    err = (out.double() - want).abs()
    assert bool((err <= bound).all()), (float((err / bound).max()), float(err.max()))
    hh, dh, v, dv = X.rms_norm(out, stream1, gamma, EPS)
    X.check_bf16(stream2, hh, dh, "next stream")
    X.check_bf16(nxt, v, dv, "next hidden")

    # captured: both parities in one graph, replayed with eager work between
    first = [t.clone() for t in (out, nxt, stream2)]
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        status.zero_()
        layer(1)
        status.zero_()
        layer(0)
    for _ in range(3):
        for t in (out, nxt, stream2):
            t.fill_(float("nan"))
        (x.float() @ x.float().t()).sum().item()
        ll.ll_moe_clean_signals(lay, cap, h, e, pay, 1)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for t, f in zip((out, nxt, stream2), first):
            assert torch.equal(t, f)
