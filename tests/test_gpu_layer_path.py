"""A layer from hidden states to hidden states as it is used: norm, router,
dispatch, expert products, combine, and the shared expert that joins the
combine's output; eager, and captured with batches of several sizes."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - collected on CPU machines too
    pytest.skip("no GPU", allow_module_level=True)

import combine_ll_moe_amd as ll  # noqa: E402
import _experts as X  # noqa: E402
import _router as R  # noqa: E402
from _gpu import DEV, say  # noqa: E402

BF16, F8 = torch.bfloat16, torch.float8_e4m3fn
EPS, H, INTER, E, K, GROUPS, KEPT, CAP = 1e-6, 512, 256, 24, 3, 4, 2, 48


class Layer:
    """The buffers and weights that a program keeps; one call is one layer."""

    def __init__(self, tokens, seed=7):
        g = torch.Generator(device=DEV).manual_seed(seed)
        rn = lambda *s: torch.randn(s, generator=g, device=DEV)  # noqa: E731
        q8 = lambda *s: (80 * rn(*s)).clamp(-448, 448).to(F8)  # noqa: E731
        sc = lambda r, c, *e: (torch.rand(*e, -(-r // 128), c // 128, generator=g, device=DEV) + 0.5) / (80 * c ** 0.5)  # noqa: E731
        self.t = tokens
        self.x, self.res = rn(tokens, H).to(BF16), (4 * rn(tokens, H)).to(BF16)
        self.gamma = (1 + rn(H) / 8).to(BF16)
        self.router, self.bias = rn(E, H) / H ** 0.5, (rn(E) * 30).round() / 1000
        self.w1, self.s1 = q8(E, 2 * INTER, H), sc(2 * INTER, H, E)
        self.w2, self.s2 = q8(E, H, INTER), sc(H, INTER, E)
        self.v1, self.t1 = q8(2 * INTER, H), sc(2 * INTER, H)
        self.v2, self.t2 = q8(H, INTER), sc(H, INTER)
        rows, new = E * CAP, lambda *s, d=torch.float32: torch.empty(s, dtype=d, device=DEV)
        self.lay = torch.zeros(ll.ll_moe_layout_bytes(CAP, H, E, ll.FP8_E4M3), dtype=torch.uint8, device=DEV)
        self.stream1, self.hidden, self.stream2, self.next = (new(tokens, H, d=BF16) for _ in range(4))
        self.codes, self.codes_s = new(tokens, H, d=F8), new(tokens, H // 128)
        self.logits, self.idx, self.wt = new(tokens, E), new(tokens, K, d=torch.int32), new(tokens, K)
        self.valid = torch.tensor([tokens], dtype=torch.int32, device=DEV)
        self.pay, self.pay_s = new(rows, H, d=F8), new(rows, H // 128)
        self.src, self.counts = new(rows, d=torch.int32), new(E, d=torch.int32)
        self.status = torch.zeros(1, dtype=torch.int32, device=DEV)
        self.mid, self.mid_s, self.y = new(rows, INTER, d=F8), new(rows, INTER // 128), new(rows, H, d=BF16)
        self.sh, self.sh_s = new(tokens, INTER, d=F8), new(tokens, INTER // 128)
        self.out = new(tokens, H)
        self.space = new(ll.DENSE_WORKSPACE, d=torch.uint8)

    def __call__(self, q, n):
        t = self.t
        ll.ll_moe_rms_norm(t, H, ll.BF16, ll.BF16, EPS, self.x, self.res, self.gamma, self.stream1, self.hidden)
        ll.ll_moe_rms_norm(t, H, ll.BF16, ll.FP8_E4M3, EPS, self.x, self.res, self.gamma, None, self.codes, self.codes_s)
        ll.ll_moe_gate(t, H, E, ll.FP32, self.hidden, self.router, self.logits)
        ll.ll_moe_route(t, E, K, ll.FP32, ll.SCORE_SIGMOID, GROUPS, KEPT, 2, True, 2.5, self.logits, self.bias, self.valid,
                        self.idx, self.wt)
        ll.ll_moe_dispatch(self.lay, CAP, t, H, E, K, ll.FP8_E4M3, q, self.hidden, self.idx)
        ll.ll_moe_dispatch_recv(self.lay, CAP, H, E, ll.FP8_E4M3, q, n * K, self.pay, self.pay_s, self.src, self.counts,
                                1 << 20, self.status)
        ll.ll_moe_expert_gemm(CAP, INTER, H, E, ll.FP8_E4M3, ll.ACT_SILU_MUL, ll.FP8_E4M3, self.pay, self.pay_s, self.w1,
                              self.s1, self.counts, self.mid, self.mid_s)
        ll.ll_moe_expert_gemm(CAP, H, INTER, E, ll.FP8_E4M3, ll.ACT_NONE, ll.BF16, self.mid, self.mid_s, self.w2, self.s2,
                              self.counts, self.y)
        ll.ll_moe_combine(self.lay, CAP, t, H, E, K, ll.FP8_E4M3, q, self.y, self.idx, self.wt, self.out)
        # the shared expert joins the combine's output where that stands
        ll.ll_moe_dense_gemm(t, INTER, H, ll.ACT_SILU_MUL, ll.FP8_E4M3, self.codes, self.codes_s, self.v1, self.t1, None,
                             self.sh, self.sh_s, self.space)
        ll.ll_moe_dense_gemm(t, H, INTER, ll.ACT_NONE, ll.FP32, self.sh, self.sh_s, self.v2, self.t2, self.out, self.out,
                             None, self.space)
        ll.ll_moe_rms_norm(t, H, ll.FP32, ll.BF16, EPS, self.out, self.stream1, self.gamma, self.stream2, self.next)

    def check(self, n):
        """Each operator's outputs from its own inputs, then the sum."""
        t = self.t
        assert int(self.status.item()) & ~ll.RECV_WAITED == ll.RECV_READY
        hh, dh, v, dv = X.rms_norm(self.x, self.res, self.gamma, EPS)
        X.check_bf16(self.hidden, v, dv, "hidden")
        X.check_fp8(self.codes, self.codes_s, v, dv, "codes")
        p, dp = X.product(self.hidden.double(), self.router.double())
        assert bool(((self.logits.double() - p).abs() <= 3 * dp).all())
        R.check(self.idx.cpu(), self.wt.cpu(), self.logits.cpu().numpy(), self.bias.cpu().numpy(), n, K, True, GROUPS, KEPT,
                2, True, 2.5, "route")
        picks = self.idx[self.idx >= 0]
        assert self.counts.tolist() == torch.bincount(picks, minlength=E).tolist()
        # the shared expert from the norm's codes on
        a = self.codes.double() * X.along(self.codes_s, H)
        v, dv = X.gated(*X.product(a, self.v1.double() * X.spread(self.t1, 2 * INTER, H)), INTER)
        X.check_fp8(self.sh, self.sh_s, v, dv, "shared")
        a = self.sh.double() * X.along(self.sh_s, INTER)
        p, dp = X.product(a, self.v2.double() * X.spread(self.t2, H, INTER))
        # and the routed experts' outputs, as the combine weighs them
        slot = {}
        for e in range(E):
            for j in range(int(self.counts[e])):
                slot[int(self.src[e * CAP + j]), e] = e * CAP + j
        for r in range(t):
            mag = torch.zeros_like(p[r])
            for k in range(K):
                e = int(self.idx[r, k])
                if e >= 0:
                    o = float(self.wt[r, k]) * self.y[slot[r, e]].double()
                    p[r] += o
                    mag += o.abs()
            dp[r] += (K + 2) * X.U * mag
        dp = dp + 2 * X.U * (p.abs() + dp)
        assert bool(((self.out.double() - p).abs() <= dp).all())
        hh, dh, v, dv = X.rms_norm(self.out, self.stream1, self.gamma, EPS)
        X.check_bf16(self.next, v, dv, "next")


@pytest.mark.parametrize("tokens,valid", [(1, 1), (37, 37), (37, 30), (48, 0)])
def test_layer(tokens, valid):
    say("layer with its router", tokens, valid)
    layer = Layer(tokens)
    layer.valid.fill_(valid)
    layer(0, valid)
    torch.cuda.synchronize()
    layer.check(valid)


def test_a_captured_layer_matches_the_eager_one():
    say("captured layer with its router")
    layer = Layer(33)
    layer(0, 33)
    torch.cuda.synchronize()
    layer.check(33)
    keep = [t.clone() for t in (layer.idx, layer.wt, layer.out, layer.next)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.status.zero_()
        layer(1, 33)
        layer.status.zero_()
        layer(0, 33)
    for _ in range(3):
        for t in (layer.out, layer.next, layer.wt):
            t.fill_(float("nan"))
        layer.idx.fill_(-7)
        (layer.x.float() @ layer.x.float().t()).sum().item()
        ll.ll_moe_clean_signals(layer.lay, CAP, H, E, ll.FP8_E4M3, 1)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for t, k in zip((layer.idx, layer.wt, layer.out, layer.next), keep):
            assert torch.equal(t, k)
