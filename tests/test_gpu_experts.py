"""The operators around the expert side on the GPU, against plain 64-bit forms
(tests/_experts.py): products grouped by expert in bf16, fp8 and with 4-bit
weights, plain and gated, and the norm. Rows that no count fills are poisoned
with NaN on the way in and filled with a sentinel on the way out."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - collected on CPU machines too
    pytest.skip("no GPU", allow_module_level=True)

import combine_ll_moe_amd as ll  # noqa: E402
import _experts as X  # noqa: E402
from _gpu import DEV, say  # noqa: E402

BF16, F8 = torch.bfloat16, torch.float8_e4m3fn
SENT = 0xA5


class Gemm:
    """Inputs and sentinel-filled outputs of one grouped product."""

    def __init__(self, kind, counts, cap, n, k, gated=False, out_fp8=False, group=128, zeros=False, seed=0,
                 poison=True):
        self.kind, self.cap, self.n, self.k, self.gated, self.group = kind, cap, n, k, gated, group
        self.e, self.given = len(counts), list(counts)
        self.counts = torch.tensor(counts, dtype=torch.int32, device=DEV)
        self.rows_of = [max(0, min(c, cap)) for c in counts]
        g = torch.Generator(device=DEV).manual_seed(seed)
        rn = lambda *s: torch.randn(s, generator=g, device=DEV)  # noqa: E731
        rows, rw = self.e * cap, (2 * n if gated else n)
        self.rw = rw
        fill = torch.zeros(rows, dtype=torch.bool, device=DEV)
        for i, c in enumerate(self.rows_of):
            fill[i * cap:i * cap + c] = True
        self.fill = fill
        self.a_scales = self.w_scales = self.w_zeros = self.out_scales = None
        nan = float("nan") if poison else 0.0
        if kind == "fp8":
            a = (rn(rows, k) * 80).clamp(-448, 448).to(F8)
            self.a = torch.where(fill[:, None], a.view(torch.uint8), torch.full_like(a.view(torch.uint8), 0x7F)).view(F8)
            self.a_scales = torch.where(fill[:, None], torch.rand(rows, k // 128, generator=g, device=DEV) + 0.1,
                                        torch.full((), nan, device=DEV))
            self.w = (rn(self.e, rw, k) * 80).clamp(-448, 448).to(F8)
            self.w_scales = (torch.rand(self.e, -(-rw // 128), k // 128, generator=g, device=DEV) + 0.1) / (6400 * k ** 0.5)
        else:
            self.a = torch.where(fill[:, None], rn(rows, k), torch.full((), nan, device=DEV)).to(BF16)
            if kind == "w4":
                self.w = torch.randint(0, 256, (self.e, rw, k // 2), generator=g, device=DEV, dtype=torch.uint8)
                self.w_scales = (rn(self.e, rw, k // group) / (4 * k ** 0.5)).to(BF16)
                if zeros:
                    self.w_zeros = torch.randint(0, 16, (self.e, rw, k // group), generator=g, device=DEV,
                                                 dtype=torch.uint8)
            else:
                self.w = (rn(self.e, rw, k) / k ** 0.5).to(BF16)
        self.out_fp8 = out_fp8
        self.out = torch.empty(rows, n, dtype=F8 if out_fp8 else BF16, device=DEV)
        if out_fp8:
            self.out_scales = torch.empty(rows, n // 128, device=DEV)
        self.clear()

    def clear(self):
        self.out.view(torch.uint8).fill_(SENT)
        if self.out_scales is not None:
            self.out_scales.fill_(-7.0)

    def run(self, stream=None):
        act = ll.ACT_SILU_MUL if self.gated else ll.ACT_NONE
        if self.kind == "w4":
            ll.ll_moe_expert_gemm_w4(self.cap, self.n, self.k, self.e, self.group, act, self.a, self.w, self.w_scales,
                                     self.w_zeros, self.counts, self.out, stream=stream)
        else:
            ll.ll_moe_expert_gemm(self.cap, self.n, self.k, self.e, ll.FP8_E4M3 if self.kind == "fp8" else ll.BF16,
                                  act, ll.FP8_E4M3 if self.out_fp8 else ll.BF16, self.a, self.a_scales, self.w,
                                  self.w_scales, self.counts, self.out, self.out_scales, stream=stream)
        return self

    def expect(self, e):
        r = slice(e * self.cap, e * self.cap + self.rows_of[e])
        a = self.a[r].double()
        if self.kind == "w4":
            z = self.w_zeros[e].double() if self.w_zeros is not None else torch.full_like(self.w_scales[e].double(), 8)
            p, dp = X.product_w4(a, X.unpack4(self.w[e]), self.w_scales[e], z, self.group)
        else:
            w = self.w[e].double()
            if self.kind == "fp8":
                a = a * X.along(self.a_scales[r], self.k)
                w = w * X.spread(self.w_scales[e], self.rw, self.k)
            p, dp = X.product(a, w)
        if self.gated:
            p, dp = X.gated(p, dp, self.n)
        return r, p, dp

    def check(self, experts=None):
        torch.cuda.synchronize()
        for e in range(self.e) if experts is None else experts:
            if not self.rows_of[e]:
                continue
            r, p, dp = self.expect(e)
            what = (self.kind, "expert", e, "rows", self.rows_of[e])
            if self.out_fp8:
                X.check_fp8(self.out[r], self.out_scales[r], p, dp, what)
            else:
                X.check_bf16(self.out[r], p, dp, what)
        rest = ~self.fill
        assert bool((self.out.view(torch.uint8)[rest] == SENT).all()), "a row behind the count was written"
        if self.out_scales is not None:
            assert bool((self.out_scales[rest] == -7.0).all()), "scales behind the count were written"


COUNTS = [0, 1, 15, 16, 17, 3, 32, 33, 0, 63, 64, 65, 70, -5, 1000]  # capacity 70: the last is taken as 70

KINDS = [
    dict(kind="bf16"), dict(kind="bf16", gated=True),
    dict(kind="fp8"), dict(kind="fp8", gated=True), dict(kind="fp8", gated=True, out_fp8=True),
    dict(kind="w4", group=128), dict(kind="w4", group=128, zeros=True, gated=True),
    dict(kind="w4", group=64, zeros=True), dict(kind="w4", group=64, gated=True),
    dict(kind="w4", group=32, gated=True, zeros=True), dict(kind="w4", group=32),
]
IDS = ["-".join(str(v) for v in c.values()) for c in KINDS]


def _say(**kw):
    say("case", kw)


@pytest.mark.parametrize("c", KINDS, ids=IDS)
def test_ragged_counts(c):
    _say(**c)
    Gemm(counts=COUNTS, cap=70, n=256, k=512, **c).run().check()


SIZES = [(8, 8), (24, 40), (40, 72), (1000, 1000), (72, 2056), (136, 64), (520, 136)]


@pytest.mark.parametrize("n,k", SIZES)
@pytest.mark.parametrize("gated", [False, True])
def test_odd_sizes_bf16(n, k, gated):
    _say(n=n, k=k, gated=gated)
    Gemm("bf16", [2, 0, 19, 40], 41, n, k, gated=gated, seed=n + k).run().check()


@pytest.mark.parametrize("n,k", [(16, 128), (48, 256), (144, 384), (1040, 640), (112, 1152)])
@pytest.mark.parametrize("gated", [False, True])
def test_odd_sizes_fp8(n, k, gated):
    _say(n=n, k=k, gated=gated)
    Gemm("fp8", [2, 0, 19, 40], 41, n, k, gated=gated, seed=n + k).run().check()


@pytest.mark.parametrize("n,k,group", [(8, 32, 32), (24, 96, 32), (200, 2016, 32), (40, 64, 64), (136, 1088, 64),
                                       (8, 128, 128), (120, 1408, 128)])
@pytest.mark.parametrize("gated", [False, True])
def test_odd_sizes_w4(n, k, group, gated):
    _say(n=n, k=k, group=group, gated=gated)
    Gemm("w4", [2, 0, 19, 40], 41, n, k, gated=gated, group=group, zeros=True, seed=n + k).run().check()


@pytest.mark.parametrize("c", KINDS, ids=IDS)
def test_one_token_many_experts(c):
    """One row each for 8 of 300 experts: more experts than threads."""
    _say(**c)
    counts = [0] * 300
    for e in (0, 7, 8, 100, 255, 256, 298, 299):
        counts[e] = 1
    Gemm(counts=counts, cap=1, n=128, k=256, **c).run().check()


@pytest.mark.parametrize("c", KINDS, ids=IDS)
def test_many_rows(c):
    _say(**c)
    Gemm(counts=[700, 5, 129, 256, 257, 0], cap=700, n=384, k=640, seed=3, **c).run().check()


@pytest.mark.parametrize("kind", ["bf16", "fp8", "w4"])
def test_capacity_of_128_with_large_weights(kind):
    """Up to 128 rows an expert, weights of over 256 MiB."""
    n, k = (4096, 4096) if kind == "bf16" else (8192, 4096) if kind == "fp8" else (8192, 8192)
    _say(kind=kind, n=n, k=k)
    Gemm(kind, [128, 3, 0, 65, 100, 64, 1, 17, 0, 90], 128, n, k, seed=9).run().check()


@pytest.mark.parametrize("c", KINDS, ids=IDS)
def test_no_rows_at_all(c):
    _say(**c)
    Gemm(counts=[0, 0, -1], cap=5, n=128, k=256, **c).run().check()


@pytest.mark.parametrize("kind", ["bf16", "fp8", "w4"])
def test_largest_expert_count(kind):
    counts = [0] * 4096
    counts[0], counts[4095], counts[2000] = 2, 2, 1
    _say(kind=kind, experts=4096)
    Gemm(kind, counts, 2, 16, 128).run().check(experts=[0, 2000, 4095])
    # and with whole row tiles
    counts[0], counts[4095] = 300, 150
    Gemm(kind, counts, 300, 16, 128).run().check(experts=[0, 2000, 4095])


@pytest.mark.parametrize("c", KINDS, ids=IDS)
def test_a_rows_nan_and_infinity_stay_in_it(c):
    """One row with a NaN and one with an infinity: every other row is what it
    is without them, bit for bit."""
    _say(**c)
    g = Gemm(counts=[20, 3, 90], cap=90, n=128, k=256, seed=5, **c)
    g.run()
    want = g.out.view(torch.uint8).clone()
    bad_rows = [4, 90 + 1, 180 + 77]
    for i, r in enumerate(bad_rows):
        if g.kind == "fp8":
            g.a.view(torch.uint8)[r, 9 * i] = 0x7F
        else:
            g.a[r, 9 * i] = float("nan") if i else float("inf")
    g.clear()
    g.run()
    torch.cuda.synchronize()
    keep = torch.ones(len(want), dtype=torch.bool, device=DEV)
    keep[bad_rows] = False
    assert torch.equal(g.out.view(torch.uint8)[keep], want[keep])
    if not g.out_fp8:
        assert not torch.isfinite(g.out[bad_rows].float()).any()


@pytest.mark.parametrize("c", KINDS, ids=IDS)
def test_zero_rows_give_zeros(c):
    _say(**c)
    g = Gemm(counts=[3, 80], cap=80, n=128, k=256, **c)
    g.a.view(torch.uint8)[1] = 0
    g.a.view(torch.uint8)[100] = 0
    g.run().check()
    assert not g.out[[1, 100]].float().any()
    if g.out_scales is not None:
        assert not g.out_scales[[1, 100]].any()


@pytest.mark.parametrize("c", KINDS, ids=IDS)
def test_repeats_are_the_same_bits(c):
    _say(**c)
    g = Gemm(counts=[40, 100, 3], cap=100, n=256, k=384, **c).run()
    torch.cuda.synchronize()
    first = g.out.view(torch.uint8).clone()
    for _ in range(3):
        g.clear()
        g.run()
        torch.cuda.synchronize()
        assert torch.equal(g.out.view(torch.uint8), first)


def test_row_offsets_past_32_bits():
    """Activations of more than 4 GiB: the last expert's rows stand behind."""
    cap, k, n = 150_000, 4096, 16
    _say(rows=4 * cap, k=k)
    a = torch.empty(4 * cap, k, dtype=BF16, device=DEV)
    w = (torch.randn(4, n, k, device=DEV) / 64).to(BF16)
    rows = slice(3 * cap, 3 * cap + 100)
    a[rows] = torch.randn(100, k, device=DEV).to(BF16)
    out = torch.zeros(4 * cap, n, dtype=BF16, device=DEV)
    counts = torch.tensor([0, 0, 0, 100], dtype=torch.int32, device=DEV)
    ll.ll_moe_expert_gemm(cap, n, k, 4, ll.BF16, ll.ACT_NONE, ll.BF16, a, None, w, None, counts, out)
    p, dp = X.product(a[rows].double(), w[3].double())
    X.check_bf16(out[rows], p, dp)
    assert int((out != 0).any(1).sum()) == 100


@pytest.mark.parametrize("kind", ["bf16", "w4"])
def test_weight_offsets_past_32_bits(kind):
    e, n, k = 600, 1024, 4096 if kind == "bf16" else 16384
    _say(kind=kind, experts=e, n=n, k=k)
    g = Gemm(kind, [0, 0], 2, 8, 128)  # sizes only
    del g
    w = torch.empty(e, n, k if kind == "bf16" else k // 2, dtype=BF16 if kind == "bf16" else torch.uint8, device=DEV)
    a = torch.full((2 * e, k), float("nan"), dtype=BF16, device=DEV)
    a[-2] = torch.randn(k, device=DEV).to(BF16)
    counts = torch.zeros(e, dtype=torch.int32, device=DEV)
    counts[-1] = 1
    out = torch.zeros(2 * e, n, dtype=BF16, device=DEV)
    if kind == "bf16":
        w[-1] = (torch.randn(n, k, device=DEV) / 64).to(BF16)
        ll.ll_moe_expert_gemm(2, n, k, e, ll.BF16, ll.ACT_NONE, ll.BF16, a, None, w, None, counts, out)
        p, dp = X.product(a[-2:-1].double(), w[-1].double())
    else:
        w[-1] = torch.randint(0, 256, (n, k // 2), dtype=torch.uint8, device=DEV)
        s = torch.ones(e, n, k // 128, dtype=BF16, device=DEV) / 64
        ll.ll_moe_expert_gemm_w4(2, n, k, e, 128, ll.ACT_NONE, a, w, s, None, counts, out)
        p, dp = X.product_w4(a[-2:-1].double(), X.unpack4(w[-1]), s[-1], torch.full_like(s[-1].double(), 8), 128)
    X.check_bf16(out[-2:-1], p, dp)
    assert int((out != 0).any(1).sum()) == 1


@pytest.mark.parametrize("c", [KINDS[1], KINDS[4], KINDS[6]], ids=[IDS[1], IDS[4], IDS[6]])
def test_captured_and_replayed(c):
    """A captured call reads the counts of the replay: other counts, other
    rows, with eager work between the replays."""
    _say(**c)
    g = Gemm(counts=[90, 90, 90], cap=90, n=128, k=256, **c)
    s = torch.cuda.Stream()
    g.run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        g.run()
    for counts in ([3, 0, 90], [0, 0, 0], [70, 17, 1], [90, 64, 65]):
        g.clear()
        g.counts.copy_(torch.tensor(counts, dtype=torch.int32))
        g.rows_of = counts
        g.fill = torch.zeros_like(g.fill)
        for i, n in enumerate(counts):
            g.fill[90 * i:90 * i + n] = True
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        g.check()


@pytest.mark.parametrize("c", [KINDS[0], KINDS[4], KINDS[9]], ids=[IDS[0], IDS[4], IDS[9]])
def test_two_calls_at_once(c):
    """Two streams, two calls of other inputs: no shared workspace."""
    _say(**c)
    a = Gemm(counts=[40, 300], cap=300, n=256, k=1024, seed=1, **c)
    b = Gemm(counts=[300, 9], cap=300, n=256, k=1024, seed=2, **c)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(4):
        a.run(stream=s1)
        b.run(stream=s2)
    a.check()
    b.check()


def test_strided_and_host_tensors_are_refused():
    g = Gemm("bf16", [3], 4, 16, 16)
    for name in ("a", "w", "out"):
        keep = getattr(g, name)
        for bad in (torch.cat([keep, keep], -1)[..., ::2], keep.cpu()):
            setattr(g, name, bad)
            with pytest.raises(ll.LLMoEError) as ei:
                g.run()
            assert ei.value.status == ll.INVALID_ARGUMENT
        setattr(g, name, keep)
    g.run().check()


# ---- the norm ---------------------------------------------------------------

NORM_SHAPES = [(1, 8), (3, 24), (5, 512), (4, 520), (7, 1024), (9, 1000), (2, 2048), (130, 2056), (3, 4096),
               (6, 7168), (2, 8192), (3, 8200), (2, 16384), (3, 22520), (2, 32768)]


def _norm(t, h, x_fp32, residual, out_fp8, seed=0, in_place=False, mutate=None):
    g = torch.Generator(device=DEV).manual_seed(seed)
    rn = lambda *s: torch.randn(s, generator=g, device=DEV)  # noqa: E731
    x = rn(t, h) * 3 if x_fp32 else (rn(t, h) * 3).to(BF16)
    if mutate:
        mutate(x)
    res = (rn(t, h) * 5).to(BF16) if residual else None
    keep = res.clone() if residual else None
    w = (1 + rn(h) / 4).to(BF16)
    new = None
    if residual:
        new = res if in_place else torch.empty(t + 1, h, dtype=BF16, device=DEV)[:t]
    full = torch.empty(t + 1, h, dtype=F8 if out_fp8 else BF16, device=DEV)
    full.view(torch.uint8).fill_(SENT)
    scales = torch.full((t + 1, h // 128), -7.0, device=DEV) if out_fp8 else None
    ll.ll_moe_rms_norm(t, h, ll.FP32 if x_fp32 else ll.BF16, ll.FP8_E4M3 if out_fp8 else ll.BF16, 1e-6, x, res, w,
                       new, full[:t], scales[:t] if out_fp8 else None)
    torch.cuda.synchronize()
    assert bool((full.view(torch.uint8)[t] == SENT).all())
    if out_fp8:
        assert bool((scales[t] == -7.0).all())
    return x, keep, w, new, full[:t], scales[:t] if out_fp8 else None


@pytest.mark.parametrize("t,h", NORM_SHAPES)
@pytest.mark.parametrize("x_fp32", [False, True])
@pytest.mark.parametrize("residual", [False, True])
def test_norm_bf16(t, h, x_fp32, residual):
    _say(t=t, h=h, x_fp32=x_fp32, residual=residual)
    x, res, w, new, out, _ = _norm(t, h, x_fp32, residual, False)
    hh, dh, y, dy = X.rms_norm(x, res, w, 1e-6)
    X.check_bf16(out, y, dy, "out")
    if residual:
        X.check_bf16(new, hh, dh, "residual")


@pytest.mark.parametrize("t,h", [(1, 128), (5, 512), (3, 1024), (9, 1152), (2, 2176), (129, 4096), (6, 7168),
                                 (2, 8320), (3, 16384), (2, 32768)])
@pytest.mark.parametrize("x_fp32", [False, True])
def test_norm_fp8(t, h, x_fp32):
    _say(t=t, h=h, x_fp32=x_fp32)
    x, res, w, new, out, scales = _norm(t, h, x_fp32, True, True)
    hh, dh, y, dy = X.rms_norm(x, res, w, 1e-6)
    X.check_fp8(out, scales, y, dy, "out")
    X.check_bf16(new, hh, dh, "residual")


@pytest.mark.parametrize("t,h", [(5, 512), (3, 7168)])
def test_norm_residual_in_place(t, h):
    _say(t=t, h=h)
    x, res, w, new, out, _ = _norm(t, h, False, True, False, in_place=True)
    hh, dh, y, dy = X.rms_norm(x, res, w, 1e-6)
    X.check_bf16(out, y, dy, "out")
    X.check_bf16(new, hh, dh, "residual")


def test_norm_of_zeros_infinities_and_nan():
    """A row of zeros gives zeros, rows with a NaN or an infinity stay apart."""
    def mutate(x):
        x[0] = 0
        x[2, 5] = float("nan")
        x[4, 7] = float("inf")
    for out_fp8 in (False, True):
        _say(out_fp8=out_fp8)
        x, _, w, _, out, scales = _norm(6, 1024, False, False, out_fp8, mutate=mutate)
        assert not out[0].float().any()
        good = [1, 3, 5]
        _, _, y, dy = X.rms_norm(x[good], None, w, 1e-6)
        if out_fp8:
            assert not scales[0].any()
            X.check_fp8(out[good], scales[good], y, dy)
        else:
            X.check_bf16(out[good], y, dy)
            assert torch.isnan(out[2].float()).all()
            v = out[4].float()  # inf / inf at its place, finite / inf = 0 elsewhere
            assert torch.isnan(v[7]) and not v[torch.arange(1024, device=DEV) != 7].any()


def test_norm_large_batch_offsets():
    """More than 4 GiB of rows."""
    t, h = 330_000, 8192
    _say(t=t, h=h)
    x = torch.zeros(t, h, dtype=BF16, device=DEV)
    x[-3:] = torch.randn(3, h, device=DEV).to(BF16)
    w = torch.ones(h, dtype=BF16, device=DEV)
    out = torch.empty_like(x)
    ll.ll_moe_rms_norm(t, h, ll.BF16, ll.BF16, 1e-6, x, None, w, None, out)
    _, _, y, dy = X.rms_norm(x[-4:], None, w, 1e-6)
    X.check_bf16(out[-4:], y, dy)
    assert not out[:-3].any()


def test_norm_empty_batch():
    w = torch.ones(64, dtype=BF16, device=DEV)
    ll.ll_moe_rms_norm(0, 64, ll.BF16, ll.BF16, 1e-6, None, None, w, None, None)
