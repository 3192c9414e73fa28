"""The router's logits on the GPU against the same product in 64 bits."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - collected on CPU machines too
    pytest.skip("no GPU", allow_module_level=True)

import combine_ll_moe_amd as ll  # noqa: E402
import _experts as X  # noqa: E402
from _gpu import DEV, say  # noqa: E402

BF16, F32 = torch.bfloat16, torch.float32


def run(x, w):
    t, e = x.shape[0], w.shape[0]
    out = torch.full((t + 1, e), 77.0, device=DEV)  # a row behind, left as it is
    ll.ll_moe_gate(t, x.shape[1], e, ll.FP32 if w.dtype == F32 else ll.BF16, x, w, out)
    torch.cuda.synchronize()
    assert bool((out[t] == 77).all())
    return out[:t]


def verify(x, w, what=""):
    got = run(x, w).double()
    # exact products, fp32 sums; three products a column for an fp32 weight
    p, bound = X.product(x.double(), w.double())
    bound = bound * (3 if w.dtype == F32 else 1)
    bad = ~((got - p).abs() <= bound)
    assert not bad.any(), (what, int(bad.sum()), got[bad][:4].tolist(), p[bad][:4].tolist())


def make(t, h, e, wtype, seed=1):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn(t, h, generator=g, device=DEV).to(BF16)
    return x, (torch.randn(e, h, generator=g, device=DEV) / h ** 0.5).to(wtype)


@pytest.mark.parametrize("wtype", [BF16, F32])
@pytest.mark.parametrize("t,h,e", [
    (1, 7168, 256), (1, 8, 1), (2, 16, 3), (3, 72, 17), (5, 1000, 63), (8, 4096, 64), (9, 264, 255), (15, 7168, 16),
    (16, 1024, 8), (17, 512, 129), (31, 2048, 160), (33, 520, 33), (64, 7168, 256), (65, 640, 257), (100, 4096, 161),
    (128, 7168, 256), (129, 1536, 100), (200, 7168, 384), (257, 776, 65), (500, 1024, 512), (1000, 2056, 130),
    (4096, 256, 64), (3001, 1024, 61), (2, 32768, 5), (7, 128, 4096), (300, 64, 4096)])
def test_sizes(t, h, e, wtype):
    say("gate", t, h, e, wtype)
    verify(*make(t, h, e, wtype))


@pytest.mark.parametrize("t", [0, 4, 12, 40, 150, 1100])
def test_nothing_is_written_behind_the_last_token(t):
    x, w = make(t, 512, 40, BF16)
    verify(x, w)


@pytest.mark.parametrize("t", [3, 20, 140, 2100])
@pytest.mark.parametrize("wtype", [BF16, F32])
def test_a_row_s_infinities_and_nans_stay_in_it(t, wtype):
    x, w = make(t, 328, 50, wtype)
    clean = run(x, w)
    y = x.clone()
    y[1, 5], y[t - 1, 300] = float("nan"), float("inf")
    got = run(y, w)
    rest = [i for i in range(t) if i not in (1, t - 1)]
    assert torch.equal(got[rest], clean[rest])
    assert bool(got[1].isnan().all())
    if wtype == BF16:
        assert torch.equal(got[t - 1], torch.sign(w[:, 300].float()) * float("inf"))
    else:
        assert not bool(got[t - 1].isfinite().any())


@pytest.mark.parametrize("t", [1, 30, 1500])
def test_no_bit_of_an_fp32_weight_is_lost(t):
    """One column a weight, x = 1: the logits are the weights."""
    e, h = 48, 64
    g = torch.Generator(device=DEV).manual_seed(4)
    w = torch.zeros(e, h, device=DEV)
    at = torch.randint(0, h, (e,), generator=g, device=DEV)
    v = torch.randn(e, generator=g, device=DEV) * torch.exp(20 * torch.randn(e, generator=g, device=DEV))
    w[torch.arange(e, device=DEV), at] = v
    x = torch.ones(t, h, device=DEV).to(BF16)
    assert torch.equal(run(x, w), v.expand(t, e))


def test_weights_that_are_not_finite():
    x, w = make(6, 128, 20, F32)
    clean = run(x, w)
    w[3, 7], w[9, 100] = float("inf"), float("nan")
    got = run(x, w)
    assert bool(got[:, [3, 9]].isnan().all())
    rest = [i for i in range(20) if i not in (3, 9)]
    assert torch.equal(got[:, rest], clean[:, rest])


def test_captured():
    x, w = make(50, 1024, 96, BF16)
    want = run(x, w)
    out = torch.empty(50, 96, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ll.ll_moe_gate(50, 1024, 96, ll.BF16, x, w, out)
    for _ in range(3):
        out.fill_(float("nan"))
        (x.float() @ x.float().t()).sum().item()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


@pytest.mark.parametrize("t", [1, 4, 30, 200, 9000])
@pytest.mark.parametrize("wtype", [BF16, F32])
def test_tiny_values(t, wtype):
    """Weights from 2^-100 to fp32's subnormals: an fp32 weight is off by less
    than 2^-133, and a sum whose weights lie below 2^-126 by 2^-16 of its
    magnitudes."""
    g = torch.Generator(device=DEV).manual_seed(t)
    for power in (-100, -115, -125, -130, -140):
        x = (torch.randn(t, 64, generator=g, device=DEV) * 2.0 ** 90).to(BF16)
        w = (torch.randn(48, 64, generator=g, device=DEV).double() * 2.0 ** power).to(wtype)
        got = run(x, w).double()
        p, bound = X.product(x.double(), w.double())
        size = x.double().abs() @ w.double().abs().t()
        bound = 3 * bound + x.double().abs().sum(1, keepdim=True) * 2.0 ** -133 * (wtype == F32) + size * 2.0 ** -16
        assert bool(((got - p).abs() <= bound).all()), (power, ((got - p).abs() / bound).max().item())
