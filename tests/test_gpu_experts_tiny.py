"""fp8 outputs whose 128 columns hold nothing but tiny values on the GPU: finite
inputs give finite codes and scales that stand for the values."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - collected on CPU machines too
    pytest.skip("no GPU", allow_module_level=True)

import combine_ll_moe_amd as ll  # noqa: E402
from _gpu import DEV, say  # noqa: E402

BF16, F8 = torch.bfloat16, torch.float8_e4m3fn


def _check(codes, scales, v):
    """codes * scales against v (float64): half a step of e4m3 (2^-4 of the
    value), or half its smallest step (2^-10) of the scale, and 1e-5 of the
    value for the fp32 arithmetic (an exponential of 88 is off by 88 x 1.44 x
    2^-24 and some steps)."""
    c, s = codes.float().double(), scales.double().repeat_interleave(128, 1)
    assert int(torch.isnan(c).sum()) == 0 and int((~torch.isfinite(s)).sum()) == 0
    tol = 2.0 ** -4 * v.abs() + 2.0 ** -10 * s + 1e-5 * v.abs()
    assert bool(((c * s - v).abs() <= tol).all()), ((c * s)[0, :8], v[0, :8])
    assert int((c[v == 0] != 0).sum()) == 0


@pytest.mark.parametrize("rows", [3, 300])
def test_gates_far_below_zero(rows):
    """silu(-88) is 5e-37 and silu(-192) is zero in fp32."""
    say("case", rows)
    n, k = 128, 128
    x = torch.zeros(rows, k, device=DEV)
    x[:, 3] = 1
    w = torch.zeros(1, 2 * n, k, device=DEV)
    w[0, :n, 3] = torch.tensor([-88.0, -192.0], device=DEV).repeat(n // 2)
    w[0, n:, 3] = 1
    out = torch.zeros(rows, n, dtype=F8, device=DEV)
    scales = torch.full((rows, 1), -7.0, device=DEV)
    one = torch.ones(rows, 1, device=DEV)
    ll.ll_moe_expert_gemm(rows, n, k, 1, ll.FP8_E4M3, ll.ACT_SILU_MUL, ll.FP8_E4M3, x.to(F8), one, w.to(F8),
                          torch.ones(1, 2, 1, device=DEV), torch.tensor([rows], dtype=torch.int32, device=DEV), out, scales)
    torch.cuda.synchronize()
    g = w[0, :n, 3].double()
    v = torch.where(g < -100, torch.zeros_like(g), g * torch.exp(g)).expand(rows, n)
    _check(out, scales, v)


@pytest.mark.parametrize("t,h", [(2, 128), (3, 1152), (300, 4224)])
def test_norm_of_tiny_rows(t, h):
    """h = 2^-127 and zeros, weights of 2^-10, eps 1e-6: y about 1000 x 2^-137."""
    say("case", t, h)
    x = torch.zeros(t, h, device=DEV)
    x[:, ::3] = 2.0 ** -127
    x[0] = 0
    w = torch.full((h,), 2.0 ** -10, dtype=BF16, device=DEV)
    out = torch.zeros(t, h, dtype=F8, device=DEV)
    scales = torch.full((t, h // 128), -7.0, device=DEV)
    ll.ll_moe_rms_norm(t, h, ll.FP32, ll.FP8_E4M3, 1e-6, x, None, w, None, out, scales)
    torch.cuda.synchronize()
    eps = float(torch.tensor(1e-6, dtype=torch.float32))
    v = x.double() / (x.double().square().mean(1, keepdim=True) + eps).sqrt() * w.double()
    # y is a subnormal of fp32 here: half its step, 2^-150, besides
    c, s = out.float().double(), scales.double().repeat_interleave(128, 1)
    assert int(torch.isnan(c).sum()) == 0 and int((~torch.isfinite(s)).sum()) == 0
    assert bool(((c * s - v).abs() <= 2.0 ** -4 * v.abs() + 2.0 ** -10 * s + 2.0 ** -149).all())
    assert int((c[v == 0] != 0).sum()) == 0 and not scales[0].any() and bool((scales[1:] > 0).all())
