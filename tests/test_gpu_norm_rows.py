"""The norm over more rows than one grid holds (2^32 threads)."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - collected on CPU machines too
    pytest.skip("no GPU", allow_module_level=True)

import combine_ll_moe_amd as ll  # noqa: E402
import _experts as X  # noqa: E402
from _gpu import DEV, say  # noqa: E402

BF16, F8 = torch.bfloat16, torch.float8_e4m3fn


@pytest.mark.parametrize("x_fp32", [False, True])
def test_short_rows_to_bf16(x_fp32):
    """2^26 rows and three of 8 columns: 64 threads a row."""
    t, h = (1 << 26) + 3, 8
    say("case", t, h, x_fp32)
    x = torch.randn(t, h, device=DEV, dtype=torch.float32 if x_fp32 else BF16)
    res = (2 * torch.randn(t, h, device=DEV, dtype=torch.float32)).to(BF16)
    w = (1 + torch.randn(h, device=DEV) / 4).to(BF16)
    new, out = torch.zeros(t, h, dtype=BF16, device=DEV), torch.zeros(t + 1, h, dtype=BF16, device=DEV)
    ll.ll_moe_rms_norm(t, h, ll.FP32 if x_fp32 else ll.BF16, ll.BF16, 1e-6, x, res, w, new, out[:t])
    torch.cuda.synchronize()
    for lo in range(0, t, 1 << 24):
        r = slice(lo, min(lo + (1 << 24), t))
        hh, dh, y, dy = X.rms_norm(x[r], res[r], w, 1e-6)
        X.check_bf16(out[r], y, dy, "out")
        X.check_bf16(new[r], hh, dh, "residual")
    assert not out[t].any()


def test_long_rows_to_fp8():
    """2^24 rows and one of 1152 columns: 256 threads a row, 38 GiB in. Rows
    repeat every 4099, so that one slice's results stand for all."""
    t, h, period = (1 << 24) + 1, 1152, 4099
    say("case", t, h)
    part = torch.randn(period, h, device=DEV).to(BF16)
    x = torch.empty(t, h, dtype=BF16, device=DEV)
    for lo in range(0, t, period):
        n = min(period, t - lo)
        x[lo:lo + n] = part[:n]
    w = (1 + torch.randn(h, device=DEV) / 4).to(BF16)
    out = torch.zeros(t, h, dtype=torch.uint8, device=DEV)
    scales = torch.zeros(t, h // 128, device=DEV)
    ll.ll_moe_rms_norm(t, h, ll.BF16, ll.FP8_E4M3, 1e-6, x, None, w, None, out, scales)
    torch.cuda.synchronize()
    _, _, y, dy = X.rms_norm(part, None, w, 1e-6)
    X.check_fp8(out[:period].view(F8), scales[:period], y, dy)
    for lo in range(0, t, period):
        n = min(period, t - lo)
        assert torch.equal(out[lo:lo + n], out[:n]) and torch.equal(scales[lo:lo + n], scales[:n]), lo
