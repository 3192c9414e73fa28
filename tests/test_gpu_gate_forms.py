"""Every form that the router's logits can take, at its edges: calls that go
to tiles of both sizes, with columns, experts and tokens that fill none."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - collected on CPU machines too
    pytest.skip("no GPU", allow_module_level=True)

import combine_ll_moe_amd as ll  # noqa: E402
from _gpu import DEV, say  # noqa: E402
from test_gpu_gate import BF16, F32, make, run, verify  # noqa: E402


@pytest.mark.parametrize("wtype", [BF16, F32])
@pytest.mark.parametrize("t,h,e", [
    (1025, 1024, 256), (1537, 520, 257), (5000, 64, 100), (6001, 72, 66), (2000, 8, 300), (700, 1096, 1000),
    (12300, 256, 256), (12289, 328, 255), (24600, 136, 97), (9000, 64, 401), (3100, 64, 1030), (800, 192, 4096),
    (262145, 8, 2), (300000, 16, 1), (8000, 200, 250), (16001, 72, 127), (40000, 136, 64)])
def test_sizes(t, h, e, wtype):
    say("gate forms", t, h, e, wtype)
    verify(*make(t, h, e, wtype))


@pytest.mark.parametrize("t,e", [(2000, 200), (8100, 230), (12500, 250)])
@pytest.mark.parametrize("wtype", [BF16, F32])
def test_nan_behind_the_rows_and_columns_is_not_read(t, e, wtype):
    """The operands inside larger buffers of NaN."""
    x, w = make(t, 136, e, wtype)
    want = run(x, w)
    xs = torch.full((t * 136 + 4096,), float("nan"), device=DEV).to(BF16)
    ws = torch.full((e * 136 + 4096,), float("nan"), device=DEV).to(wtype)
    xs[:t * 136], ws[:e * 136] = x.view(-1), w.view(-1)
    out = torch.full((t * e + 64,), 7.0, device=DEV)
    ll.ll_moe_gate(t, 136, e, ll.FP32 if wtype == F32 else ll.BF16, xs, ws, out)
    torch.cuda.synchronize()
    assert torch.equal(out[:t * e].view(t, e), want) and bool((out[t * e:] == 7).all())
