"""Every form that a dense product can take, at sizes that choose it: tiles of
16, 32, 64, 128 and 256 rows, plain, gated to bf16 and to fp8, whole or split along
k, with rows and columns that fill none of them."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - collected on CPU machines too
    pytest.skip("no GPU", allow_module_level=True)

import combine_ll_moe_amd as ll  # noqa: E402
from _gpu import DEV  # noqa: E402
from test_gpu_dense import BF16, F8, F32, make, run, verify  # noqa: E402


# around the numbers of workgroups up to which the few rows' own forms are taken, too
@pytest.mark.parametrize("m,n,k,out,addend", [
    (1, 8208, 256, F32, True), (16, 8224, 384, BF16, False), (17, 4112, 128, F32, True), (32, 4128, 640, BF16, True),
    (33, 4112, 256, F32, True), (65, 2000, 1664, BF16, False), (200, 720, 4096, F32, True), (130, 1040, 7168, BF16, False),
    (500, 272, 3200, F32, True), (256, 7168, 128, F32, True), (300, 7184, 256, BF16, True), (700, 784, 1792, F32, False),
    (1500, 1040, 2048, BF16, False), (3000, 272, 1024, F32, True), (5000, 2064, 128, BF16, True), (500, 2064, 5248, F32, True),
    (1, 12304, 256, F32, True), (16, 16400, 128, BF16, False), (30, 12320, 384, BF16, True), (20, 3216, 640, BF16, False),
    (31, 3200, 1920, F32, True), (33, 2064, 256, BF16, True), (64, 3600, 512, F32, True), (40, 4128, 256, BF16, False),
    (130, 1552, 7168, F32, True), (65, 2800, 5376, BF16, False), (200, 1200, 4096, F32, True), (9, 8208, 7168, BF16, False)])
def test_plain(m, n, k, out, addend):
    verify(m, n, k, False, out, addend)


@pytest.mark.parametrize("m,n,k", [
    (1, 4112, 1792, ), (7, 4208, 128), (16, 4128, 2048), (17, 2064, 256), (40, 1392, 1920), (64, 2192, 128),
    (100, 592, 3584), (129, 2064, 256), (300, 464, 7168), (700, 1040, 896), (2000, 272, 2048), (4100, 80, 384),
    (5000, 400, 256), (4097, 2064, 128), (200, 1040, 640),
    (3, 6160, 640), (16, 8208, 128), (11, 2576, 5376), (20, 1616, 896), (31, 2064, 256), (64, 1808, 384), (40, 2064, 1920),
    (64, 4112, 384), (3500, 2064, 256), (15001, 400, 128), (7500, 2064, 128), (300, 32912, 128), (950, 2064, 3200),
    (1900, 2064, 3328)])
def test_gated_to_bf16(m, n, k):
    verify(m, n, k, True, BF16)


@pytest.mark.parametrize("m,n,k", [
    (1, 2176, 1792), (9, 4096, 128), (16, 2304, 2048), (17, 1152, 256), (40, 1024, 1920), (64, 2176, 128), (100, 384, 3584),
    (129, 2048, 256), (300, 256, 7168), (700, 1024, 896), (2000, 256, 2048), (4100, 128, 384), (5000, 384, 256),
    (4097, 2176, 128), (3, 6272, 512), (16, 2304, 3328), (20, 1664, 896), (40, 2176, 1920), (60, 1664, 512), (64, 896, 256),
    (3601, 2176, 128), (4000, 2176, 256), (12000, 512, 128), (300, 32896, 128), (1100, 2048, 3200), (2300, 2048, 3328)])
def test_gated_to_fp8(m, n, k):
    verify(m, n, k, True, F8)


def test_sums_that_the_workspace_does_not_hold():
    """64 MiB are 2^24 sums."""
    verify(1050, 16016, 128, False, BF16)
    verify(1030, 8192, 128, True, F8)
    verify(60, 147456, 128, True, BF16)


@pytest.mark.parametrize("m,n,k,out", [(16, 524304, 128, BF16), (9, 1 << 20, 128, F8), (2, 1 << 20, 128, BF16)])
def test_the_widest_weights_stay_inside_the_workspace(m, n, k, out):
    a, a_s, w, w_s, _ = make(m, n, k, True, 4)
    space = torch.full((ll.DENSE_WORKSPACE * 3,), 0x5A, dtype=torch.uint8, device=DEV)
    o = torch.empty(m, n, device=DEV).to(out)
    s = torch.empty(m, n // 128, device=DEV) if out == F8 else None
    ll.ll_moe_dense_gemm(m, n, k, ll.ACT_SILU_MUL, ll.FP8_E4M3 if out == F8 else ll.BF16, a, a_s, w, w_s, None, o, s, space)
    torch.cuda.synchronize()
    assert bool((space[ll.DENSE_WORKSPACE:] == 0x5A).all())
    del space
    verify(m, n, k, True, out)


@pytest.mark.parametrize("m,n,k,gated,out", [
    (5, 8208, 256, False, BF16), (40, 1392, 1920, True, BF16), (130, 1040, 7168, False, F32), (700, 1040, 896, True, BF16),
    (3000, 272, 1024, False, F32), (4100, 384, 256, True, F8), (100, 384, 3584, True, F8), (16, 256, 512, True, F8), (3500, 2176, 128, True, F8), (40, 2064, 1920, True, BF16), (130, 1552, 7168, False, F32), (20, 3216, 640, False, BF16),
    (20, 1664, 896, True, F8), (30, 12320, 384, False, F32), (3, 6160, 640, True, BF16), (4000, 2064, 128, True, BF16)])
def test_nothing_behind_the_operands_is_read(m, n, k, gated, out):
    """The operands inside larger buffers of NaN, the workspace too."""
    t = make(m, n, k, gated, 3)
    want, want_s = run(*t, n, gated, out)
    inside = []
    for x in t[:4]:
        big = torch.full((x.numel() * x.element_size() + 65536,), 0x7F if x.dtype == F8 else 0xFF, dtype=torch.uint8, device=DEV)
        big[:x.numel() * x.element_size()] = x.reshape(-1).view(torch.uint8)
        inside.append(big.view(x.dtype))
    rows_w = 2 * n if gated else n
    a, a_s, w, w_s = inside
    o = torch.full((m * n + 4096,), 7.0, device=DEV).to(out)
    s = torch.full((m * (n // 128) + 64,), 7.0, device=DEV) if out == F8 else None
    space = torch.full((ll.DENSE_WORKSPACE,), 0xFF, dtype=torch.uint8, device=DEV)
    ll.ll_moe_dense_gemm(m, n, k, ll.ACT_SILU_MUL if gated else ll.ACT_NONE,
                         {BF16: ll.BF16, F8: ll.FP8_E4M3, F32: ll.FP32}[out], a, a_s, w, w_s, None, o, s, space)
    torch.cuda.synchronize()
    raw = torch.uint8 if out == F8 else out
    assert torch.equal(o[:m * n].view(raw).view(m, n), want.view(raw)) and bool((o[m * n:].float() == 7).all())
    if s is not None:
        assert torch.equal(s[:m * (n // 128)].view(m, -1), want_s) and bool((s[m * (n // 128):] == 7).all())
    assert rows_w * k == t[2].numel()


def test_the_same_call_gives_the_same_bits():
    for m, n, k, gated, out in ((1, 2048, 7168, True, F8), (128, 1040, 7168, False, F32), (777, 512, 7168, True, BF16)):
        t = make(m, n, k, gated, 5)
        first = run(*t, n, gated, out)[0].view(torch.uint8)
        for _ in range(3):
            assert torch.equal(run(*t, n, gated, out)[0].view(torch.uint8), first)


def test_captured_in_two_parts():
    """Rows that go out in two parts, of which the second uses the workspace."""
    m, n, k = 4100, 2176, 256
    t = make(m, n, k, True, 6)
    want = run(*t, n, True, F8)
    o, s = torch.empty(m, n, dtype=F8, device=DEV), torch.empty(m, n // 128, device=DEV)
    space = torch.empty(ll.DENSE_WORKSPACE, dtype=torch.uint8, device=DEV)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        ll.ll_moe_dense_gemm(m, n, k, ll.ACT_SILU_MUL, ll.FP8_E4M3, *t, o, s, space)
    for i in range(3):
        o.view(torch.uint8).fill_(0x7F)
        s.fill_(float("nan"))
        space.fill_(0xFF)
        run(*make(40 + i, 640, 512, True, i), 640, True, F8)  # eager calls between the replays
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o.view(torch.uint8), want[0].view(torch.uint8)) and torch.equal(s, want[1])
