"""The dense fp8 products on the GPU against the same in 64 bits."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - collected on CPU machines too
    pytest.skip("no GPU", allow_module_level=True)

import combine_ll_moe_amd as ll  # noqa: E402
import _experts as X  # noqa: E402
from _gpu import DEV, say  # noqa: E402

BF16, F8, F32 = torch.bfloat16, torch.float8_e4m3fn, torch.float32
LL = {BF16: ll.BF16, F8: ll.FP8_E4M3, F32: ll.FP32}


def make(m, n, k, gated, seed=1, addend=False):
    g = torch.Generator(device=DEV).manual_seed(seed)
    rows_w = 2 * n if gated else n
    a = (100 * torch.randn(m, k, generator=g, device=DEV)).clamp(-448, 448).to(F8)
    a_s = (0.5 + torch.rand(m, k // 128, generator=g, device=DEV)) / 100
    w = (100 * torch.randn(rows_w, k, generator=g, device=DEV)).clamp(-448, 448).to(F8)
    w_s = (0.5 + torch.rand(-(-rows_w // 128), k // 128, generator=g, device=DEV)) / (100 * k ** 0.5)
    add = torch.randn(m, n, generator=g, device=DEV) if addend else None
    return a, a_s, w, w_s, add


def workspace():
    return torch.full((ll.DENSE_WORKSPACE,), 0xFF, dtype=torch.uint8, device=DEV)  # NaN, read as fp32


def run(a, a_s, w, w_s, add, n, gated, out, space=None, into=None, stream=None):
    """out: the output's type."""
    m, k = a.shape
    o = torch.full((m + 1, n), 7.0, device=DEV).to(out) if into is None else into  # a row behind, left as it is
    s = torch.full((m + 1, n // 128), 7.0, device=DEV) if out == F8 else None
    ll.ll_moe_dense_gemm(m, n, k, ll.ACT_SILU_MUL if gated else ll.ACT_NONE, LL[out], a, a_s, w, w_s, add, o, s,
                         workspace() if space is None else space, stream=stream)
    torch.cuda.synchronize()
    if into is None:
        assert bool((o[m].float() == 7).all()) and (s is None or bool((s[m] == 7).all()))
    return o[:m], None if s is None else s[:m]


def exact(a, a_s, w, w_s, add, n, gated):
    k = a.shape[1]
    p, dp = X.product(a.double() * X.along(a_s, k), w.double() * X.spread(w_s, w.shape[0], k))
    if gated:
        return X.gated(p, dp, n)
    if add is not None:
        p = p + add.double()
        dp = dp + X.U * (p.abs() + dp)
    return p, dp


def verify(m, n, k, gated, out, addend=False, seed=1):
    say("dense", m, n, k, gated, out, addend)
    t = make(m, n, k, gated, seed, addend)
    v, dv = exact(*t, n, gated)
    o, s = run(*t, n, gated, out)
    if out == F8:
        X.check_fp8(o, s, v, dv)
    elif out == BF16:
        X.check_bf16(o, v, dv)
    else:
        bad = ~((o.double() - v).abs() <= dv + X.U * (v.abs() + dv))
        assert not bad.any(), (int(bad.sum()), o[bad][:4].tolist(), v[bad][:4].tolist())


SIZES = [(1, 128, 128), (1, 2048, 7168), (2, 256, 384), (3, 128, 1024), (7, 384, 640), (15, 256, 2048), (16, 512, 512),
         (17, 128, 4096), (31, 640, 256), (33, 256, 1536), (48, 128, 128), (63, 384, 2048), (64, 256, 1152), (65, 512, 896),
         (100, 1024, 2048), (127, 128, 512), (128, 2048, 1024), (129, 256, 256), (200, 384, 768), (255, 128, 1280),
         (257, 640, 384), (300, 2048, 2048), (511, 256, 128), (700, 1152, 640), (1025, 896, 512), (2049, 256, 384)]


@pytest.mark.parametrize("m,n,k", SIZES)
def test_gated_to_fp8(m, n, k):
    verify(m, n, k, True, F8)


@pytest.mark.parametrize("m,n,k", [(m, n + d, k) for (m, n, k), d in zip(SIZES, [0, 16, 32, 48, 64, 80, 96, 112, -16, 16] * 3)])
def test_gated_to_bf16(m, n, k):
    verify(m, n, k, True, BF16)


@pytest.mark.parametrize("m,n,k", [(m, n - d, k) for (m, n, k), d in zip(SIZES, [0, 16, 32, 48, 64, 80, 96, 112, 16] * 3)])
@pytest.mark.parametrize("out,addend", [(BF16, False), (BF16, True), (F32, False), (F32, True)])
def test_plain(m, n, k, out, addend):
    verify(m, n, k, False, out, addend)


@pytest.mark.parametrize("m", [1, 16, 40, 130, 600])
def test_narrow_and_long(m):
    verify(m, 16, 16384, False, F32, True)
    verify(m, 16, 8192, True, BF16)
    verify(m, 4112, 128, False, BF16)


def test_many_rows():
    verify(5000, 512, 512, True, F8)
    verify(4500, 1040, 256, False, F32, True)
    verify(8200, 160, 256, True, BF16)


@pytest.mark.parametrize("m", [0, 1, 20, 70, 300, 1500])
def test_no_rows_and_the_addend_in_place(m):
    t = make(m, 272, 384, False, addend=True)
    want, _ = run(*t, 272, False, F32)
    here = t[4].clone()
    got, _ = run(*t[:4], here, 272, False, F32, into=here)
    assert torch.equal(got, want)


@pytest.mark.parametrize("m", [1, 20, 140, 700, 2300])
@pytest.mark.parametrize("gated", [True, False])
def test_a_nan_stays_in_its_row(m, gated):
    t = make(m, 256, 512, gated)
    clean, _ = run(*t, 256, gated, BF16)
    a = t[0].clone()
    a.view(torch.uint8)[m // 2, 77] = 0x7F
    got, _ = run(a, *t[1:], 256, gated, BF16)
    rest = [i for i in range(m) if i != m // 2]
    assert torch.equal(got[rest], clean[rest])
    assert bool(got[m // 2].isnan().all())


@pytest.mark.parametrize("m", [1, 20, 140, 700])
def test_zeros_and_tiny_values_have_scales(m):
    a, a_s, w, w_s, _ = make(m, 256, 384, True)
    a = a.clone()
    a.view(torch.uint8)[0] = 0
    o, s = run(a, a_s, w, w_s, None, 256, True, F8)
    assert bool((s[0] == 0).all()) and bool((o[0].float() == 0).all())
    # every gate far below zero: silu's values are next to nothing
    w_s = w_s * 4e4
    v, dv = exact(a, a_s, w, w_s, None, 256, True)
    o, s = run(a, a_s, w, w_s, None, 256, True, F8)
    assert not bool(o.float().isnan().any()) and bool(s.isfinite().all())
    X.check_fp8(o, s, v, dv)


@pytest.mark.parametrize("m", [1, 20, 140, 700, 2300])
def test_captured_on_another_stream_and_two_at_once(m):
    t, u = make(m, 256, 640, True, 3), make(m, 384, 512, False, 4, True)
    want = run(*t, 256, True, F8)
    want_u, _ = run(*u, 384, False, F32)
    space, space_u = workspace(), workspace()
    o, s = torch.empty(m, 256, dtype=F8, device=DEV), torch.empty(m, 2, device=DEV)
    o_u = torch.empty(m, 384, device=DEV)
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        ll.ll_moe_dense_gemm(m, 256, 640, ll.ACT_SILU_MUL, ll.FP8_E4M3, *t, o, s, space)
    for _ in range(3):
        o.view(torch.uint8).fill_(0x7F)
        s.fill_(float("nan"))
        o_u.fill_(float("nan"))
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            ll.ll_moe_dense_gemm(m, 384, 512, ll.ACT_NONE, ll.FP32, *u, o_u, None, space_u)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o.view(torch.uint8), want[0].view(torch.uint8)) and torch.equal(s, want[1])
        assert torch.equal(o_u, want_u)
