"""Refusals of the operators around the expert side, without a GPU: every case
fails validation before anything is enqueued."""
import pytest

torch = pytest.importorskip("torch")  # first: its HIP runtime is the one that the library then uses

import combine_ll_moe_amd as ll  # noqa: E402

M = 1 << 32  # addresses far apart, never dereferenced


def _gemm(**kw):
    a = dict(cap=128, n=256, k=512, e=8, dtype=0, act=0, out_dtype=0, a=M, a_scales=0, w=2 * M, w_scales=0,
             counts=3 * M, out=4 * M, out_scales=0)
    a.update(kw)
    return ll.raw_status("ll_moe_expert_gemm", *a.values(), None)


def _fp8(**kw):
    return _gemm(**{**dict(dtype=1, act=1, out_dtype=1, a_scales=5 * M, w_scales=6 * M, out_scales=7 * M), **kw})


def _w4(**kw):
    a = dict(cap=128, n=256, k=512, e=8, group=64, act=0, a=M, w=2 * M, s=3 * M, z=4 * M, counts=5 * M, out=6 * M)
    a.update(kw)
    return ll.raw_status("ll_moe_expert_gemm_w4", *a.values(), None)


def _norm(**kw):
    a = dict(t=16, h=1024, x_dtype=0, out_dtype=0, eps=1e-6, x=M, res=2 * M, w=3 * M, new=4 * M, out=5 * M, scales=6 * M)
    a.update(kw)
    return ll.raw_status("ll_moe_rms_norm", *a.values(), None)


@pytest.mark.parametrize("case", [
    dict(cap=0), dict(cap=-1), dict(n=0), dict(n=12), dict(n=(1 << 20) + 8), dict(k=0), dict(k=12),
    dict(k=(1 << 20) + 8), dict(e=0), dict(e=4097), dict(cap=1 << 30), dict(dtype=2), dict(dtype=-1), dict(act=2),
    dict(act=-1), dict(out_dtype=1), dict(out_dtype=2), dict(a=0), dict(w=0), dict(counts=0), dict(out=0),
    dict(a=M + 8), dict(w=2 * M + 4), dict(counts=3 * M + 2), dict(out=4 * M + 8),
    dict(out=M), dict(out=M - 16), dict(out=2 * M + 16), dict(out=M + 128 * 8 * 512 * 2 - 16), dict(counts=4 * M + 64),
])
def test_gemm_refuses(case):
    assert _gemm(**case) == ll.INVALID_ARGUMENT


@pytest.mark.parametrize("case", [
    dict(k=64), dict(k=192), dict(n=136), dict(n=144), dict(act=0), dict(a_scales=0), dict(w_scales=0),
    dict(out_scales=0), dict(a_scales=5 * M + 2), dict(w_scales=6 * M + 1), dict(out_scales=7 * M + 2),
    dict(out_scales=4 * M), dict(out_scales=5 * M), dict(out_scales=6 * M), dict(out=5 * M), dict(n=24, out_dtype=0),
])
def test_fp8_gemm_refuses(case):
    assert _fp8(**case) == ll.INVALID_ARGUMENT


@pytest.mark.parametrize("case", [
    dict(group=16), dict(group=0), dict(group=256), dict(k=544), dict(n=4), dict(act=3), dict(e=0), dict(a=0),
    dict(w=0), dict(s=0), dict(counts=0), dict(out=0), dict(a=M + 2), dict(w=2 * M + 8), dict(s=3 * M + 8), dict(z=4 * M + 4),
    dict(counts=5 * M + 1), dict(out=6 * M + 4), dict(out=4 * M), dict(out=3 * M), dict(out=2 * M), dict(cap=1 << 29),
    dict(cap=1, e=1, n=1 << 20, k=1 << 15, group=32, out=1 << 50, w=1 << 51),
])
def test_w4_gemm_refuses(case):
    assert _w4(**case) == ll.INVALID_ARGUMENT


@pytest.mark.parametrize("case", [
    dict(t=-1), dict(h=0), dict(h=1020), dict(h=32776), dict(x_dtype=1), dict(x_dtype=3), dict(out_dtype=2),
    dict(out_dtype=1, h=1032), dict(eps=-1e-6), dict(eps=float("nan")), dict(eps=float("inf")), dict(x=0), dict(w=0),
    dict(out=0), dict(out_dtype=1, scales=0), dict(x=M + 8), dict(res=2 * M + 8), dict(w=3 * M + 2),
    dict(new=4 * M + 8), dict(out=5 * M + 4), dict(out_dtype=1, scales=6 * M + 2), dict(out=M), dict(out=2 * M),
    dict(new=M), dict(new=2 * M + 16), dict(out=4 * M), dict(out=3 * M), dict(x_dtype=2, out=M + 16 * 1024 * 2),
    dict(out_dtype=1, scales=5 * M),
])
def test_norm_refuses(case):
    assert _norm(**case) == ll.INVALID_ARGUMENT


def test_host_tensors_are_refused():
    b = torch.zeros(4, 64, dtype=torch.bfloat16)
    w = torch.zeros(64, dtype=torch.bfloat16)
    with pytest.raises(ll.LLMoEError) as ei:
        ll.ll_moe_rms_norm(4, 64, ll.BF16, ll.BF16, 1e-6, b, None, w, None, torch.zeros_like(b), stream=0)
    assert ei.value.status == ll.INVALID_ARGUMENT
    assert ll._operands("call", 7, 4096, None) == [4096, None, 7]


def test_empty_norm_needs_no_gpu():
    assert _norm(t=0, x=0, out=0, res=0, new=0) == ll.SUCCESS
