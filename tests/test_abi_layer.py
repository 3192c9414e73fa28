"""Refusals of the router and the dense products, without a GPU: every case
fails validation before anything is enqueued."""
import pytest

torch = pytest.importorskip("torch")  # first: its HIP runtime is the one that the library then uses

import combine_ll_moe_amd as ll  # noqa: E402

M = 1 << 32  # addresses far apart, never dereferenced
NAN, INF = float("nan"), float("inf")


def _gate(**kw):
    a = dict(t=16, h=1024, e=64, w_dtype=0, x=M, w=2 * M, logits=3 * M)
    a.update(kw)
    return ll.raw_status("ll_moe_gate", *a.values(), None)


def _route(**kw):
    a = dict(t=16, e=64, topk=4, dtype=2, score=1, groups=8, kept=4, best=2, renormalize=1, scale=1.0, logits=M, bias=2 * M,
             valid=3 * M, idx=4 * M, weights=5 * M)
    a.update(kw)
    return ll.raw_status("ll_moe_route", *a.values(), None)


def _dense(**kw):
    a = dict(t=16, n=256, k=512, act=0, out_dtype=2, a=M, a_s=2 * M, w=3 * M, w_s=4 * M, add=5 * M, out=6 * M, out_s=0,
             space=8 * M)
    a.update(kw)
    return ll.raw_status("ll_moe_dense_gemm", *a.values(), None)


def _fp8(**kw):
    return _dense(**{**dict(act=1, out_dtype=1, add=0, out_s=7 * M), **kw})


@pytest.mark.parametrize("case", [
    dict(t=-1), dict(h=0), dict(h=-8), dict(h=1020), dict(h=32776), dict(e=0), dict(e=-1), dict(e=4097), dict(w_dtype=1),
    dict(w_dtype=3), dict(w_dtype=-1), dict(x=0), dict(w=0), dict(logits=0), dict(x=M + 8), dict(w=2 * M + 4),
    dict(logits=3 * M + 8), dict(logits=M), dict(logits=M + 16 * 1024 * 2 - 16), dict(logits=2 * M),
    dict(logits=2 * M - 16), dict(w_dtype=2, logits=2 * M + 64 * 1024 * 2),
])
def test_gate_refuses(case):
    assert _gate(**case) == ll.INVALID_ARGUMENT


@pytest.mark.parametrize("case", [
    dict(t=-1), dict(e=0), dict(e=4104), dict(topk=0), dict(topk=17), dict(topk=33), dict(dtype=1), dict(dtype=3),
    dict(score=2), dict(score=-1), dict(groups=0), dict(groups=65, e=130), dict(groups=7), dict(groups=-8), dict(kept=0),
    dict(kept=9), dict(best=0), dict(best=3), dict(groups=64, kept=64), dict(topk=9, kept=1), dict(renormalize=2),
    dict(renormalize=-1), dict(scale=NAN), dict(scale=INF), dict(scale=-INF), dict(logits=0), dict(idx=0),
    dict(weights=0), dict(logits=M + 8), dict(bias=2 * M + 2), dict(valid=3 * M + 1), dict(idx=4 * M + 2),
    dict(weights=5 * M + 2), dict(idx=M), dict(weights=M + 16 * 64 * 4 - 4), dict(idx=2 * M), dict(weights=3 * M),
    dict(weights=4 * M + 252), dict(t=1 << 30), dict(e=3, groups=1, kept=1, topk=4),
])
def test_route_refuses(case):
    assert _route(**case) == ll.INVALID_ARGUMENT


@pytest.mark.parametrize("case", [
    dict(t=-1), dict(n=0), dict(n=8), dict(n=24), dict(n=(1 << 20) + 16), dict(k=0), dict(k=64), dict(k=200),
    dict(k=(1 << 20) + 128), dict(act=2), dict(act=-1), dict(out_dtype=1), dict(out_dtype=3), dict(a=0), dict(a_s=0),
    dict(w=0), dict(w_s=0), dict(out=0), dict(space=0), dict(a=M + 8), dict(a_s=2 * M + 2), dict(w=3 * M + 8),
    dict(w_s=4 * M + 1), dict(add=5 * M + 8), dict(out=6 * M + 4), dict(space=8 * M + 8), dict(out=M), dict(out=2 * M),
    dict(out=3 * M), dict(out=4 * M), dict(out=5 * M + 16), dict(out=5 * M - 16), dict(out=5 * M, out_dtype=0),
    dict(space=M), dict(space=3 * M), dict(space=5 * M), dict(space=6 * M), dict(space=6 * M - (64 << 20) + 16),
])
def test_dense_refuses(case):
    assert _dense(**case) == ll.INVALID_ARGUMENT


@pytest.mark.parametrize("case", [
    dict(add=5 * M), dict(out_dtype=2), dict(out_dtype=3), dict(n=144), dict(out_s=0), dict(out_s=7 * M + 2),
    dict(out_s=6 * M), dict(out_s=2 * M), dict(out_s=8 * M + 16), dict(add=5 * M, out_dtype=0),
])
def test_gated_dense_refuses(case):
    assert _fp8(**case) == ll.INVALID_ARGUMENT


def test_empty_calls_need_no_gpu():
    assert _gate(t=0, x=0, logits=0) == ll.SUCCESS
    assert _route(t=0, logits=0, idx=0, weights=0) == ll.SUCCESS
    assert _dense(t=0, a=0, out=0, space=0) == ll.SUCCESS
    assert _gate(t=0, h=12) == _route(t=0, topk=0) == _dense(t=0, k=100) == ll.INVALID_ARGUMENT


def test_host_tensors_are_refused():
    x, w, l = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(8, 64, dtype=torch.bfloat16), torch.zeros(4, 8)
    i = torch.zeros(4, 2, dtype=torch.int32)
    for call in (lambda: ll.ll_moe_gate(4, 64, 8, ll.BF16, x, w, l, stream=0),
                 lambda: ll.ll_moe_route(4, 8, 2, ll.FP32, 0, 1, 1, 1, True, 1.0, l, None, None, i, l, stream=0)):
        with pytest.raises(ll.LLMoEError) as ei:
            call()
        assert ei.value.status == ll.INVALID_ARGUMENT
