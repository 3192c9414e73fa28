"""The binding's checks of the router's and the dense products' tensors,
without a GPU: stand-ins for device tensors, and a recorder in the library's
place."""
import pytest

torch = pytest.importorskip("torch")  # first: its HIP runtime is the one that the library then uses

import combine_ll_moe_amd as ll  # noqa: E402
from test_binding_experts import Stand  # noqa: E402

T, H, E, K, N, KK = 5, 64, 24, 3, 256, 384
# operand: (bytes of an element, elements that the call reads or writes)
GATE = dict(x=(2, T * H), weight=(4, E * H), logits=(4, T * E))
ROUTE = dict(logits=(2, T * E), bias=(4, E), num_valid=(4, 1), topk_idx=(4, T * K), topk_weights=(4, T * K))
FP8 = dict(a=(1, T * KK), a_scales=(4, T * 3), w=(1, 2 * N * KK), w_scales=(4, 4 * 3), out=(1, T * N), out_scales=(4, T * 2))
FP32 = dict(a=(1, T * KK), a_scales=(4, T * 3), w=(1, N * KK), w_scales=(4, 2 * 3), addend=(4, T * N), out=(4, T * N))
SPACE = Stand(1, ll.DENSE_WORKSPACE)


@pytest.fixture
def calls(monkeypatch):
    seen = []
    for name in ("ll_moe_gate", "ll_moe_route", "ll_moe_dense_gemm"):
        monkeypatch.setattr(ll._lib, name, lambda *a, name=name: seen.append(name) or 0)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    return seen


def _gate(x, weight, logits):
    ll.ll_moe_gate(T, H, E, ll.FP32, x, weight, logits, stream=0)


def _route(logits, bias, num_valid, topk_idx, topk_weights):
    ll.ll_moe_route(T, E, K, ll.BF16, ll.SCORE_SIGMOID, 4, 2, 2, True, 2.5, logits, bias, num_valid, topk_idx,
                    topk_weights, stream=0)


def _fp8(a, a_scales, w, w_scales, out, out_scales):
    ll.ll_moe_dense_gemm(T, N, KK, ll.ACT_SILU_MUL, ll.FP8_E4M3, a, a_scales, w, w_scales, None, out, out_scales, SPACE,
                         stream=0)


def _fp32(a, a_scales, w, w_scales, addend, out):
    ll.ll_moe_dense_gemm(T, N, KK, ll.ACT_NONE, ll.FP32, a, a_scales, w, w_scales, addend, out, None, SPACE, stream=0)


CALLS = [(_gate, GATE), (_route, ROUTE), (_fp8, FP8), (_fp32, FP32)]


@pytest.mark.parametrize("call,sizes", CALLS, ids=["gate", "route", "fp8", "fp32"])
def test_whole_and_larger_tensors_pass(calls, call, sizes):
    call(**{k: Stand(*v) for k, v in sizes.items()})
    call(**{k: Stand(v[0], v[1] + 9) for k, v in sizes.items()})
    assert len(calls) == 2


@pytest.mark.parametrize("call,sizes,name", [(c, s, n) for c, s in CALLS for n in s])
def test_a_short_tensor_or_another_type_is_refused(calls, call, sizes, name):
    item, count = sizes[name]
    for bad in (Stand(item, count - 1), Stand(2 * item, count), Stand(8, count)):
        with pytest.raises(ll.LLMoEError) as ei:
            call(**{**{k: Stand(*v) for k, v in sizes.items()}, name: bad})
        assert ei.value.status == ll.INVALID_ARGUMENT
    assert not calls


def test_a_short_workspace_is_refused(calls):
    t = {k: Stand(*v) for k, v in FP32.items()}
    for space in (Stand(1, ll.DENSE_WORKSPACE - 1), Stand(4, ll.DENSE_WORKSPACE // 4 - 1)):
        with pytest.raises(ll.LLMoEError):
            ll.ll_moe_dense_gemm(T, N, KK, ll.ACT_NONE, ll.FP32, *t.values(), None, space, stream=0)
    ll.ll_moe_dense_gemm(T, N, KK, ll.ACT_NONE, ll.FP32, *t.values(), None, Stand(4, ll.DENSE_WORKSPACE // 4), stream=0)
    assert len(calls) == 1


def test_operands_that_may_be_missing(calls):
    t = {k: Stand(*v) for k, v in ROUTE.items()}
    _route(**{**t, "bias": None, "num_valid": None})
    d = {k: Stand(*v) for k, v in FP32.items()}
    _fp32(**{**d, "addend": None})
    assert len(calls) == 2
