"""The binding's checks of the expert-side operators' tensors, without a GPU:
stand-ins for device tensors, and a recorder in the library's place."""
import pytest

torch = pytest.importorskip("torch")  # first: its HIP runtime is the one that the library then uses

import combine_ll_moe_amd as ll  # noqa: E402


class Stand:
    """What the binding asks of a tensor on device 0."""

    def __init__(self, item, count):
        self.item, self.count = item, count

    def get_device(self):
        return 0

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 1 << 32

    def element_size(self):
        return self.item

    def numel(self):
        return self.count

    itemsize = property(element_size)
    nbytes = property(lambda self: self.item * self.count)


@pytest.fixture
def calls(monkeypatch):
    seen = []
    for name in ("ll_moe_expert_gemm", "ll_moe_expert_gemm_w4", "ll_moe_rms_norm"):
        monkeypatch.setattr(ll._lib, name, lambda *a, name=name: seen.append(name) or 0)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    return seen


E, CAP, N, K, T, H = 3, 5, 256, 384, 7, 512
# operand: (bytes of an element, elements that the call reads or writes)
BF16 = dict(a=(2, E * CAP * K), w=(2, E * N * K), counts=(4, E), out=(2, E * CAP * N))
FP8 = dict(a=(1, E * CAP * K), a_scales=(4, E * CAP * 3), w=(1, E * 2 * N * K), w_scales=(4, E * 4 * 3), counts=(4, E),
           out=(1, E * CAP * N), out_scales=(4, E * CAP * 2))
W4 = dict(a=(2, E * CAP * K), w=(1, E * 2 * N * K // 2), w_scales=(2, E * 2 * N * 6), w_zeros=(1, E * 2 * N * 6),
          counts=(4, E), out=(2, E * CAP * N))
NORM = dict(x=(4, T * H), residual=(2, T * H), weight=(2, H), residual_out=(2, T * H), out=(1, T * H),
            out_scales=(4, T * 4))


def _bf16(a, w, counts, out):
    ll.ll_moe_expert_gemm(CAP, N, K, E, ll.BF16, ll.ACT_NONE, ll.BF16, a, None, w, None, counts, out, stream=0)


def _fp8(a, a_scales, w, w_scales, counts, out, out_scales):
    ll.ll_moe_expert_gemm(CAP, N, K, E, ll.FP8_E4M3, ll.ACT_SILU_MUL, ll.FP8_E4M3, a, a_scales, w, w_scales, counts,
                          out, out_scales, stream=0)


def _w4(a, w, w_scales, w_zeros, counts, out):
    ll.ll_moe_expert_gemm_w4(CAP, N, K, E, 64, ll.ACT_SILU_MUL, a, w, w_scales, w_zeros, counts, out, stream=0)


def _norm(x, residual, weight, residual_out, out, out_scales):
    ll.ll_moe_rms_norm(T, H, ll.FP32, ll.FP8_E4M3, 1e-6, x, residual, weight, residual_out, out, out_scales, stream=0)


CALLS = [(_bf16, BF16), (_fp8, FP8), (_w4, W4), (_norm, NORM)]


@pytest.mark.parametrize("call,sizes", CALLS, ids=["bf16", "fp8", "w4", "norm"])
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


def test_raw_addresses_and_ignored_operands_are_not_measured(calls):
    t = {k: Stand(*v) for k, v in BF16.items()}
    _bf16(**{**t, "a": 4096})
    ll.ll_moe_expert_gemm(CAP, N, K, E, ll.BF16, ll.ACT_NONE, ll.BF16, t["a"], Stand(4, 1), t["w"], Stand(4, 1),
                          t["counts"], t["out"], Stand(4, 1), stream=0)
    n = {k: Stand(*v) for k, v in NORM.items()}
    _norm(**{**n, "residual": None, "residual_out": None})
    assert len(calls) == 3


@pytest.mark.parametrize("group", [0, -1, 96])
def test_a_wrong_group_is_the_library_s_to_refuse(calls, group):
    t = {k: Stand(*v) for k, v in W4.items()}
    ll.ll_moe_expert_gemm_w4(CAP, N, K, E, group, ll.ACT_SILU_MUL, t["a"], t["w"], t["w_scales"], t["w_zeros"],
                             t["counts"], t["out"], stream=0)
    assert calls == ["ll_moe_expert_gemm_w4"]
