"""Which scales the routing takes, without a GPU: every finite fp32."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")  # first: its HIP runtime is the one that the library then uses

import combine_ll_moe_amd as ll  # noqa: E402

MOST, TINY = float(np.finfo(np.float32).max), float(np.finfo(np.float32).smallest_subnormal)


def _status(scale):
    return ll.raw_status("ll_moe_route", 0, 64, 4, ll.FP32, ll.SCORE_SIGMOID, 8, 4, 2, 1, scale, 0, 0, 0, 0, 0, None)


@pytest.mark.parametrize("scale", [0.0, -0.0, 1.0, -2.5, TINY, 3.4e38, 3.402e38, MOST, -MOST])
def test_finite_scales_are_taken(scale):
    assert _status(scale) == ll.SUCCESS


@pytest.mark.parametrize("scale", [float("inf"), -float("inf"), float("nan")])
def test_others_are_refused(scale):
    assert _status(scale) == ll.INVALID_ARGUMENT
