"""The routing on the GPU against its definition, row by row in 64 bits."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - collected on CPU machines too
    pytest.skip("no GPU", allow_module_level=True)

import combine_ll_moe_amd as ll  # noqa: E402
import _router as R  # noqa: E402
from _gpu import DEV, say  # noqa: E402

INF, LOW = float("inf"), float(np.finfo(np.float32).min)


def run(logits, topk, sigmoid=True, bias=None, groups=1, topk_groups=1, best=1, renormalize=True, scale=1.0, valid=None,
        stream=None):
    t, e = logits.shape
    idx = torch.full((t + 1, topk), 77, dtype=torch.int32, device=DEV)  # a row behind, left as it is
    w = torch.full((t + 1, topk), 77.0, device=DEV)
    v = None if valid is None else torch.tensor([valid], dtype=torch.int32, device=DEV)
    ll.ll_moe_route(t, e, topk, ll.FP32 if logits.dtype == torch.float32 else ll.BF16,
                    ll.SCORE_SIGMOID if sigmoid else ll.SCORE_SOFTMAX, groups, topk_groups, best, renormalize, scale,
                    logits, bias, v, idx, w, stream=stream)
    torch.cuda.synchronize()
    assert bool((idx[t] == 77).all()) and bool((w[t] == 77).all())
    return idx[:t].cpu(), w[:t].cpu()


def verify(logits, topk, sigmoid=True, bias=None, groups=1, topk_groups=1, best=1, renormalize=True, scale=1.0,
           valid=None):
    idx, w = run(logits, topk, sigmoid, bias, groups, topk_groups, best, renormalize, scale, valid)
    R.check(idx, w, logits.float().cpu().numpy(), None if bias is None else bias.cpu().numpy(),
            len(logits) if valid is None else valid, topk, sigmoid, groups, topk_groups, best, renormalize, scale)
    return idx, w


def make(t, e, dtype=torch.float32, seed=1, bias=False, sigmoid=True):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn(t, e, generator=g, device=DEV) + torch.randn(e, generator=g, device=DEV) / 2
    b = (torch.randn(e, generator=g, device=DEV) * 30).round() * (1e-3 if sigmoid else 1e-3 / e) if bias else None
    return x.to(dtype), b


@pytest.mark.parametrize("e,topk,groups,topk_groups", [
    (1, 1, 1, 1), (2, 1, 2, 1), (3, 3, 1, 1), (8, 2, 1, 1), (16, 16, 1, 1), (60, 4, 6, 2), (63, 8, 1, 1), (64, 6, 8, 3),
    (65, 7, 1, 1), (72, 5, 4, 4), (128, 8, 8, 4), (160, 6, 8, 3), (161, 7, 7, 2), (255, 8, 1, 1), (256, 8, 8, 4),
    (256, 8, 1, 1), (256, 16, 64, 8), (257, 8, 1, 1), (384, 8, 8, 8), (512, 10, 4, 2), (1000, 8, 10, 3), (1024, 8, 1, 1),
    (1030, 9, 10, 2), (4096, 16, 64, 5)])
@pytest.mark.parametrize("sigmoid", [True, False])
@pytest.mark.parametrize("bias", [True, False])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_forms(e, topk, groups, topk_groups, sigmoid, bias, dtype):
    say("route", e, topk, groups, sigmoid, bias, dtype)
    x, b = make(13, e, dtype, e + topk, bias, sigmoid)
    for best in (1, 2):
        if groups > 1 and best > e // groups:
            continue
        verify(x, topk, sigmoid, b, groups, topk_groups, best, best == 1, 2.5 if best == 2 else 1.0, 11)


@pytest.mark.parametrize("t", [0, 1, 2, 3, 4, 5, 7, 63, 257, 1000])
@pytest.mark.parametrize("e,groups,topk_groups", [(256, 8, 4), (64, 1, 1), (40, 4, 2)])
def test_rows(t, e, groups, topk_groups):
    x, b = make(t, e, seed=t, bias=True)
    verify(x, 4, True, b, groups, topk_groups, 2, True, 2.5, max(0, t - 2))
    verify(x, 4, False, None, groups, topk_groups, 1, False, 1.0)


@pytest.mark.parametrize("valid", [-5, 0, 1, 9, 10, 1000])
def test_rows_behind_the_valid_ones(valid):
    x, b = make(10, 96, bias=True)
    x[9] = float("nan")
    idx, w = run(x, 4, bias=b, valid=valid)
    n = min(max(valid, 0), 10)
    R.check(idx, w, x.cpu().numpy(), b.cpu().numpy(), n, 4, True, 1, 1, 1, True, 1.0)


@pytest.mark.parametrize("e,groups,topk_groups", [(256, 8, 4), (64, 1, 1), (40, 4, 3), (512, 4, 2)])
@pytest.mark.parametrize("sigmoid", [True, False])
@pytest.mark.parametrize("best", [1, 2])
def test_masked_and_special_logits(e, groups, topk_groups, sigmoid, best):
    x, b = make(24, e, seed=5, bias=True, sigmoid=sigmoid)
    x[0] = -INF                      # nothing left
    x[1] = float("nan")
    x[2, :] = -INF
    x[2, e - 1] = 0.5                # one expert left
    x[3, ::2] = -INF                 # half masked
    x[4, 1::3] = float("nan")
    x[5] = LOW                       # the type's lowest value everywhere
    x[6, 1:] = LOW                   # all but one
    x[7, 3] = INF
    x[8, 3], x[8, e - 2] = INF, INF
    x[9] = INF
    x[10] = 0.25                     # all equal
    x[11, :e // 2] = x[11, 0]        # half equal
    x[12] = x[12].abs().round()      # few values
    x[13] = -800.0 - x[13].abs()     # every score underflows, renormalised or not
    x[14] = 1e4 * x[14]
    x[15, 2:] = -INF                 # fewer than topk
    x[16] = -INF
    x[16, :3] = LOW
    x[17] = -0.0
    x[17, ::3] = 0.0
    x[18] = 1e-42                    # subnormal
    for bias in (None, b):
        for renormalize in (True, False):
            verify(x, 4, sigmoid, bias, groups, topk_groups, best, renormalize, 1.5)


@pytest.mark.parametrize("groups,topk_groups,best", [(1, 1, 1), (4, 2, 2), (4, 2, 1)])
def test_special_biases(groups, topk_groups, best):
    x, b = make(16, 64, seed=9, bias=True)
    for at, v in ((3, -INF), (7, float("nan")), (12, INF), (13, INF), (40, 3e38), (50, -3e38), (20, LOW)):
        b[at] = v
        verify(x, 6, True, b, groups, topk_groups, best)
    b[:] = -INF
    idx, w = verify(x, 6, True, b, groups, topk_groups, best)
    assert bool((idx == -1).all()) and bool((w == 0).all())
    b[:] = 0.0
    verify(x, 6, True, b, groups, topk_groups, best)


def near_rows():
    """fp32 logits whose sigmoids with their biases are within fp32's rounding
    of each other, but not in 64 bits: l and b move against each other."""
    rng = np.random.default_rng(3)
    e, rows = 128, []
    l = rng.standard_normal((64, e)).astype(np.float32)
    target = 0.9
    b = (target - 1 / (1 + np.exp(-l[0].astype(np.float64)))).astype(np.float32)
    for t in range(64):
        row = l[0].copy()
        # single steps of the logits: the sums differ by some 1e-8
        steps = rng.integers(-3, 4, e)
        row = (row.view(np.int32) + steps.astype(np.int32)).view(np.float32)
        rows.append(row)
    return np.stack(rows), b


@pytest.mark.parametrize("groups,topk_groups,best", [(1, 1, 1), (8, 3, 2), (8, 3, 1)])
def test_scores_within_32_bit_rounding(groups, topk_groups, best):
    rows, b = near_rows()
    x, bias = torch.from_numpy(rows).to(DEV), torch.from_numpy(b).to(DEV)
    verify(x, 8, True, bias, groups, topk_groups, best, True, 1.0)
    # softmax: p + b alike, around the same sum
    p = np.exp(rows[0].astype(np.float64))
    bias = torch.from_numpy((0.5 - p / p.sum()).astype(np.float32)).to(DEV)
    verify(x, 8, False, bias, groups, topk_groups, best, False, 1.0)
    # without a bias, logits one step apart
    near = torch.from_numpy((np.full((8, 128), 1.0, np.float32).view(np.int32)
                             + np.random.default_rng(4).integers(-4, 5, (8, 128)).astype(np.int32)).view(np.float32)).to(DEV)
    verify(near, 8, True, None, groups, topk_groups, best)
    verify(near, 8, False, None, groups, topk_groups, best)


def test_many_equal_values():
    g = torch.Generator(device=DEV).manual_seed(2)
    x = torch.randint(0, 3, (64, 256), generator=g, device=DEV).to(torch.bfloat16)
    b = torch.randint(0, 2, (256,), generator=g, device=DEV).float() / 8
    for bias in (None, b):
        verify(x, 8, True, bias, 8, 4, 2)
        verify(x, 8, False, bias, 1, 1, 1)


@pytest.mark.parametrize("shape", [(3000, 256, 8, 8, 4, 2), (2500, 64, 6, 1, 1, 1), (2000, 160, 6, 8, 3, 1)])
def test_many_rows_match_a_second_call_on_another_stream(shape):
    t, e, k, groups, kept, best = shape
    x, b = make(t, e, bias=True)
    say("route many", shape)
    a = run(x, k, True, b, groups, kept, best)
    sample = torch.randperm(t)[:200]
    R.check(a[0][sample], a[1][sample], x[sample.to(DEV)].cpu().numpy(), b.cpu().numpy(), 200, k, True, groups, kept, best,
            True, 1.0)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    o = run(x, k, True, b, groups, kept, best, stream=s)
    assert torch.equal(a[0], o[0]) and torch.equal(a[1], o[1])


def test_captured_calls_follow_the_valid_count():
    x, b = make(40, 256, bias=True)
    valid = torch.tensor([40], dtype=torch.int32, device=DEV)
    idx, w = torch.empty(40, 8, dtype=torch.int32, device=DEV), torch.empty(40, 8, device=DEV)
    call = lambda: ll.ll_moe_route(40, 256, 8, ll.FP32, ll.SCORE_SIGMOID, 8, 4, 2, True, 2.5, x, b, valid, idx, w)  # noqa: E731
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for n in (40, 0, 17, 39):
        valid.fill_(n)
        idx.fill_(5)
        w.fill_(5)
        graph.replay()
        torch.cuda.synchronize()
        R.check(idx.cpu(), w.cpu(), x.cpu().numpy(), b.cpu().numpy(), n, 8, True, 8, 4, 2, True, 2.5)


def _sigmoid_near(target, rng):
    """fp32 logits whose sigmoids are within fp32's rounding of `target`."""
    x = np.float32(np.log(target / (1 - target)))
    return (x.view(np.int32) + np.int32(rng.integers(-3, 4))).view(np.float32)


@pytest.mark.parametrize("e,groups,topk_groups,best", [(256, 1, 1, 1), (256, 8, 4, 2), (128, 4, 2, 1), (100, 1, 1, 1),
                                                       (64, 16, 5, 2), (512, 2, 1, 2), (96, 8, 3, 2)])
@pytest.mark.parametrize("sigmoid", [True, False])
def test_single_pairs_within_32_bit_rounding(e, groups, topk_groups, best, sigmoid):
    """Each row has a pair of experts with different biases whose values differ
    by some 1e-8, among the largest: the choice of fp32 would be a toss."""
    rng = np.random.default_rng(e + groups)
    rows = rng.standard_normal((96, e)).astype(np.float32)
    bias = (rng.standard_normal(e) * 0.05).astype(np.float32)
    for t, row in enumerate(rows):
        a, c = rng.choice(e, 2, replace=False)
        if sigmoid:
            value = 0.9 + 0.01 * rng.random()
            row[a], row[c] = (_sigmoid_near(value - bias[x], rng) for x in (a, c))
        else:
            # their scores and biases sum up alike: p_c = p_a + b_a - b_c, the
            # rest of the row giving the sum
            rest = np.exp(np.delete(row.astype(np.float64), (a, c))).sum()
            pa = 0.3
            pc = pa + float(bias[a]) - float(bias[c])
            z = rest / (1 - pa - pc)
            row[a], row[c] = np.float32(np.log(pa * z)), np.float32(np.log(pc * z))
    x, b = torch.from_numpy(rows).to(DEV), torch.from_numpy(bias).to(DEV)
    verify(x, 4, sigmoid, b, groups, topk_groups, best, True, 1.0)
    verify(x, 1, sigmoid, b, groups, topk_groups, best, False, 2.0)


@pytest.mark.parametrize("e,groups,topk_groups", [(256, 8, 4), (128, 4, 1), (64, 16, 7), (512, 2, 1), (96, 8, 3), (60, 6, 2)])
@pytest.mark.parametrize("best", [1, 2])
@pytest.mark.parametrize("with_bias", [True, False])
def test_groups_within_32_bit_rounding(e, groups, topk_groups, best, with_bias):
    """The last group that stays and the first that does not differ by some
    1e-8; sometimes more than one of a group's members are near its best."""
    rng = np.random.default_rng(e + groups + best)
    rows = (rng.standard_normal((80, e)) - 1).astype(np.float32)
    bias = (rng.standard_normal(e) * 0.05).astype(np.float32) if with_bias else np.zeros(e, np.float32)
    per = e // groups
    for t, row in enumerate(rows):
        order = rng.permutation(groups)
        for place, g in enumerate(order):
            at = g * per + rng.choice(per, min(best + (t % 3 == 0), per), replace=False)
            # values fall from group to group, but for the border's two
            step = min(place, topk_groups - 1) if place <= topk_groups else place
            for x in at:
                row[x] = _sigmoid_near(0.75 - 0.02 * step - bias[x], rng)
    x = torch.from_numpy(rows).to(DEV)
    b = torch.from_numpy(bias).to(DEV) if with_bias else None
    verify(x, min(4, topk_groups * per), True, b, groups, topk_groups, best, True, 1.0)


@pytest.mark.parametrize("e,groups,topk_groups", [(64, 8, 3), (256, 8, 4), (256, 16, 5), (48, 4, 2), (32, 2, 1)])
@pytest.mark.parametrize("best", [1, 2])
@pytest.mark.parametrize("sigmoid", [True, False])
def test_groups_of_one_value(e, groups, topk_groups, best, sigmoid):
    """Groups whose best values are the same numbers, each once in its group:
    those of a smaller number stay."""
    g = torch.Generator(device=DEV).manual_seed(e + groups)
    per = e // groups
    x = -2.0 - torch.rand(40, e, generator=g, device=DEV)
    at = torch.rand(40, groups, per, generator=g, device=DEV).argsort(2) + torch.arange(groups, device=DEV)[:, None] * per
    for t in range(40):
        level = torch.randint(0, 3, (groups,), generator=g, device=DEV).float()  # three values for all groups
        x[t, at[t, :, 0]] = 1.0 + level / 4
        x[t, at[t, :, 1]] = 0.5 - level / 4 if t % 2 else 0.5 * torch.ones_like(level)
    for bias in (torch.zeros(e, device=DEV), torch.full((e,), 0.125, device=DEV), None):
        verify(x, 4, sigmoid, bias, groups, topk_groups, best)
        verify(x.bfloat16(), 4, sigmoid, bias, groups, topk_groups, best)


@pytest.mark.parametrize("best", [1, 2])
def test_groups_whose_values_and_members_are_near(best):
    """Scores of exactly 1/2 and biases, so that values are exact: members and
    groups some 1e-6 apart, in clusters of up to some 1e-5."""
    rng = np.random.default_rng(8)
    for t in range(60):
        wide = (2e-6, 6e-6, 2e-5)[t % 3]
        v = 0.2 + rng.uniform(-wide, wide, 64)
        v[rng.random(64) < 0.6] = 0.1  # a few members each
        b = torch.from_numpy((v - 0.5).astype(np.float32)).to(DEV)
        verify(torch.zeros(3, 64, device=DEV), 4, True, b, 4, 2, best)
    # one group clearly best, by less than what its two nearest members differ
    off = 2.0 ** -19 + 0.6 * 2.0 ** -20
    for above in np.arange(0.6, 2.6, 0.1):
        v = np.full((4, 16), 0.05)
        v[0, :3] = 0.3 - 0.9 * off * np.arange(3)
        total = v[0, 0] + (v[0, 1] if best == 2 else 0.0) - above * off
        for g, (first, less) in enumerate(((0.31, 0.0), (0.29, 0.4), (0.2, 40.0)), 1):
            v[g, 5] = first if best == 2 else total - less * off
            v[g, 6] = total - less * off - first if best == 2 else 0.01
        b = torch.from_numpy((v.ravel() - 0.5).astype(np.float32)).to(DEV)
        verify(torch.zeros(2, 64, device=DEV), 4, True, b, 4, 2, best)


@pytest.mark.parametrize("e,groups,topk_groups", [(64, 1, 1), (256, 1, 1), (256, 8, 4), (161, 1, 1), (512, 1, 1), (128, 2, 1)])
@pytest.mark.parametrize("sigmoid", [True, False])
def test_rows_of_many_equal_logits(e, groups, topk_groups, sigmoid):
    """Rows of zeros (tokens of padding), of two values, of a few above many."""
    g = torch.Generator(device=DEV).manual_seed(e)
    x = torch.randn(41, e, generator=g, device=DEV)
    x[1::4] = 0.0
    x[2::8] = x[2::8].round()
    x[3::8] = (x[3::8] > 1.5).float()
    x[6::8] = x[6::8].clamp(max=0.3)
    x[7, : e // 2] = -INF
    x[5, 20:] = -INF
    for topk in (1, 3, 8, 16):
        for dtype in (torch.float32, torch.bfloat16):
            verify(x.to(dtype), topk, sigmoid, None, groups, topk_groups, 1, topk == 8)
