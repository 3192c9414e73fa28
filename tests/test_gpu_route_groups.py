"""Groups that count by their best two, on the GPU against the definition in 64
bits: groups whose own best members are equal or near, clear of a border
between two groups that are equal or near."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - collected on CPU machines too
    pytest.skip("no GPU", allow_module_level=True)

import combine_ll_moe_amd as ll  # noqa: E402
import _router as R  # noqa: E402
from _gpu import DEV, say  # noqa: E402

INF, MOST = float("inf"), float(np.finfo(np.float32).max)


def run(logits, topk, sigmoid, bias, groups, topk_groups, best=2, renormalize=True, scale=1.0):
    t, e = logits.shape
    idx, w = torch.full((t, topk), 77, dtype=torch.int32, device=DEV), torch.full((t, topk), 77.0, device=DEV)
    ll.ll_moe_route(t, e, topk, ll.FP32 if logits.dtype == torch.float32 else ll.BF16,
                    ll.SCORE_SIGMOID if sigmoid else ll.SCORE_SOFTMAX, groups, topk_groups, best, renormalize, scale,
                    logits, bias, None, idx, w)
    torch.cuda.synchronize()
    return idx.cpu(), w.cpu()


def verify(logits, topk, sigmoid, bias, groups, topk_groups, best=2, renormalize=True, scale=1.0):
    """Row by row, in plain Python."""
    idx, w = run(logits, topk, sigmoid, bias, groups, topk_groups, best, renormalize, scale)
    R.check(idx, w, logits.float().cpu().numpy(), None if bias is None else bias.cpu().numpy(), len(logits), topk, sigmoid,
            groups, topk_groups, best, renormalize, scale)


def scores(l, sigmoid):
    l = l.astype(np.float64)
    if sigmoid:
        return 1 / (1 + np.exp(-l))
    p = np.exp(l - l.max(1, keepdims=True))
    return p / p.sum(1, keepdims=True)


def verify_rows(logits, topk, sigmoid, bias, groups, topk_groups):
    """The same for many rows of finite logits at once: stable sorts in 64
    bits, best two a group, renormalised. Tolerance of the weights: as in
    R.check, for the same reasons."""
    idx, w = run(logits, topk, sigmoid, bias, groups, topk_groups)
    l = logits.float().cpu().numpy()
    t, e = l.shape
    s = scores(l, sigmoid)
    v = s if bias is None else s + bias.cpu().numpy().astype(np.float64)
    two = -np.sort(-v.reshape(t, groups, -1), axis=2)[..., :2].sum(2)
    kept = np.argsort(-two, axis=1, kind="stable")[:, :topk_groups]
    inside = np.zeros((t, groups), bool)
    np.put_along_axis(inside, kept, True, 1)
    order = np.where(np.repeat(inside, e // groups, 1), l.astype(np.float64) if bias is None else v, -INF)
    want = np.argsort(-order, axis=1, kind="stable")[:, :topk]
    bad = (idx.numpy() != want).any(1)
    assert not bad.any(), (int(bad.sum()), np.flatnonzero(bad)[:4], idx.numpy()[bad][:2], want[bad][:2])
    x = np.take_along_axis(s, want, 1)
    x /= x.sum(1, keepdims=True)
    assert (np.abs(w.numpy() - x) <= x * (2.0 ** -24 + 2.0 ** -30)).all()


SHAPES = [(64, 4, 2), (256, 8, 4), (128, 8, 3), (64, 16, 5), (256, 16, 8), (512, 2, 1), (96, 8, 3), (48, 4, 3), (32, 16, 4),
          (60, 6, 3)]


@pytest.mark.parametrize("e,groups,topk_groups", SHAPES)
@pytest.mark.parametrize("sigmoid", [True, False])
@pytest.mark.parametrize("members", [2, 3])
def test_equal_members_clear_of_a_tied_border(e, groups, topk_groups, sigmoid, members):
    """Logits alone. One group clear of the border, or all of those, have two or
    three members of one value, or a step of fp32 apart; the border's two groups
    have one of 2 and one of 1/4 each, equal or a step apart."""
    say("tied members", e, groups, topk_groups, sigmoid, members)
    rng = np.random.default_rng(e + groups + members)
    per = e // groups
    members = min(members, per)
    rows = np.full((64, e), -5.0, np.float32)
    for t, row in enumerate(rows):
        # side by side (one lane, where that has so many) or anywhere in the group
        at = [g * per + (np.arange(members) + rng.integers(per - members + 1) if t % 2 else
                         rng.choice(per, members, replace=False)) for g in rng.permutation(groups)]
        clear = [p for p in range(groups) if not topk_groups - 1 <= p <= topk_groups]
        tied = clear if t % 4 == 0 or not clear else [clear[t % len(clear)] if t % 4 == 1 else clear[0]]
        for place, x in enumerate(at):
            if place in clear:
                row[x] = np.float32(3 + place) if place < topk_groups else np.float32(-1 - place / 8)
                if place not in tied:
                    row[x[1:]] -= np.arange(1, members, dtype=np.float32) / 2
            else:
                row[x[:2]] = 2.0, 0.25
        for x in [at[topk_groups]] if t % 8 < 4 else [at[topk_groups - 1], *(at[p] for p in tied)]:
            row[x[1]] = np.nextafter(row[x[1]], np.float32(-INF))
    x = torch.from_numpy(rows).to(DEV)
    for bias in (None, torch.zeros(e, device=DEV), torch.full((e,), 0.125, device=DEV)):
        verify(x, min(4, topk_groups * per), sigmoid, bias, groups, topk_groups)
        verify(x, min(7, topk_groups * per), sigmoid, bias, groups, topk_groups, 1, False, 2.5)
    verify(x.bfloat16(), min(4, topk_groups * per), sigmoid, None, groups, topk_groups)


@pytest.mark.parametrize("e,groups,topk_groups", SHAPES)
@pytest.mark.parametrize("sigmoid", [True, False])
def test_near_members_clear_of_a_near_border_with_a_bias(e, groups, topk_groups, sigmoid):
    """Values are set by the bias: score + bias is a level of the member's group,
    to the bias's rounding (some 1e-8); logits move by single steps from row to
    row. One group clear of the border, or all of those, have two or three members of
    one level."""
    say("near members", e, groups, topk_groups, sigmoid)
    rng = np.random.default_rng(3 * e + groups)
    per = e // groups
    for draw in range(24):
        base = rng.standard_normal(e).astype(np.float32)
        level = np.full(e, -0.5) - 0.3 * rng.random(e)
        tied = 0 if draw % 2 else None  # the first group alone, or all that are clear
        for place, g in enumerate(rng.permutation(groups)):
            at = g * per + rng.choice(per, min(2 + draw % 3 % 2, per), replace=False)
            if topk_groups - 1 <= place <= topk_groups:
                level[at] = 0.1
                level[at[:2]] = 0.5, 0.3
            else:
                level[at] = 0.7 + 0.02 * (groups - place) if place < topk_groups else 0.2 - 0.01 * place
                if tied is not None and place != tied:
                    level[at[1:]] -= 0.05 * np.arange(1, len(at))
                elif draw % 4 >= 2:
                    base[at] = base[at[0]]  # the same bias, too: the same number
        bias = (level - scores(base[None], sigmoid)[0]).astype(np.float32)
        steps = rng.integers(-2, 3, (6, e)).astype(np.int32)
        steps[0] = 0
        x = torch.from_numpy((base.view(np.int32) + steps).view(np.float32)).to(DEV)
        verify(x, min(4, topk_groups * per), sigmoid, torch.from_numpy(bias).to(DEV), groups, topk_groups)


@pytest.mark.parametrize("e,groups,topk_groups,t,steps", [
    (256, 8, 4, 16384, 16), (256, 8, 4, 4096, 8), (256, 8, 4, 4096, 4), (64, 4, 2, 4096, 4), (64, 4, 2, 4096, 16),
    (512, 4, 2, 2048, 16), (96, 8, 3, 4096, 8), (128, 16, 6, 4096, 8), (256, 2, 1, 2048, 2)])
@pytest.mark.parametrize("sigmoid", [True, False])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_coarse_logits(e, groups, topk_groups, t, steps, sigmoid, dtype):
    """Logits on a grid, so that members are often equal. The grid is a third
    of a step off zero: sums of different scores are not equal by symmetry."""
    say("coarse", e, groups, topk_groups, t, steps, sigmoid, dtype)
    g = torch.Generator(device=DEV).manual_seed(e + t + steps)
    x = ((torch.randn(t, e, generator=g, device=DEV) * steps).round() + 1 / 3) / steps
    verify_rows(x.to(dtype), 8, sigmoid, None, groups, topk_groups)


@pytest.mark.parametrize("e,groups,topk_groups", [(256, 8, 4), (64, 4, 2), (128, 16, 6)])
@pytest.mark.parametrize("sigmoid", [True, False])
def test_rows_of_zeros_with_a_stepped_bias(e, groups, topk_groups, sigmoid):
    """Tokens of padding under a balancing bias, which moves by fixed steps."""
    rng = np.random.default_rng(e)
    x = torch.zeros(2, e, device=DEV)
    for _ in range(300):
        b = (np.round(rng.standard_normal(e) * 30) * 1e-3).astype(np.float32)
        verify_rows(x, 8, sigmoid, torch.from_numpy(b).to(DEV), groups, topk_groups)


@pytest.mark.parametrize("e,groups,topk_groups", SHAPES)
@pytest.mark.parametrize("sigmoid", [True, False])
def test_sums_of_two_beyond_fp32(e, groups, topk_groups, sigmoid):
    """Biases that mask by the type's lowest value and others as large: a
    group's sum of two leaves fp32, but it stands before a group that has fewer
    than two experts left, and in its place among the others."""
    say("sums beyond fp32", e, groups, topk_groups, sigmoid)
    rng = np.random.default_rng(e + groups)
    per = e // groups
    for draw in range(24):
        x = rng.standard_normal((5, e)).astype(np.float32)
        x[1] = 0.5
        x[2, ::2] = -INF
        x[3, : e // 2] = -MOST
        b = (rng.standard_normal((groups, per)) * 0.05).astype(np.float32)
        for g in range(groups):
            kind = rng.integers(0, 7) if draw % 2 else (0, 1, 2, 0)[g % 4]
            if kind == 0:
                b[g] = -INF                               # none left
            elif kind == 1:
                b[g] = -MOST                              # all masked by the lowest value
            elif kind == 2:
                b[g] = -3e38 + 1e37 * rng.integers(0, 3)  # sums beyond it, of different size
            elif kind == 3:
                b[g] = 3e38
            elif kind == 4:
                b[g, 1:] = -INF                           # one left
            elif kind == 5:
                b[g, ::2] = -MOST
        bias = torch.from_numpy(b.ravel()).to(DEV)
        verify(torch.from_numpy(x).to(DEV), min(4, topk_groups * per), sigmoid, bias, groups, topk_groups)


@pytest.mark.parametrize("sigmoid", [True, False])
@pytest.mark.parametrize("renormalize", [True, False])
def test_the_largest_scale(sigmoid, renormalize):
    """Scores are at most 1, so weights stay finite."""
    g = torch.Generator(device=DEV).manual_seed(6)
    x = torch.randn(9, 64, generator=g, device=DEV)
    x[1], x[2] = 0.0, -200.0
    x[3, 5], x[4, 1:] = INF, -INF
    for groups, topk_groups in ((8, 4), (1, 1)):
        verify(x, 6, sigmoid, None, groups, topk_groups, 1, renormalize, MOST)
        verify(x, 1, sigmoid, torch.zeros(64, device=DEV), groups, topk_groups, 2, renormalize, -MOST)


@pytest.mark.parametrize("e,groups,topk_groups,best", [(256, 1, 1, 1), (256, 8, 4, 2), (128, 4, 2, 1), (100, 1, 1, 1),
                                                       (64, 16, 5, 2), (512, 2, 1, 2), (96, 8, 3, 2)])
def test_single_near_pairs_that_exist(e, groups, topk_groups, best):
    """A pair of experts with different biases whose sigmoids with them differ
    by some 1e-8, among the largest; biases are within 0.05, so that the scores
    that make such a pair, 0.9 less the bias, lie between 0 and 1."""
    rng = np.random.default_rng(e + groups)
    rows = (rng.standard_normal((96, e)) - 1).astype(np.float32)
    bias = (rng.standard_normal(e) * 0.02).clip(-0.05, 0.05).astype(np.float32)
    for row in rows:
        a, c = rng.choice(e, 2, replace=False)
        value = 0.9 + 0.01 * rng.random()
        for x in (a, c):
            target = value - float(bias[x])
            assert 0 < target < 1
            l = np.float32(np.log(target / (1 - target)))
            row[x] = (l.view(np.int32) + np.int32(rng.integers(-3, 4))).view(np.float32)
    x, b = torch.from_numpy(rows).to(DEV), torch.from_numpy(bias).to(DEV)
    assert bool(x.isfinite().all())
    verify(x, 4, True, b, groups, topk_groups, best)
    verify(x, 1, True, b, groups, topk_groups, best, False, 2.0)
