"""Sums of the fp8 and 4-bit products on the GPU: fp32 in every kernel, so that a
row's result does not depend on how many rows its expert has; every code and
zero point."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - collected on CPU machines too
    pytest.skip("no GPU", allow_module_level=True)

import combine_ll_moe_amd as ll  # noqa: E402
from _gpu import DEV, say  # noqa: E402
from test_gpu_experts import Gemm  # noqa: E402

BF16, F8 = torch.bfloat16, torch.float8_e4m3fn


def _inputs(rows, rw, k, seed):
    """Codes whose products are multiples of 2^-6 of at most 2^14, the large
    ones in pairs that cancel: with scales of 1, every partial sum in any
    order is a multiple of 2^-6 below 2^16 (a 128-column block has 4 large
    products and 124 of at most 1/2), 22 bits, so fp32 sums are exact."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    ri = lambda lo, hi, *s: torch.randint(lo, hi, s, generator=g, device=DEV)  # noqa: E731
    a = ri(-4, 5, rows, k) / 8.0   # multiples of 2^-3, at most 1/2
    w = ri(-4, 5, rw, k) / 8.0
    for block in range(0, k, 128):
        at = block + torch.randperm(128, generator=g, device=DEV)[:4]
        a[:, at] = 128.0 * torch.tensor([1, 1, -1, -1], device=DEV)
        w[:, at] = 128.0 * torch.tensor([1, -1, 1, -1], device=DEV)
    return a, w


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("n,k", [(144, 128), (256, 640)])
def test_fp8_sums_are_fp32_in_every_kernel(gated, n, k):
    """The same 300 rows in one expert (whole tiles and 44 rows behind them)
    and dealt to experts of up to 60: the same bits, and plain products equal
    to the exact ones rounded once."""
    say("case", gated, n, k)
    cap, rows, rw = 300, 300, 2 * n if gated else n
    a, w = _inputs(rows, rw, k, n + k)
    counts = [300, 60, 60, 60, 60, 60]
    at = torch.cat([torch.arange(300), *[e * cap + torch.arange(60) for e in range(1, 6)]]).to(DEV)
    x = torch.full((6 * cap, k), 0x7F, dtype=torch.uint8, device=DEV)
    x[at] = torch.cat([a, a]).to(F8).view(torch.uint8)
    xs = torch.ones(6 * cap, k // 128, device=DEV)
    ws = torch.ones(6, -(-rw // 128), k // 128, device=DEV)
    w8 = w.to(F8).view(torch.uint8).repeat(6, 1, 1).view(F8)
    out = torch.zeros(6 * cap, n, dtype=BF16, device=DEV)
    ll.ll_moe_expert_gemm(cap, n, k, 6, ll.FP8_E4M3, ll.ACT_SILU_MUL if gated else ll.ACT_NONE, ll.BF16, x.view(F8), xs,
                          w8, ws, torch.tensor(counts, dtype=torch.int32, device=DEV), out)
    torch.cuda.synchronize()
    got = out[at]
    if not gated:
        want = (a.double() @ w.double().t()).float().to(BF16)  # fp32 holds the exact sum
        assert torch.equal(got[:300], want) and torch.equal(got[300:], want), \
            (int((got[:300] != want).sum()), int((got[300:] != want).sum()))
    assert torch.equal(got[:300], got[300:]), int((got[:300] != got[300:]).sum())


@pytest.mark.parametrize("side", ["weights", "activations"])
def test_every_e4m3_code(side):
    """One product a sum: all 256 codes, subnormals and NaN among them, come out
    as the values they stand for (bf16 holds each), in few rows and in tiles."""
    say("case", side)
    cap, n, k = 300, 256, 128
    codes = torch.arange(256, dtype=torch.uint8, device=DEV)
    one = torch.ones((), device=DEV).to(F8).view(torch.uint8)
    counts = [300, 60]
    x = torch.zeros(2 * cap, k, dtype=torch.uint8, device=DEV)
    w = torch.zeros(2, n, k, dtype=torch.uint8, device=DEV)
    if side == "weights":
        x[:, 5], w[:, :, 5] = one, codes
        want = codes.view(F8).float().expand(2 * cap, n)
    else:
        x[:, 5] = codes.repeat(3)[:2 * cap]
        w[:, :, 5] = one
        want = x[:, 5].view(F8).float()[:, None].expand(2 * cap, n)
    out = torch.zeros(2 * cap, n, dtype=BF16, device=DEV)
    ll.ll_moe_expert_gemm(cap, n, k, 2, ll.FP8_E4M3, ll.ACT_NONE, ll.BF16, x.view(F8), torch.ones(2 * cap, 1, device=DEV),
                          w.view(F8), torch.ones(2, 2, 1, device=DEV),
                          torch.tensor(counts, dtype=torch.int32, device=DEV), out)
    torch.cuda.synchronize()
    for rows in (slice(0, 300), slice(cap, cap + 60)):
        got, ref = out[rows].float(), want[rows]
        nan = torch.isnan(ref)
        assert torch.equal(torch.isnan(got), nan) and torch.equal(got[~nan], ref[~nan])
    assert not out[cap + 60:].any()


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("gated", [False, True])
def test_zero_points_of_all_eight_bits(group, gated):
    """Zero points are bytes: codes lie up to 255 below them. Few rows and
    tiles, against 64 bits."""
    say("case", group, gated)
    g = Gemm("w4", [300, 60, 1], 300, 136, 3 * 128, gated=gated, group=group, zeros=True, seed=group)
    gen = torch.Generator(device=DEV).manual_seed(1)
    g.w_zeros = torch.randint(0, 256, g.w_zeros.shape, generator=gen, device=DEV, dtype=torch.uint8)
    g.run().check()
