"""Every form of the expert products and of the norm on the GPU, against plain
64-bit forms (tests/_experts.py). Which form a call takes goes by its sizes and
counts; the rule is repeated here, and each case asserts that it takes the form
it is there for, so that a changed limit cannot move it silently."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - collected on CPU machines too
    pytest.skip("no GPU", allow_module_level=True)

import _experts as X  # noqa: E402
from _gpu import DEV, say  # noqa: E402
from test_gpu_experts import IDS, KINDS, Gemm, _norm  # noqa: E402

FEW, TILE = 64, 256  # rows of the few-rows kernel's and of the tile kernel's tiles
MIB = 1 << 20


def _strip_cost(kind, rows):
    if kind == "bf16":
        return 8 if rows <= 32 else 9
    if kind == "fp8":
        return 8 if rows <= 16 else 9 if rows <= 32 else 10
    return 8 if rows <= 16 else 10 if rows <= 32 else 16


def _forms(g: Gemm):
    """(tiles, long list, strips a workgroup, weights past the caches)."""
    bits = {"bf16": 16, "fp8": 8, "w4": 4}[g.kind]
    weights = g.e * g.rw * g.k * bits // 8
    most = 1 << 30 if g.cap <= FEW or (g.cap <= 2 * FEW and weights < 256 * MIB) else FEW
    places = tiles = 0
    for c in g.rows_of:
        few = c if c <= most else c % TILE if c % TILE <= FEW else 0
        tiles += 0 if c <= most else c // TILE + (c % TILE > FEW)
        places += few // FEW * _strip_cost(g.kind, FEW) + (_strip_cost(g.kind, few % FEW) if few % FEW else 0)
    units = g.n // 128 if g.out_fp8 else -(-g.n // 16)
    strips = 2 if g.gated else 4
    share = places * units // 512
    return tiles > 0, g.out_fp8 or share >= 8 * 4 * strips, share / 8, weights >= 64 * MIB


CYCLE = [0, 1, 16, 17, 32, 33, 63, 64]
# k with which 96 experts of 2048 weight rows have 64 MiB, and with which not
LONG_K = {"bf16": (200, 72), "fp8": (384, 256), "w4": (1024, 384)}


@pytest.mark.parametrize("stream", [True, False])
@pytest.mark.parametrize("c", KINDS, ids=IDS)
def test_long_lists(c, stream):
    """Wavefronts beside each other over all of k, sharing A; runs that cross
    strips, row counts and experts."""
    say("case", c, "stream", stream)
    counts = [CYCLE[i * 5 % 8] for i in range(96)]
    n = 1024 if c.get("out_fp8") else 1040 if c["kind"] == "fp8" else 1032
    n *= 1 if c.get("gated") else 2
    k = LONG_K[c["kind"]][0 if stream else 1]
    g = Gemm(counts=counts, cap=64, n=n, k=k, seed=21, **c)
    tiles, long, _, past = _forms(g)
    assert (tiles, long, past) == (False, True, stream)
    g.run().check()


@pytest.mark.parametrize("stream", [True, False])
@pytest.mark.parametrize("c", [c for c in KINDS if not c.get("out_fp8")],
                         ids=[i for i, c in zip(IDS, KINDS) if not c.get("out_fp8")])
def test_short_lists_of_several_strips(c, stream):
    """k split over the wavefronts, with whole sets of strips and remainders,
    across experts."""
    say("case", c, "stream", stream)
    counts = [CYCLE[i * 3 % 8] for i in range(24)]
    n = 1040 if c.get("gated") else 2064
    k = {"bf16": (800, 136), "fp8": (1408, 384), "w4": (2816, 640)}[c["kind"]][0 if stream else 1]
    g = Gemm(counts=counts, cap=64, n=n, k=k, seed=22, **c)
    tiles, long, strips, past = _forms(g)
    assert (tiles, long, past) == (False, False, stream) and strips >= (2 if g.gated else 4)
    g.run().check()


COUNTS = [330, 65, 255, 257, 321, 0, 7, 64, 256]
TILE_SIZES = [("bf16", 24, 72, 128), ("bf16", 1000, 1000, 128), ("bf16", 136, 2056, 128), ("bf16", 520, 8, 128),
              ("fp8", 16, 128, 128), ("fp8", 48, 256, 128), ("fp8", 144, 384, 128), ("fp8", 208, 128, 128),
              ("fp8", 1040, 640, 128),
              ("w4", 24, 96, 32), ("w4", 200, 2016, 32), ("w4", 1000, 32, 32), ("w4", 136, 1088, 64),
              ("w4", 72, 2112, 64), ("w4", 120, 4736, 128), ("w4", 264, 128, 128)]


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("kind,n,k,group", TILE_SIZES)
def test_tiles_of_odd_sizes(kind, n, k, group, gated):
    """Tails of k, of columns and of rows, halves that lie in two weight
    blocks, a last group in half a step, more groups than the ring holds."""
    say("case", kind, n, k, group, gated)
    g = Gemm(kind, COUNTS, 330, n, k, gated=gated, group=group, zeros=n % 16 == 8, seed=n + k)
    assert _forms(g)[0]
    g.run().check()


@pytest.mark.parametrize("n,k", [(128, 256), (384, 128), (1024, 896)])
def test_tiles_with_fp8_out(n, k):
    say("case", n, k)
    g = Gemm("fp8", COUNTS, 330, n, k, gated=True, out_fp8=True, seed=n + k)
    assert _forms(g)[0]
    g.run().check()


@pytest.mark.parametrize("c", KINDS, ids=IDS)
def test_tile_rows_with_nan_and_infinity_stay_apart(c):
    """Rows in a whole tile, in the rows behind it, in a tile of its own: all
    others are what they are without them, bit for bit."""
    say("case", c)
    cap = 330
    g = Gemm(counts=[300, 3, 90], cap=cap, n=128, k=384, seed=5, **c)
    assert _forms(g)[0]
    g.run()
    want = g.out.view(torch.uint8).clone()
    bad_rows = [4, 131, 299, cap + 1, 2 * cap + 77]
    for i, r in enumerate(bad_rows):
        if g.kind == "fp8":
            g.a.view(torch.uint8)[r, 70 * i] = 0x7F
        else:
            g.a[r, 70 * i] = float("nan") if i % 2 else float("inf")
    g.clear()
    g.run()
    torch.cuda.synchronize()
    keep = torch.ones(len(want), dtype=torch.bool, device=DEV)
    keep[bad_rows] = False
    assert torch.equal(g.out.view(torch.uint8)[keep], want[keep])
    if not g.out_fp8:
        assert not torch.isfinite(g.out[bad_rows].float()).any()


@pytest.mark.parametrize("c", KINDS, ids=IDS)
def test_tiles_zero_rows_and_repeats(c):
    say("case", c)
    g = Gemm(counts=[3, 290, 330], cap=330, n=256, k=384, **c)
    assert _forms(g)[0]
    zero = [1, 330 + 17, 330 + 289, 660 + 300]
    g.a.view(torch.uint8)[zero] = 0
    g.run().check()
    assert not g.out[zero].float().any()
    first = g.out.view(torch.uint8).clone()
    for _ in range(3):
        g.clear()
        g.run()
        torch.cuda.synchronize()
        assert torch.equal(g.out.view(torch.uint8), first)


@pytest.mark.parametrize("c", KINDS, ids=IDS)
def test_tiles_captured_and_replayed(c):
    """A replay reads its own counts: rows move between the two kernels."""
    say("case", c)
    cap = 330
    g = Gemm(counts=[cap] * 3, cap=cap, n=128, k=256, **c)
    g.run()
    torch.cuda.synchronize()
    graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=s):
        g.run()
    for counts in ([3, 0, 330], [0, 0, 0], [256, 64, 65], [320, 321, 1], [330, 257, 255]):
        g.clear()
        g.counts.copy_(torch.tensor(counts, dtype=torch.int32))
        g.rows_of = counts
        g.fill = torch.zeros_like(g.fill)
        for i, n in enumerate(counts):
            g.fill[cap * i:cap * i + n] = True
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        g.check()


# Rows of more tokens than kFewTokens (256): 256 threads of two and four chunks
# of 8 columns, the last of them partial, and 512 and 1024 threads.
@pytest.mark.parametrize("t,h", [(257, 2056), (300, 4096), (257, 4104), (300, 7168), (257, 8192), (300, 8200),
                                 (257, 16392)])
@pytest.mark.parametrize("x_fp32", [False, True])
@pytest.mark.parametrize("residual", [False, True])
def test_norm_of_many_rows(t, h, x_fp32, residual):
    say("case", t, h, x_fp32, residual)
    x, res, w, new, out, _ = _norm(t, h, x_fp32, residual, False, seed=h)
    hh, dh, y, dy = X.rms_norm(x, res, w, 1e-6)
    X.check_bf16(out, y, dy, "out")
    if residual:
        X.check_bf16(new, hh, dh, "residual")


@pytest.mark.parametrize("t,h", [(257, 2176), (300, 4096), (257, 4224), (300, 7168), (257, 8192), (300, 8320)])
@pytest.mark.parametrize("x_fp32", [False, True])
def test_norm_of_many_rows_fp8(t, h, x_fp32):
    say("case", t, h, x_fp32)
    x, res, w, new, out, scales = _norm(t, h, x_fp32, True, True, seed=h)
    hh, dh, y, dy = X.rms_norm(x, res, w, 1e-6)
    X.check_fp8(out, scales, y, dy, "out")
    X.check_bf16(new, hh, dh, "residual")
