"""Plain 64-bit forms of the operators around the expert side, with bounds on
what a right 32-bit kernel may be off by.

Not collected by pytest (no test_ prefix). Torch only; shares no code with the
library.

Every form returns (value, bound) in float64. U = 2^-24 is half a step of
fp32. A sum of m fp32 products in any order is off by at most (m + 2) U times
the sum of the products' magnitudes (first order; one product rounding and at
most m additions, each of a partial sum that this sum bounds), and we count
m + 16 for the scalings around it.
"""
import torch

U = 2.0 ** -24
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float8_e4m3fn: 2.0 ** -4}
BLOCK = 128


def spread(scales, rows, cols, block=BLOCK):
    """A scale per block x block as one per element."""
    r = torch.arange(rows, device=scales.device) // block
    c = torch.arange(cols, device=scales.device) // block
    return scales.double()[r][:, c]


def along(scales, cols, block=BLOCK):
    """A scale per `block` columns as one per element."""
    return scales.double()[:, torch.arange(cols, device=scales.device) // block]


def unpack4(w):
    """Codes 0..15, the low half of a byte first, as float64."""
    out = torch.empty(*w.shape[:-1], 2 * w.shape[-1], dtype=torch.float64, device=w.device)
    out[..., 0::2] = (w & 15).double()
    out[..., 1::2] = (w >> 4).double()
    return out


def product(a, w):
    """P = A W^T and its bound; a [r, k], w [i, k] float64."""
    p = a @ w.t()
    return p, (a.shape[1] + 16) * U * (a.abs() @ w.abs().t())


def product_w4(a, codes, scale, zero, group):
    """The same from 4-bit codes: scale and zero [i, k / group] float64. The
    kernel sums (16 + code) A and (16 + zero) A apart, in fp32, so the bound
    counts the magnitudes of both."""
    k = a.shape[1]
    s, z = along(scale, k, group), along(zero, k, group)
    p = a @ (s * (codes - z)).t()
    return p, (k + 16) * U * (a.abs() @ (s.abs() * (32 + codes + z)).t())


def gated(p, dp, n):
    """silu(gate) * up: |silu'| < 1.1; exp by a base-2 power is off by some
    steps plus the rounding of its argument (|g| log2(e) U, twice), and the
    exponential's smallest values may be flushed to zero."""
    g, u = p[:, :n], p[:, n:]
    dg, du = dp[:, :n], dp[:, n:]
    s = g * torch.sigmoid(g)
    v = s * u
    dv = 1.1 * dg * (u.abs() + du) + s.abs() * du + v.abs() * (16 + 4 * g.abs()) * U + 1e-36 * (1 + u.abs())
    return v, dv


def check_bf16(got, v, dv, what=""):
    got = got.double()
    tol = dv + HALF_STEP[torch.bfloat16] * (v.abs() + dv) + 2.0 ** -133
    bad = ~((got - v).abs() <= tol)
    assert not bad.any(), (what, int(bad.sum()), got[bad][:4].tolist(), v[bad][:4].tolist(), tol[bad][:4].tolist())


def check_fp8(codes, scales, v, dv, what=""):
    """codes float8 [r, n], scales fp32 [r, n / 128] against v: a scale is
    the largest magnitude / 448, a code half a step (or half the smallest
    step, 2^-9) from v / scale."""
    r, n = v.shape
    vb, db = v.view(r, n // BLOCK, BLOCK), dv.view(r, n // BLOCK, BLOCK)
    amax = vb.abs().amax(-1)
    da = db.amax(-1)
    s = scales.double()
    bad = ~((s - amax / 448).abs() <= da / 448 + 4 * U * amax / 448 + 2.0 ** -149)
    assert not bad.any(), (what, "scales", int(bad.sum()), s[bad][:4].tolist(), (amax / 448)[bad][:4].tolist())
    zero = s == 0
    inv = torch.where(zero, torch.zeros_like(s), 1 / torch.where(zero, torch.ones_like(s), s))[..., None]
    q = vb * inv
    got = codes.double().view_as(vb)
    tol = db * inv + q.abs() * 8 * U
    tol = tol + torch.maximum(HALF_STEP[torch.float8_e4m3fn] * (q.abs() + tol), torch.full_like(q, 2.0 ** -10))
    bad = ~((got - q).abs() <= tol)
    assert not bad.any(), (what, "codes", int(bad.sum()), got[bad][:4].tolist(), q[bad][:4].tolist())


def rms_norm(x, residual, weight, eps):
    """(h, dh, y, dy): the new residual before its rounding, and the output."""
    h = x.double() + (residual.double() if residual is not None else 0)
    dh = U * h.abs()
    m = x.shape[1]
    y = h / ((h * h).mean(1, keepdim=True) + eps).sqrt() * weight.double()
    # mean of squares: (m + 4) U relative, half of it in the root; the row's
    # own rounding 3 U more, the products and the quotient 6 U
    return h, dh, y, y.abs() * ((m + 4) / 2 + 12) * U
