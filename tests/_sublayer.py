"""Oracles and tolerances of the sub-layer operator tests: plain 64-bit torch on the CPU.

Tolerances are bounds from the arithmetic, for fp32 computation and one rounding of the output:
  * u = 2^-24 is half a step of fp32, h(dt) half a step of the storage type (bf16 2^-8, fp32 u);
  * a sum of terms in fp32 of which one goes through at most c additions is off by at most
    c u sum|terms| (first order).
"""
import math

import torch

U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: U}
ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")
GELU_C = math.sqrt(2.0 / math.pi)


def half(dt):
    return HALF[dt]


def act64(z, name):
    if name == "none":
        return z
    if name == "relu":
        return z.clamp(min=0)
    if name == "gelu":
        return 0.5 * z * torch.special.erfc(-z / math.sqrt(2.0))
    if name == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(GELU_C * (z + 0.044715 * z ** 3)))
    return z * torch.sigmoid(z)


def slope64(z, name):
    if name == "none":
        return torch.ones_like(z)
    if name == "relu":
        return (z > 0).to(z.dtype)
    if name == "gelu":
        return 0.5 * torch.special.erfc(-z / math.sqrt(2.0)) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":
        t = torch.tanh(GELU_C * (z + 0.044715 * z ** 3))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * GELU_C * (1 + 3 * 0.044715 * z * z)
    s = torch.sigmoid(z)
    return s * (1 + z * (1 - s))


def ln64(x, w, b, eps):
    """(y, mean, rstd, xh) of x [T, d] in 64 bits."""
    x = x.double()
    mean = x.mean(1)
    var = ((x - mean[:, None]) ** 2).mean(1)
    rstd = 1.0 / torch.sqrt(var + eps)
    xh = (x - mean[:, None]) * rstd[:, None]
    y = xh if w is None else xh * w.double()
    if b is not None:
        y = y + b.double()
    return y, mean, rstd, xh


def row_adds(d):
    """Additions one term of a row sum goes through: at most 32 in its thread (d / 1024 in the
    kernel of long rows), 5 between lanes and 32 between warps."""
    return 32 + d / 1024 + 5 + 32


def ln_tol(x, w, b, eps, dt):
    """Bounds on the errors of (y, mean, rstd)."""
    y, mean, rstd, xh = ln64(x, w, b, eps)
    xd = x.double()
    c = (row_adds(x.shape[1]) + 4) * U
    wa = torch.ones(x.shape[1], dtype=torch.float64) if w is None else w.double().abs()
    ba = torch.zeros_like(wa) if b is None else b.double().abs()
    m = c * xd.abs().mean(1)                      # the mean's error
    # rstd: half the relative error of the variance, whose terms (x - mean)^2 carry 2 u each and the
    # square of the mean's error, and 3 u of its own division and root
    r = rstd * (0.5 * (c + 2 * U) + 3 * U) + 0.5 * rstd ** 3 * m ** 2
    ty = half(dt) * y.abs() + wa * (rstd * m)[:, None] + wa * xh.abs() * ((r / rstd)[:, None] + 4 * U) + 2 * U * ba
    return ty, m + U * mean.abs(), r


def ln_bwd64(x, w, mean, rstd, dy):
    xd, g0 = x.double(), dy.double()
    xh = (xd - mean.double()[:, None]) * rstd.double()[:, None]
    g = g0 if w is None else g0 * w.double()
    a, k = g.mean(1, keepdim=True), (g * xh).mean(1, keepdim=True)
    dx = rstd.double()[:, None] * (g - a - xh * k)
    return dx, (g0 * xh).sum(0), g0.sum(0)


def ln_bwd_tol(x, w, mean, rstd, dy, dt):
    """Bounds on the errors of (dx, dweight, dbias).  xh carries the rounding of x - mean and of its
    product with rstd (2 u |xh|)."""
    xd, g0, rs = x.double(), dy.double(), rstd.double()[:, None]
    T, d = x.shape
    xh = (xd - mean.double()[:, None]) * rs
    g = g0 if w is None else g0 * w.double()
    c = (row_adds(d) + 4) * U
    a, k = g.abs().mean(1, keepdim=True), (g * xh).abs().mean(1, keepdim=True)
    dx = ln_bwd64(x, w, mean, rstd, dy)[0]
    tdx = half(dt) * dx.abs() + rs * (c * (a + xh.abs() * k) + 6 * U * (g.abs() + a + xh.abs() * k))
    # a column term is added to its block's running sum (T / blocks rows, at most T), then to the
    # other warps' (8) and the other blocks' (8 chains of 56)
    n = (T + 8 + 64 + 4) * U
    return tdx, n * (g0 * xh).abs().sum(0), n * g0.abs().sum(0)


def sum_tol(K):
    """Relative bound, against sum|terms|, on an fp32 sum of K products.  The worst case K u is far
    from what roundings of either sign do; the bound that holds with a probability of 1 - 2 exp(-l^2 / 2)
    per output is l sqrt(K) u.  l = 8 (1e-13), and one bit per addition for an accumulator that
    truncates: its errors have one sign, at most 2 u each, over the K / 16 steps of a tensor-core sum."""
    return (8 * math.sqrt(K) + 16) * U + (K / 16) * 2 * U


def check(got, ref, tol, what):
    g = got.detach().cpu().double()
    assert g.shape == ref.shape, what
    assert torch.isfinite(g).all(), what
    err = (g - ref).abs()
    bad = err > tol
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} beyond the bound, worst "
                           f"{float((err / tol.clamp(min=1e-300)).max()):.2f} times it")
