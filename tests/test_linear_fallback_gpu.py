"""fp32 backward products with values that have no bf16 parts: every finite element of all three gradients is
right, whichever operand holds the others, with and without an activation, and each gradient asked for alone."""
import pytest

from _sublayer import U, slope64, sum_tol
from test_linear_gpu import _bwd, _case

torch = pytest.importorskip("torch")
mhc = pytest.importorskip("mhc_hyper_connections_b200")

pytestmark = pytest.mark.gpu
F32 = torch.float32


def _plant(t):
    t[3, 5] = float("inf")
    t[7, t.shape[1] - 1] = -float("inf")
    t[11, 0] = float("nan")
    t[13, 64] = 3.4e38


def _check(got, ref, tol, what):
    got, r32 = got.cpu().double(), ref.float().double()        # past fp32's range: infinite
    assert torch.equal(torch.isnan(got), torch.isnan(r32)), what
    inf = torch.isinf(r32)
    assert torch.equal(got[inf], r32[inf]), what
    fin = torch.isfinite(r32)
    assert fin.double().mean() > 0.9, what
    err = (got - ref).abs()
    assert (err <= U * ref.abs() + tol)[fin].all(), what


# multiples of the tiles and not; dW's tiles shared along K; odd widths
@pytest.mark.parametrize("T,K,N", [(600, 2048, 1030), (512, 1024, 512), (301, 1031, 777)])
@pytest.mark.parametrize("act", ["none", "gelu"])
@pytest.mark.parametrize("which", ["x", "W", "dy", "z"])
def test_finite_elements_of_the_gradients(which, act, T, K, N):
    if which == "z" and act == "none":
        return
    c = _case(T, K, N, F32, 31)
    z = torch.randn(T, N, generator=torch.Generator().manual_seed(32))
    if which == "z":
        z[11, 0] = float("nan")
    else:
        _plant(c[which])
    x, W, dy = (c[k].double() for k in ("x", "W", "dy"))
    dz = dy if act == "none" else dy * slope64(z.double(), act)
    dz = torch.where(torch.isinf(dz.float()), dz.float().double(), dz)    # dz is an fp32 number: infinite past its range
    e = torch.zeros_like(dz) if act == "none" else 32 * U * dy.abs()      # dz's own error
    zc = None if act == "none" else z
    got = _bwd(c, zc, act)
    clean = lambda t: torch.nan_to_num(t, 0.0, 0.0, 0.0)                  # bounds of elements that no such value meets
    a, ea, xa, Wa = (clean(t.abs()) for t in (dz, e, x, W))
    _check(got[0], dz @ W, ea @ Wa + sum_tol(N) * (a @ Wa), "dx")
    _check(got[1], dz.T @ x, ea.T @ xa + sum_tol(T) * (a.T @ xa), "dW")
    _check(got[2], dz.sum(0), ea.sum(0) + (T + 80) * U * a.sum(0), "dbias")
    for k in range(3):
        alone = _bwd(c, zc, act, tuple(j == k for j in range(3)))[k]
        assert torch.equal(torch.nan_to_num(alone, 7.0), torch.nan_to_num(got[k], 7.0))
