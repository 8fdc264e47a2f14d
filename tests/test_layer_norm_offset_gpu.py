"""mhc_layer_norm on rows whose values lie close together and far from zero, constant rows among them, in
every kernel that takes a row."""
import pytest

from _sublayer import U, check, half, ln64, row_adds

torch = pytest.importorskip("torch")
mhc = pytest.importorskip("mhc_hyper_connections_b200")

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32

# few and many rows; by lanes, warp and block, odd widths, rows longer than the registers of a block
SHAPES = [(3, 1), (10, 1000), (10, 1037), (3, 9000), (3, 9001), (3000, 40), (3000, 104), (3000, 250), (3000, 257),
          (3000, 504), (3000, 1000), (3000, 1537), (700, 2560), (2400, 2563), (700, 4088), (700, 5000), (2400, 5003),
          (700, 7000), (700, 9000), (200, 20000)]


def _fwd(x, w, b, eps):
    T = x.shape[0]
    y, mean, rstd = torch.empty_like(x), torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    mhc.mhc_layer_norm(x, w, b, eps, y, mean, rstd)
    return y, mean, rstd


@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("T,d", SHAPES)
def test_a_row_of_one_value_is_the_bias(T, d, dt):
    b = torch.randn(d, generator=torch.Generator().manual_seed(d)).cuda()
    w = torch.full((d,), 3.0, device="cuda")
    v = torch.tensor([100.0, 0.1, 12345.678, -3e4, 1.0, -7e-5, 1e15, 0.0, 3e-39]).to(dt)
    x = v[torch.arange(T) % len(v)][:, None].expand(T, d).contiguous().cuda()
    for eps in (1e-5, 1e-12):
        y, mean, rstd = _fwd(x, w, b, eps)
        assert torch.equal(y, b.to(dt).expand(T, d))
        # the mean of equal values, to the last place
        assert torch.equal(mean, x[:, 0].float())
        # one root and one division of fp32's eps: 2 u each at most
        want = torch.full((T,), float(torch.tensor(eps, dtype=F32)), dtype=torch.float64).rsqrt()
        check(rstd, want, 4 * U * want, "rstd")


@pytest.mark.parametrize("T,d", SHAPES[1:])
@pytest.mark.parametrize("offset", [300.0, -2e4, 1e6])
def test_rows_far_from_zero(T, d, offset):
    g = torch.Generator().manual_seed(T + d)
    x = torch.randn(T, d, generator=g) + offset
    w, b = 1 + 0.2 * torch.randn(d, generator=g), 0.3 * torch.randn(d, generator=g)
    eps = 1e-5
    y, mean, rstd = _fwd(x.cuda(), w.cuda(), b.cuda(), eps)
    ry, rm, rr, xh = ln64(x, w, b, eps)
    xd = x.double()
    c = (row_adds(d) + 4) * U
    # the mean: the rounding of its last sum, and the errors of the sum of x - mean, whose terms are the row's
    # deviations and the first mean's error e0 in each
    e0 = c * xd.abs().mean(1)
    dev = (xd - rm[:, None]).abs().mean(1) + e0
    m = U * rm.abs() + c * dev + U * e0
    check(mean, rm, m, "mean")
    # the variance: relative errors of its sum's terms and additions, and of the e0^2 taken off again
    rv = c + 3 * U + 2 * c * (e0 * rr) ** 2 + 2 * (c + 3 * U) * e0 * dev * rr ** 2
    r = rr * (0.5 * rv + 3 * U)
    check(rstd, rr, r, "rstd")
    wa = w.double().abs()
    ty = half(F32) * ry.abs() + wa * (rr * m)[:, None] + wa * xh.abs() * ((r / rr)[:, None] + 4 * U) \
        + 2 * U * b.double().abs()
    check(y, ry, ty, "y")


@pytest.mark.parametrize("T,d", [(9, 1024), (9, 1000), (3000, 257), (700, 2560), (700, 5000), (3, 9001)])
def test_infinite_nan_and_huge_rows(T, d):
    x = torch.randn(T, d, generator=torch.Generator().manual_seed(1))
    y0 = _fwd(x.cuda(), None, None, 1e-5)[0]
    x[0, 3], x[1, d - 1], x[2, 0] = float("inf"), float("nan"), float("-inf")
    keep = torch.arange(T) > 2
    y, mean, rstd = _fwd(x.cuda(), None, None, 1e-5)
    assert torch.equal(y[keep], y0[keep])
    assert not torch.isfinite(y[:3]).any() and not torch.isfinite(mean[:3]).any() and torch.isnan(rstd[:3]).all()
    # a variance beyond fp32 is infinite: rstd is 0, and so is every y
    y, _, rstd = _fwd((x[3:] * 1e30).cuda(), None, None, 1e-5)
    assert not rstd.any() and not y.any()
