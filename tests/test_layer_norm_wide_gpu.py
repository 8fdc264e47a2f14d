"""mhc_layer_norm and mhc_layer_norm_backward on rows of 2049 to 8192 columns, aligned and odd, in enough
number for every kernel that takes such rows: bounds, repeatability, guard regions and non-finite rows."""
import pytest

from _canary import guarded_empty, guards_intact
from _sublayer import check, ln64, ln_bwd64, ln_bwd_tol, ln_tol
from test_layer_norm_gpu import EPS, _bwd, _case, _dev, _fwd

torch = pytest.importorskip("torch")
mhc = pytest.importorskip("mhc_hyper_connections_b200")

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32

SHAPES = [(301, 2056), (170, 3000), (300, 4104), (160, 5000), (449, 5128), (200, 7168), (170, 7176), (297, 8192),
          # odd widths: 16 rows per SM and more, the last row ending inside a word
          (2370, 4351), (2401, 4803), (2369, 6121), (2379, 8191), (2377, 4090)]


@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("T,d", SHAPES)
def test_forward_and_backward(T, d, dt):
    x, w, b, dy = _case(T, d, dt, 21)
    y, mean, rstd = _fwd(x, w, b)
    for got, ref, tol, what in zip((y, mean, rstd), ln64(x, w, b, EPS)[:3], ln_tol(x, w, b, EPS, dt),
                                   ("y", "mean", "rstd")):
        check(got, ref, tol, what)
    assert torch.equal(_fwd(x, w, b, stats=False)[0], y)
    m, r = mean.cpu(), rstd.cpu()
    got = _bwd(x, w, m, r, dy)
    for g, ref, tol, what in zip(got, ln_bwd64(x, w, m, r, dy), ln_bwd_tol(x, w, m, r, dy, dt),
                                 ("dx", "dweight", "dbias")):
        check(g, ref, tol, what)
    assert all(torch.equal(p, q) for p, q in zip(_bwd(x, w, m, r, dy), got))
    assert mhc.mhc_device_status() == 0


@pytest.mark.parametrize("T,d,dt", [(300, 5000, F32), (200, 7176, BF), (2379, 8191, BF), (2401, 4803, BF)])
def test_writes_stay_inside_the_outputs(T, d, dt):
    x, w, b, dy = _dev(*_case(T, d, dt, 22))
    y0, mean, rstd = _fwd(x, w, b)
    ref = _bwd(x, w, mean, rstd, dy)
    bufs, o = zip(*[guarded_empty(s, t, "cuda") for s, t in (
        ((T, d), dt), ((T,), F32), ((T,), F32), ((T, d), dt), ((d,), F32), ((d,), F32),
        ((mhc.mhc_layer_norm_backward_workspace_bytes(T, d),), torch.uint8))])
    mhc.mhc_layer_norm(x, w, b, EPS, *o[:3])
    mhc.mhc_layer_norm_backward(x, w, o[1], o[2], dy, *o[3:])
    torch.cuda.synchronize()
    assert all(guards_intact(g) for g in bufs)
    assert all(torch.equal(p, q) for p, q in zip(o, (y0, mean, rstd, *ref)))


@pytest.mark.parametrize("T,d,dt", [(2379, 8191, BF), (2401, 4803, BF), (200, 7176, BF), (300, 5000, F32)])
def test_non_finite_rows_stay_in_their_rows(T, d, dt):
    x, w, b, _ = _case(T, d, dt, 23)
    y0 = _fwd(x, w, b)[0]
    bad = [0, 7, T // 2, T - 1]
    x[bad[0], 0], x[bad[1], d - 1], x[bad[2], :], x[bad[3], d - 1] = float("nan"), float("inf"), float("-inf"), float("nan")
    y = _fwd(x, w, b)[0]
    keep = torch.ones(T, dtype=torch.bool)
    keep[bad] = False
    assert torch.equal(y[keep.cuda()], y0[keep.cuda()])
    assert torch.isnan(y[~keep.cuda()]).all(dim=1).all()
