"""mhc_layer_norm and mhc_layer_norm_backward on rows beyond 8192 columns, several of them per block: column sums
that a block carries from row to row, batches after a ring's first, and every way of asking for the gradients."""
import pytest

from _canary import guarded_empty, guards_intact
from _sublayer import check, ln64, ln_bwd64, ln_bwd_tol, ln_tol
from test_layer_norm_gpu import EPS, _bwd, _case, _dev, _fwd

torch = pytest.importorskip("torch")
mhc = pytest.importorskip("mhc_hyper_connections_b200")

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("T,d", [(700, 8200), (700, 12288), (700, 16384), (600, 16392), (700, 8209), (513, 20001), (520, 12290)])
def test_forward_and_backward(T, d, dt):
    x, w, b, dy = _case(T, d, dt, 41)
    y, mean, rstd = _fwd(x, w, b)
    for got, ref, tol, what in zip((y, mean, rstd), ln64(x, w, b, EPS)[:3], ln_tol(x, w, b, EPS, dt),
                                   ("y", "mean", "rstd")):
        check(got, ref, tol, what)
    m, r = mean.cpu(), rstd.cpu()
    got = _bwd(x, w, m, r, dy)
    for g, ref, tol, what in zip(got, ln_bwd64(x, w, m, r, dy), ln_bwd_tol(x, w, m, r, dy, dt),
                                 ("dx", "dweight", "dbias")):
        check(g, ref, tol, what)
    for k in range(3):
        assert torch.equal(_bwd(x, w, m, r, dy, tuple(j == k for j in range(3)))[k], got[k])
    assert mhc.mhc_device_status() == 0


@pytest.mark.parametrize("T,d,dt", [(700, 8200, BF), (600, 16384, BF), (520, 12288, F32), (513, 9001, BF), (513, 9001, F32)])
def test_writes_stay_inside_the_outputs(T, d, dt):
    x, w, b, dy = _dev(*_case(T, d, dt, 42))
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
