"""mhc_layer_norm_backward on rows of odd widths at either end of each kernel's range, in enough number for the
kernels that bring such rows into shared memory."""
import pytest

from _canary import guarded_empty, guards_intact
from _sublayer import check, ln_bwd64, ln_bwd_tol
from test_layer_norm_gpu import _bwd, _case, _dev, _fwd

torch = pytest.importorskip("torch")
mhc = pytest.importorskip("mhc_hyper_connections_b200")

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("T,d,dt", [(2369, 2553, BF), (2371, 2561, BF), (2373, 3833, BF), (2375, 3841, BF), (2377, 5113, BF),
                                    (2379, 5119, BF), (2399, 5121, BF), (2371, 2041, F32), (2373, 2045, F32),
                                    (2375, 2051, F32), (2377, 2553, F32), (2379, 2555, F32), (4001, 2305, F32)])
def test_gradients(T, d, dt):
    x, w, b, dy = _case(T, d, dt, 51)
    _, mean, rstd = _fwd(x, w, b)
    m, r = mean.cpu(), rstd.cpu()
    got = _bwd(x, w, m, r, dy)
    for g, ref, tol, what in zip(got, ln_bwd64(x, w, m, r, dy), ln_bwd_tol(x, w, m, r, dy, dt),
                                 ("dx", "dweight", "dbias")):
        check(g, ref, tol, what)
    for k in range(3):
        assert torch.equal(_bwd(x, w, m, r, dy, tuple(j == k for j in range(3)))[k], got[k])
    x, w, dy = _dev(x, w, dy)
    bufs, o = zip(*[guarded_empty(s, t, "cuda") for s, t in (
        ((T, d), dt), ((d,), F32), ((d,), F32), ((mhc.mhc_layer_norm_backward_workspace_bytes(T, d),), torch.uint8))])
    mhc.mhc_layer_norm_backward(x, w, mean, rstd, dy, *o)
    torch.cuda.synchronize()
    assert all(guards_intact(g) for g in bufs)
    assert all(torch.equal(p, q) for p, q in zip(o, got))
    assert mhc.mhc_device_status() == 0
