"""The sub-layer operators reject bad arguments on the host: status codes of the C ABI (addresses
that are never dereferenced, every call refused before the library touches CUDA) and the binding's
checks on CPU tensors, which refuse a wrong shape by name before they ask for a CUDA tensor."""
import pytest

import mhc_hyper_connections_b200 as mhc
from mhc_hyper_connections_b200 import build as mbuild

torch = pytest.importorskip("torch")

A = 0x10000000
P = [A + i * 0x10000000 for i in range(12)]          # one region per argument
F32, BF16 = 0, 1


@pytest.fixture(scope="module")
def lib():
    mbuild.build()
    return mhc.load_library()


def test_layer_norm_validation(lib):
    def ln(x=P[0], w=P[1], b=P[2], T=4, d=64, dt=BF16, y=P[3], mean=P[4], rstd=P[5]):
        return lib.mhc_layer_norm(x, w, b, T, d, 1e-5, dt, y, mean, rstd, None)
    assert ln(T=0) == 0 and ln(T=0, x=0, y=0) == 0
    assert ln(d=0) == 2 and ln(T=-1) == 2 and ln(d=(1 << 30) + 1) == 2
    assert ln(T=1 << 60) == 2                        # byte counts would overflow
    assert ln(dt=2) == 4 and ln(dt=-1) == 4
    assert ln(x=0) == 1 and ln(y=0) == 1
    assert ln(mean=0) == 1 and ln(rstd=0) == 1       # both or neither
    assert ln(x=P[0] + 1) == 3 and ln(dt=F32, y=P[3] + 2) == 3
    assert ln(w=P[1] + 2) == 3 and ln(b=P[2] + 1) == 3 and ln(mean=P[4] + 2) == 3
    assert ln(y=P[0]) == 7 and ln(y=P[0] + 256) == 7
    assert ln(mean=P[5] + 8) == 7 and ln(rstd=P[1]) == 7 and ln(y=P[2] - 128) == 7


def test_layer_norm_backward_validation(lib):
    need = lib.mhc_layer_norm_backward_workspace_bytes(4, 64)
    assert need > 0
    assert lib.mhc_layer_norm_backward_workspace_bytes(0, 64) == 0
    assert lib.mhc_layer_norm_backward_workspace_bytes(4, 0) == 0
    assert lib.mhc_layer_norm_backward_workspace_bytes(-4, 8) == 0

    def lnb(x=P[0], w=P[1], mean=P[2], rstd=P[3], T=4, d=64, dt=BF16, dy=P[4], dx=P[5], dw=P[6], db=P[7], ws=P[8],
            wsb=need):
        return lib.mhc_layer_norm_backward(x, w, mean, rstd, T, d, dt, dy, dx, dw, db, ws, wsb, None)
    assert lnb(d=0) == 2 and lnb(T=-1) == 2 and lnb(dt=9) == 4
    for k in ("x", "mean", "rstd", "dy", "ws"):
        assert lnb(**{k: 0}) == 1, k
    assert lnb(x=P[0] + 1) == 3 and lnb(dx=P[5] + 1) == 3 and lnb(ws=P[8] + 16) == 3 and lnb(dw=P[6] + 2) == 3
    assert lnb(wsb=need - 1) == 8
    assert lnb(dx=P[0]) == 7 and lnb(dx=P[4] + 64) == 7 and lnb(dw=P[7]) == 7 and lnb(ws=P[4]) == 7
    assert lnb(db=P[3]) == 7
    assert lnb(dx=0, dw=0, db=0, ws=0, wsb=0) == 0   # nothing wanted: nothing launched
    assert lnb(T=0, dw=P[6] + 2) == 3 and lnb(T=0, dw=P[7] + 4) == 7


def test_linear_validation(lib):
    def lin(x=P[0], W=P[1], b=P[2], r=P[3], T=4, K=64, N=32, act=1, dt=BF16, y=P[4], z=P[5], ws=P[6], wsb=None):
        need = lib.mhc_linear_workspace_bytes(T, K, N, dt)
        return lib.mhc_linear(x, W, b, r, T, K, N, act, dt, y, z, ws, need if wsb is None else wsb, None)
    assert lin(T=0) == 0 and lin(T=0, x=0, W=0, y=0, ws=0) == 0
    assert lin(K=0) == 2 and lin(N=0) == 2 and lin(T=-1) == 2 and lin(K=(1 << 30) + 1) == 2 and lin(T=1 << 59) == 2
    assert lin(dt=2) == 4
    assert lin(act=-1) == 5 and lin(act=5) == 5
    assert lin(x=0) == 1 and lin(W=0) == 1 and lin(y=0) == 1
    assert lin(x=P[0] + 1) == 3 and lin(z=P[5] + 1) == 3 and lin(dt=F32, r=P[3] + 2) == 3 and lin(b=P[2] + 2) == 3
    assert lin(y=P[0]) == 7 and lin(y=P[1] + 64) == 7 and lin(y=P[3]) == 7 and lin(z=P[4]) == 7 and lin(z=P[2]) == 7
    assert lib.mhc_linear_workspace_bytes(0, 64, 64, BF16) == 0
    assert lib.mhc_linear_workspace_bytes(4, 0, 64, BF16) == 0 and lib.mhc_linear_workspace_bytes(4, 64, 64, 7) == 0


def test_linear_backward_validation(lib):
    need = lib.mhc_linear_backward_workspace_bytes(4, 64, 32, BF16)
    assert need > 0
    assert lib.mhc_linear_backward_workspace_bytes(0, 64, 32, BF16) == 0
    assert lib.mhc_linear_backward_workspace_bytes(4, 64, 0, BF16) == 0
    assert lib.mhc_linear_backward_workspace_bytes(4, 64, 32, 3) == 0

    def linb(x=P[0], W=P[1], z=P[2], T=4, K=64, N=32, act=2, dt=BF16, dy=P[3], dx=P[4], dW=P[5], db=P[6], ws=P[7],
             wsb=need):
        return lib.mhc_linear_backward(x, W, z, T, K, N, act, dt, dy, dx, dW, db, ws, wsb, None)
    assert linb(K=0) == 2 and linb(T=-1) == 2 and linb(dt=4) == 4 and linb(act=7) == 5
    for k in ("x", "W", "z", "dy", "ws"):
        assert linb(**{k: 0}) == 1, k
    assert linb(x=P[0] + 1) == 3 and linb(dW=P[5] + 1) == 3 and linb(db=P[6] + 2) == 3 and linb(ws=P[7] + 128) == 3
    assert linb(wsb=need - 1) == 8
    assert linb(dx=P[0]) == 7 and linb(dW=P[1]) == 7 and linb(dx=P[3]) == 7 and linb(db=P[5]) == 7
    assert linb(ws=P[2]) == 7 and linb(dW=P[4] + 32) == 7
    assert linb(T=0, dW=P[5] + 1) == 3 and linb(T=0, db=P[5]) == 7


def test_stop_hook_validation(lib):
    assert lib.mhc_debug_sublayer_stop_after(-1, 999) == 2
    assert lib.mhc_debug_sublayer_stop_after(3, 10_000_001) == 2
    assert lib.mhc_debug_sublayer_stop_after(-1, 1_000_000) == 0


# ---- the binding

def _t(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype)


f = lambda *s: _t(*s, dtype=torch.float32)
T, D, K, N = 6, 24, 16, 40


def _ln(**k):
    a = dict(x=_t(T, D), weight=f(D), bias=f(D), y=_t(T, D), mean=f(T), rstd=f(T))
    a.update(k)
    mhc.mhc_layer_norm(a["x"], a["weight"], a["bias"], 1e-5, a["y"], a["mean"], a["rstd"])


def _lnb(**k):
    a = dict(x=_t(T, D), weight=f(D), mean=f(T), rstd=f(T), dy=_t(T, D), dx=_t(T, D), dweight=f(D), dbias=f(D))
    a.update(k)
    mhc.mhc_layer_norm_backward(a["x"], a["weight"], a["mean"], a["rstd"], a["dy"], a["dx"], a["dweight"],
                                a["dbias"], _t(64, dtype=torch.uint8))


def _lin(**k):
    a = dict(x=_t(T, K), W=_t(N, K), bias=f(N), y=_t(T, N), residual=_t(T, N), z=_t(T, N))
    a.update(k)
    mhc.mhc_linear(a["x"], a["W"], a["bias"], a["y"], residual=a["residual"], z=a["z"])


def _linb(**k):
    a = dict(x=_t(T, K), W=_t(N, K), z=_t(T, N), dy=_t(T, N), dx=_t(T, K), dW=_t(N, K), dbias=f(N))
    a.update(k)
    mhc.mhc_linear_backward(a["x"], a["W"], a["z"], a["dy"], a["dx"], a["dW"], a["dbias"],
                            _t(64, dtype=torch.uint8), act=mhc.ACT_GELU)


@pytest.mark.parametrize("call", [_ln, _lnb, _lin, _linb])
def test_good_shapes_reach_the_device_check(call):
    with pytest.raises(ValueError, match="must be a CUDA tensor"):
        call()


@pytest.mark.parametrize("call,name,bad", [
    (_ln, "weight", f(D + 1)), (_ln, "bias", f(D, 1)), (_ln, "y", _t(T, D - 1)), (_ln, "mean", f(T + 1)),
    (_ln, "rstd", f(T, 1)),
    (_lnb, "weight", f(D - 1)), (_lnb, "mean", f(1)), (_lnb, "rstd", f(T - 1)), (_lnb, "dy", _t(T + 1, D)),
    (_lnb, "dx", _t(D, T)), (_lnb, "dweight", f(1)), (_lnb, "dbias", f(D + 8)),
    (_lin, "W", _t(N, K + 1)), (_lin, "bias", f(K)), (_lin, "y", _t(T, K)), (_lin, "residual", _t(1, N)),
    (_lin, "z", _t(T - 1, N)),
    (_linb, "W", _t(N, K - 1)), (_linb, "z", _t(N)), (_linb, "dy", _t(T, N + 1)), (_linb, "dx", _t(T, N)),
    (_linb, "dW", _t(K, N)), (_linb, "dbias", f(N - 1))])
def test_wrong_shapes_are_refused_by_name(call, name, bad):
    with pytest.raises(ValueError, match=f"{name} (has shape|must be two)"):
        call(**{name: bad})


@pytest.mark.parametrize("call", [_ln, _lnb, _lin, _linb])
def test_rows_are_two_dimensional_tensors(call):
    with pytest.raises(ValueError, match="x must be two-dimensional"):
        call(x=_t(2, 3, 8))
    with pytest.raises(TypeError, match="x must be a torch tensor"):
        call(x=None)


@pytest.mark.parametrize("call", [_ln, _lnb, _lin, _linb])
def test_other_storage_types_are_refused(call):
    with pytest.raises(TypeError, match="unsupported dtype"):
        call(x=_t(T, K if call in (_lin, _linb) else D, dtype=torch.float16))
    assert mhc.mhc_linear_workspace_bytes(4, 64, 64, torch.float32) >= 0
    with pytest.raises(TypeError, match="unsupported dtype"):
        mhc.mhc_linear_workspace_bytes(4, 64, 64, torch.float16)
