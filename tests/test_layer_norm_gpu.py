"""mhc_layer_norm and mhc_layer_norm_backward against 64-bit oracles (bounds in _sublayer.py):
every layout of a row (warp, block, element-wise, longer than the registers of a block), odd
widths, one token, rows far from zero, unaligned buffers, missing parameters, streams, captured
graphs, guard regions and bitwise repeatability."""
import pytest

from _canary import guarded_empty, guards_intact
from _sublayer import check, ln64, ln_bwd64, ln_bwd_tol, ln_tol

torch = pytest.importorskip("torch")
mhc = pytest.importorskip("mhc_hyper_connections_b200")

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
EPS = 1e-5

SHAPES = [(1, 1), (1, 4096), (3, 2), (5, 7), (17, 8), (40, 64), (33, 250), (257, 256), (100, 257), (64, 512),
          (70, 520), (31, 1000), (700, 1024), (301, 1037), (149, 2560), (1200, 4096), (9, 4095), (150, 4104),
          # odd widths, many rows: rows at every offset within 16 bytes, and a last row that ends inside a word
          (2375, 257), (2403, 260), (2401, 1025), (2369, 1532), (2500, 2047), (2373, 2562), (2427, 2819), (2379, 4090),
          (2399, 4102), (2377, 201), (513, 1030), (512, 515),
          (3, 8192), (160, 8191), (5, 8200), (2, 16384), (3, 20001), (2, 40000)]


def _case(T, d, dt, seed=0, offset=0.0):
    g = torch.Generator().manual_seed(1000 * T + d + seed)
    x = (torch.randn(T, d, generator=g) + offset).to(dt)
    x[:, ::97] *= 8
    w = 1 + 0.2 * torch.randn(d, generator=g)
    b = 0.3 * torch.randn(d, generator=g)
    dy = torch.randn(T, d, generator=g).to(dt)
    return x, w, b, dy


def _dev(*ts):
    return [None if t is None else t.cuda() for t in ts]


def _fwd(x, w, b, stats=True):
    T = x.shape[0]
    x, w, b = _dev(x, w, b)
    y = torch.empty_like(x)
    mean, rstd = (torch.empty(T, device="cuda"), torch.empty(T, device="cuda")) if stats else (None, None)
    mhc.mhc_layer_norm(x, w, b, EPS, y, mean, rstd)
    return y, mean, rstd


def _bwd(x, w, mean, rstd, dy, want=(True, True, True)):
    T, d = x.shape
    x, w, mean, rstd, dy = _dev(x, w, mean, rstd, dy)
    dx = torch.empty_like(x) if want[0] else None
    dw = torch.empty(d, device="cuda") if want[1] else None
    db = torch.empty(d, device="cuda") if want[2] else None
    ws = torch.empty(mhc.mhc_layer_norm_backward_workspace_bytes(T, d), dtype=torch.uint8, device="cuda")
    mhc.mhc_layer_norm_backward(x, w, mean, rstd, dy, dx, dw, db, ws)
    return dx, dw, db


@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("T,d", SHAPES)
def test_forward_and_backward(T, d, dt):
    x, w, b, dy = _case(T, d, dt)
    y, mean, rstd = _fwd(x, w, b)
    ry, rm, rr, _ = ln64(x, w, b, EPS)
    ty, tm, tr = ln_tol(x, w, b, EPS, dt)
    check(y, ry, ty, "y")
    check(mean, rm, tm, "mean")
    check(rstd, rr, tr, "rstd")
    assert torch.equal(_fwd(x, w, b, stats=False)[0], y)
    m, r = mean.cpu(), rstd.cpu()
    got = _bwd(x, w, m, r, dy)
    for name, g, ref, tol in zip(("dx", "dweight", "dbias"), got, ln_bwd64(x, w, m, r, dy),
                                 ln_bwd_tol(x, w, m, r, dy, dt)):
        check(g, ref, tol, name)
    # bitwise repeatable, whichever gradients are asked for
    again = _bwd(x, w, m, r, dy)
    assert all(torch.equal(p, q) for p, q in zip(got, again))
    assert torch.equal(_bwd(x, w, m, r, dy, (True, False, False))[0], got[0])
    assert torch.equal(_bwd(x, w, m, r, dy, (False, True, False))[1], got[1])
    assert torch.equal(_bwd(x, w, m, r, dy, (False, False, True))[2], got[2])


@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("T,d", [(40, 96), (12, 1024), (200, 2560), (3, 33)])
def test_without_parameters(T, d, dt):
    x, _, _, dy = _case(T, d, dt, 1)
    y, mean, rstd = _fwd(x, None, None)
    check(y, ln64(x, None, None, EPS)[0], ln_tol(x, None, None, EPS, dt)[0], "y")
    m, r = mean.cpu(), rstd.cpu()
    for name, g, ref, tol in zip(("dx", "dweight", "dbias"), _bwd(x, None, m, r, dy),
                                 ln_bwd64(x, None, m, r, dy), ln_bwd_tol(x, None, m, r, dy, dt)):
        check(g, ref, tol, name)


def test_rows_far_from_zero_keep_their_variance():
    # fp32 rows around 300: E[x^2] - mean^2 would lose the variance's low bits, the walk around the
    # mean does not; the bound is the same formula
    for d in (64, 1024, 5000):
        x, w, b, _ = _case(20, d, F32, 2, offset=300.0)
        y, mean, rstd = _fwd(x, w, b)
        ry, rm, rr, _ = ln64(x, w, b, EPS)
        ty, tm, tr = ln_tol(x, w, b, EPS, F32)
        check(y, ry, ty, "y")
        check(rstd, rr, tr, "rstd")


def test_constant_rows_and_non_finite_rows():
    x, w, b, _ = _case(9, 1024, BF, 3)
    x[2] = 1.5                      # no variance: y is the bias
    x[4, 100] = float("inf")
    x[6, 7] = float("nan")
    y, mean, rstd = _fwd(x, w, b)
    assert torch.equal(y[2].cpu(), b.to(BF))
    assert abs(float(rstd[2]) - EPS ** -0.5) < 1e-3
    for t in (4, 6):
        assert not torch.isfinite(y[t]).any()
    keep = [0, 1, 3, 5, 7, 8]
    assert torch.equal(y[keep], _fwd(x[keep], w, b)[0])


@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("T,d", [(2400, 515), (2371, 1537), (600, 515), (300, 520)])
def test_non_finite_rows_stay_in_their_rows(T, d, dt):
    # rows that share a 16-byte word with their neighbours among them
    x, w, b, dy = _case(T, d, dt, 8)
    y0, mean, rstd = _fwd(x, w, b)
    dx0 = _bwd(x, w, mean, rstd, dy)[0]
    bad = [1, 8, T // 2, T - 1]
    for k, t in enumerate(bad):
        x[t, :: d - 1] = float("inf") if k % 2 else float("nan")      # the row's first and last element
        dy[t, :: d - 1] = float("nan")
    y1, mean1, rstd1 = _fwd(x, w, b)
    dx1 = _bwd(x, w, mean1, rstd1, dy)[0]
    keep = torch.ones(T, dtype=torch.bool)
    keep[bad] = False
    assert torch.equal(y1[keep], y0[keep]) and torch.equal(dx1[keep], dx0[keep])
    assert torch.equal(mean1[keep], mean[keep]) and torch.equal(rstd1[keep], rstd[keep])
    assert not torch.isfinite(y1[bad]).any() and not torch.isfinite(dx1[bad]).any()


@pytest.mark.parametrize("T,d", [(3, 4096), (140, 1024), (500, 2560), (512, 1037), (513, 1037)])
def test_backward_calls_in_a_row(T, d):
    # each call's dx is the next one's dy, into buffers used in turn: nothing may start before what it
    # reads is there, nor write what is still read
    x, w, b, dy = _dev(*_case(T, d, BF, 9))
    _, mean, rstd = _fwd(x, w, b)
    n = 24
    ws = torch.empty(mhc.mhc_layer_norm_backward_workspace_bytes(T, d), dtype=torch.uint8, device="cuda")
    res = []
    for apart in (True, False):
        g, h = dy.clone(), torch.empty_like(dy)
        dw, db = torch.empty(n, d, device="cuda"), torch.empty(n, d, device="cuda")
        torch.cuda.synchronize()
        for i in range(n):
            mhc.mhc_layer_norm_backward(x, w, mean, rstd, g, h, dw[i], db[i], ws)
            if apart:
                torch.cuda.synchronize()
            g, h = h, g
        res.append((g, dw, db))
    assert all(torch.equal(p, q) for p, q in zip(*res))


@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("T,d", [(7, 64), (50, 1000), (150, 4096), (3, 8000)])
def test_unaligned_buffers(T, d, dt):
    x, w, b, dy = _case(T, d, dt, 4)
    off = lambda t: torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")[1:].view(t.shape).copy_(t)
    X, W, B, DY = off(x), off(w), off(b), off(dy)
    Y, DX = off(x), off(x)
    mean, rstd = torch.empty(T + 1, device="cuda")[1:], torch.empty(T + 1, device="cuda")[1:]
    mhc.mhc_layer_norm(X, W, B, EPS, Y, mean, rstd)
    check(Y, ln64(x, w, b, EPS)[0], ln_tol(x, w, b, EPS, dt)[0], "y")
    dw, db = torch.empty(d + 1, device="cuda")[1:], torch.empty(d + 1, device="cuda")[1:]
    ws = torch.empty(mhc.mhc_layer_norm_backward_workspace_bytes(T, d), dtype=torch.uint8, device="cuda")
    mhc.mhc_layer_norm_backward(X, W, mean, rstd, DY, DX, dw, db, ws)
    m, r = mean.cpu(), rstd.cpu()
    for name, g, ref, tol in zip(("dx", "dweight", "dbias"), (DX, dw, db), ln_bwd64(x, w, m, r, dy),
                                 ln_bwd_tol(x, w, m, r, dy, dt)):
        check(g, ref, tol, name)


def test_gradient_against_differences():
    # fp64 central differences of the forward's formula confirm the formula the oracle uses
    x, w, b, dy = _case(3, 24, F32, 5)
    _, mean, rstd, _ = ln64(x, w, b, EPS)
    dx, dw, db = ln_bwd64(x, w, mean, rstd, dy)
    f = lambda x_, w_, b_: float((ln64(x_, w_, b_, EPS)[0] * dy.double()).sum())
    h = 1e-6
    for (t, c) in ((0, 0), (1, 13), (2, 23)):
        e = torch.zeros_like(x, dtype=torch.float64)
        e[t, c] = h
        num = (f(x.double() + e, w, b) - f(x.double() - e, w, b)) / (2 * h)
        assert abs(num - float(dx[t, c])) < 1e-6 * (1 + abs(num))
    for c in (0, 11):
        e = torch.zeros(24, dtype=torch.float64)
        e[c] = h
        assert abs((f(x, w.double() + e, b) - f(x, w.double() - e, b)) / (2 * h) - float(dw[c])) < 1e-5
        assert abs((f(x, w, b.double() + e) - f(x, w, b.double() - e)) / (2 * h) - float(db[c])) < 1e-5


@pytest.mark.parametrize("T,d,dt", [(37, 64, BF), (301, 1037, F32), (150, 2560, BF), (9, 8200, BF), (3, 9001, F32),
                                    (2373, 1037, BF), (2401, 515, F32), (2369, 2563, BF)])
def test_writes_stay_inside_the_outputs(T, d, dt):
    x, w, b, dy = _dev(*_case(T, d, dt, 6))
    res = []
    spec = dict(y=((T, d), dt), mean=((T,), F32), rstd=((T,), F32), dx=((T, d), dt), dw=((d,), F32), db=((d,), F32),
                ws=((mhc.mhc_layer_norm_backward_workspace_bytes(T, d),), torch.uint8))
    for guarded in (False, True):
        o, bufs = {}, []
        for k, (shape, t) in spec.items():
            if guarded:
                buf, o[k] = guarded_empty(shape, t, "cuda")
                bufs.append(buf)
            else:
                o[k] = torch.empty(shape, dtype=t, device="cuda")
        mhc.mhc_layer_norm(x, w, b, EPS, o["y"], o["mean"], o["rstd"])
        mhc.mhc_layer_norm_backward(x, w, o["mean"], o["rstd"], dy, o["dx"], o["dw"], o["db"], o["ws"])
        torch.cuda.synchronize()
        assert all(guards_intact(q) for q in bufs)
        res.append(o)
    for k in ("y", "mean", "rstd", "dx", "dw", "db"):
        assert torch.equal(res[0][k], res[1][k]), k


def test_no_tokens():
    d = 64
    e = lambda *s: torch.empty(*s, device="cuda")
    mhc.mhc_layer_norm(e(0, d), e(d), e(d), EPS, e(0, d), e(0), e(0))
    dw, db = torch.ones(d, device="cuda"), torch.ones(d, device="cuda")
    mhc.mhc_layer_norm_backward(e(0, d), e(d), e(0), e(0), e(0, d), e(0, d), dw, db)
    assert not dw.any() and not db.any()


def test_other_stream_and_captured_graph():
    x, w, b, dy = _dev(*_case(500, 1024, BF, 7))
    y0, mean, rstd = _fwd(x, w, b)
    ref = _bwd(x, w, mean, rstd, dy)
    side = torch.cuda.Stream()
    y = torch.zeros_like(x)
    dx, dw, db = torch.zeros_like(x), torch.zeros(1024, device="cuda"), torch.zeros(1024, device="cuda")
    ws = torch.empty(mhc.mhc_layer_norm_backward_workspace_bytes(500, 1024), dtype=torch.uint8, device="cuda")
    side.wait_stream(torch.cuda.current_stream())
    mhc.mhc_layer_norm(x, w, b, EPS, y, stream=side)
    mhc.mhc_layer_norm_backward(x, w, mean, rstd, dy, dx, dw, db, ws, stream=side)
    side.synchronize()
    assert torch.equal(y, y0) and all(torch.equal(p, q) for p, q in zip((dx, dw, db), ref))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mhc.mhc_layer_norm(x, w, b, EPS, y, mean, rstd)
        mhc.mhc_layer_norm_backward(x, w, mean, rstd, dy, dx, dw, db, ws)
    for shift in (0.5, -1.0):
        x.add_(shift)
        for t in (y, dx, dw, db):
            t.zero_()
        g.replay()
        y1, m1, r1 = _fwd(x, w, b)
        ref = _bwd(x, w, m1, r1, dy)
        assert torch.equal(y, y1) and all(torch.equal(p, q) for p, q in zip((dx, dw, db), ref))
