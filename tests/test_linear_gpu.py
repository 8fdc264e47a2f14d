"""mhc_linear and mhc_linear_backward against 64-bit oracles (bounds in _sublayer.py): one token
to many, odd sizes, every activation, with and without bias, residual and saved pre-activation,
unaligned buffers, non-finite inputs, streams, captured graphs, guard regions, repeatability."""
import pytest

from _canary import guarded_empty, guards_intact
from _sublayer import ACTS, U, act64, check, half, slope64, sum_tol

torch = pytest.importorskip("torch")
mhc = pytest.importorskip("mhc_hyper_connections_b200")

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
ACT = {a: getattr(mhc, "ACT_" + a.upper()) for a in ACTS}

# (T, K, N): single tokens, tile edges either side, odd sizes, more than one tile each way, sums
# longer than one stage of any kernel
SHAPES = [(1, 1, 1), (1, 64, 64), (1, 4096, 1024), (1, 129, 37), (2, 8, 8), (3, 17, 5), (7, 64, 257), (8, 512, 136),
          (16, 1024, 512), (17, 96, 128), (33, 72, 200), (48, 2048, 520), (64, 256, 1024), (65, 130, 66),
          (100, 1027, 130), (127, 128, 127), (128, 64, 128), (129, 192, 257), (200, 320, 96), (255, 65, 511),
          (256, 256, 256), (300, 100, 300), (513, 1031, 264), (777, 264, 1029), (1024, 512, 768), (2100, 136, 520),
          # enough 256-wide tiles for the paired kernel: forward, dx and dW in turn, several tiles per
          # pair, ragged in each direction, rows of outputs that are not 16-byte aligned
          (2500, 200, 2100), (2311, 72, 2565), (5000, 64, 5000), (2500, 2100, 200), (3001, 2056, 168), (100, 2504, 2104),
          (520, 4104, 3336)]


def _case(T, K, N, dt, seed=0):
    g = torch.Generator().manual_seed(100003 * T + 101 * K + N + seed)
    r = lambda *s: torch.randn(*s, generator=g)
    return dict(x=r(T, K).to(dt), W=(r(N, K) / K ** 0.5).to(dt), bias=0.5 * r(N), residual=r(T, N).to(dt),
                dy=r(T, N).to(dt))


def _workspace(n):
    return torch.empty(n, dtype=torch.uint8, device="cuda") if n else None


def _cuda(c):
    return {k: None if v is None else v.cuda() for k, v in c.items()}


def _fwd(c, act, bias=True, residual=True, z=True):
    c = _cuda(c)
    (T, K), N = c["x"].shape, c["W"].shape[0]
    y = torch.empty(T, N, dtype=c["x"].dtype, device="cuda")
    zz = torch.empty_like(y) if z else None
    mhc.mhc_linear(c["x"], c["W"], c["bias"] if bias else None, y, act=ACT[act],
                   residual=c["residual"] if residual else None, z=zz,
                   workspace=_workspace(mhc.mhc_linear_workspace_bytes(T, K, N, y.dtype)))
    return y, zz


def _fwd_check(c, act, got, bias=True, residual=True):
    x, W, dt = c["x"].double(), c["W"].double(), c["x"].dtype
    z = x @ W.T
    s = (x.abs() @ W.abs().T)
    if bias:
        z = z + c["bias"].double()
        s = s + c["bias"].double().abs()
    y = act64(z, act)
    # the activation's slope is at most 1.13 in size, and its own fp32 evaluation is off by at most
    # 8 u |z| (a few roundings and the library function's two), or by 2^-16 |y| in its short form for
    # bf16 storage
    tz = sum_tol(x.shape[1]) * s
    ty = 1.13 * tz + 8 * U * z.abs() + (2.0 ** -16 * y.abs() if dt == BF and act != "none" else 0)
    if residual:
        y = y + c["residual"].double()
        ty = ty + 2 * U * (c["residual"].double().abs() + z.abs())
    check(got[0], y, half(dt) * y.abs() + ty, "y")
    if got[1] is not None:
        check(got[1], z, half(dt) * z.abs() + tz, "z")


def _bwd(c, z, act, want=(True, True, True)):
    c = _cuda(c)
    (T, K), N = c["x"].shape, c["W"].shape[0]
    dx = torch.empty_like(c["x"]) if want[0] else None
    dW = torch.empty_like(c["W"]) if want[1] else None
    db = torch.empty(N, device="cuda") if want[2] else None
    ws = torch.empty(mhc.mhc_linear_backward_workspace_bytes(T, K, N, c["x"].dtype), dtype=torch.uint8, device="cuda")
    mhc.mhc_linear_backward(c["x"], c["W"], None if z is None else z.cuda(), c["dy"], dx, dW, db, ws, act=ACT[act])
    return dx, dW, db


def _bwd_check(c, z, act, got):
    x, W, dy, dt = c["x"].double(), c["W"].double(), c["dy"].double(), c["x"].dtype
    T, N = dy.shape
    dz = dy if act == "none" else dy * slope64(z.double(), act)
    # dz: the slope's fp32 evaluation (16 u of 1.13 + |z| phi(z) terms below 2; 2^-16 in its short form
    # for bf16 storage) and one rounding to the storage type as the products' operand
    e0 = torch.zeros_like(dz) if act == "none" else (32 * U if dt == F32 else 2.0 ** -16) * dy.abs()
    e = e0 if act == "none" or dt == F32 else e0 + half(dt) * dz.abs()
    dx, dW, db = dz @ W, dz.T @ x, dz.sum(0)
    check(got[0], dx, half(dt) * dx.abs() + e @ W.abs() + sum_tol(N) * (dz.abs() @ W.abs()), "dx")
    check(got[1], dW, half(dt) * dW.abs() + e.T @ x.abs() + sum_tol(T) * (dz.abs().T @ x.abs()), "dW")
    check(got[2], db, e0.sum(0) + (T + 80) * U * dz.abs().sum(0), "dbias")
    # two roundings (dz, output) of at most half a step each: their rms is below half a step
    # over sqrt(3) each, whatever their signs
    for g, r in ((got[0], dx), (got[1], dW)):
        if r.numel() >= 1000 and dt == BF:
            err = (g.cpu().double() - r).square().mean().sqrt() / r.square().mean().sqrt()
            assert err < half(dt), float(err)


@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("i,T,K,N", [(i, *s) for i, s in enumerate(SHAPES)])
def test_forward_and_backward(i, T, K, N, dt):
    act = ACTS[i % len(ACTS)]
    c = _case(T, K, N, dt)
    y, z = _fwd(c, act)
    _fwd_check(c, act, (y, z))
    # bitwise repeatable, with and without the saved pre-activation
    y2, z2 = _fwd(c, act)
    assert torch.equal(y, y2) and torch.equal(z, z2) and torch.equal(_fwd(c, act, z=False)[0], y)
    _fwd_check(c, act, _fwd(c, act, bias=False, residual=False), False, False)
    zc = None if act == "none" else z.cpu()
    got = _bwd(c, zc, act)
    _bwd_check(c, zc, act, got)
    for k in range(3):
        want = tuple(j == k for j in range(3))
        assert torch.equal(_bwd(c, zc, act, want)[k], got[k])
    assert mhc.mhc_device_status() == 0


@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("T,K,N", [(2, 64, 136), (130, 128, 264)])
def test_every_activation_over_its_range(T, K, N, act, dt):
    c = _case(T, K, N, dt, 1)
    c["W"] = (c["W"].float() * 8).to(dt)              # pre-activations to |z| ~ 35
    y, z = _fwd(c, act)
    _fwd_check(c, act, (y, z))
    zc = z.cpu()
    zc[0, :16] = torch.tensor([0.0, -0.0, 1e-30, -1e-30, 6.0, -6.0, 9.5, -9.5, 40.0, -40.0, 200.0, -200.0, 1e4, -1e4,
                               1e19, -1e19]).to(dt)
    _bwd_check(c, zc, act, _bwd(c, zc, act))


@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("T,K,N", [(1, 64, 72), (40, 256, 128), (200, 128, 264)])
def test_unaligned_buffers(T, K, N, dt):
    c = _case(T, K, N, dt, 2)
    off = lambda t: torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")[1:].view(t.shape).copy_(t)
    d = {k: off(v) for k, v in c.items()}
    y, z = off(c["dy"]), off(c["dy"])
    ws = _workspace(mhc.mhc_linear_workspace_bytes(T, K, N, dt))
    mhc.mhc_linear(d["x"], d["W"], d["bias"], y, act=mhc.ACT_SILU, residual=d["residual"], z=z, workspace=ws)
    _fwd_check(c, "silu", (y, z))
    dx, dW, db = off(c["x"]), off(c["W"]), off(c["bias"])
    ws = _workspace(mhc.mhc_linear_backward_workspace_bytes(T, K, N, dt))
    mhc.mhc_linear_backward(d["x"], d["W"], z, d["dy"], dx, dW, db, ws, act=mhc.ACT_SILU)
    _bwd_check(c, z.cpu(), "silu", (dx, dW, db))


@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("T,K,N", [(5, 64, 64), (140, 136, 264), (300, 130, 70)])
def test_non_finite_tokens_stay_in_their_rows(T, K, N, dt):
    c = _case(T, K, N, dt, 3)
    c["x"][2, K - 1] = float("inf")
    c["x"][4, 0] = float("nan")
    y, z = _fwd(c, "none")
    assert not torch.isfinite(y[2]).any() and torch.isnan(y[4]).all()
    keep = [t for t in range(T) if t not in (2, 4)]
    for k in ("x", "residual", "dy"):
        c[k] = c[k][keep]
    _fwd_check(c, "none", (y[keep], z[keep]))


@pytest.mark.parametrize("which", ["x", "W", "none"])
def test_fp32_values_without_bf16_parts(which):
    # fp32 products of this size are formed from bf16 parts, which infinities, NaN and values next to
    # fp32's largest do not have: the result is that of fp32 arithmetic all the same
    T, K, N = 600, 2048, 1030
    c = _case(T, K, N, F32, 7)
    if which != "none":
        c[which][3, 5] = float("inf")
        c[which][7, K - 1] = -float("inf")
        c[which][11, 0] = float("nan")
        c[which][13, 64] = 3.4e38
    for act in ("none", "relu"):
        y, z = _fwd(c, act, residual=False)
        ref = c["x"].double() @ c["W"].double().T + c["bias"].double()
        got = z.cpu().double()
        ref32 = ref.float().double()                      # sums past fp32's range are infinite
        s = c["x"].double().abs() @ c["W"].double().abs().T + c["bias"].double().abs()
        fin = torch.isfinite(ref32)
        assert torch.equal(torch.isnan(got), torch.isnan(ref32))
        assert torch.equal(got[~fin & ~torch.isnan(ref32)], ref32[~fin & ~torch.isnan(ref32)])
        assert ((got - ref).abs() <= U * ref.abs() + sum_tol(K) * s)[fin].all()
        keep = ~torch.isnan(ref32)
        assert torch.equal(y.cpu()[keep], act64(z.cpu(), act)[keep])
    dx, dW, db = _bwd(c, None, "none")
    for g, r in ((dx, c["dy"].double() @ c["W"].double()), (dW, c["dy"].double().T @ c["x"].double())):
        r32 = r.float().double()
        assert torch.equal(torch.isnan(g.cpu()), torch.isnan(r32))
        inf = torch.isinf(r32)
        assert torch.equal(g.cpu().double()[inf], r32[inf])


def test_gradient_against_differences():
    # fp64 central differences of the forward's formula confirm the gradients the oracle uses
    c = _case(3, 6, 5, F32, 4)
    x, W, b, dy = (c[k].double() for k in ("x", "W", "bias", "dy"))
    h = 1e-6
    for act in ACTS:
        f = lambda x_, W_, b_: float((act64(x_ @ W_.T + b_, act) * dy).sum())
        dz = dy * slope64(x @ W.T + b, act)
        for grad, at, args in ((dz @ W, x, 0), (dz.T @ x, W, 1), (dz.sum(0), b, 2)):
            for flat in (0, at.numel() // 2, at.numel() - 1):
                e = torch.zeros_like(at).view(-1)
                e[flat] = h
                lo, hi = [x, W, b], [x, W, b]
                lo[args], hi[args] = at - e.view_as(at), at + e.view_as(at)
                assert abs((f(*hi) - f(*lo)) / (2 * h) - float(grad.reshape(-1)[flat])) < 1e-6


@pytest.mark.parametrize("T,K,N,dt", [(1, 64, 200, BF), (37, 130, 70, BF), (140, 128, 264, BF), (300, 264, 520, BF),
                                      (65, 100, 130, F32)])
def test_writes_stay_inside_the_outputs(T, K, N, dt):
    c = _cuda(_case(T, K, N, dt, 5))
    spec = dict(y=((T, N), dt), z=((T, N), dt), dx=((T, K), dt), dW=((N, K), dt), db=((N,), F32),
                ws=((mhc.mhc_linear_workspace_bytes(T, K, N, dt),), torch.uint8),
                wsb=((mhc.mhc_linear_backward_workspace_bytes(T, K, N, dt),), torch.uint8))
    res = []
    for guarded in (False, True):
        o, bufs = {}, []
        for k, (shape, t) in spec.items():
            if guarded:
                buf, o[k] = guarded_empty(shape, t, "cuda")
                bufs.append(buf)
            else:
                o[k] = torch.empty(shape, dtype=t, device="cuda")
        mhc.mhc_linear(c["x"], c["W"], c["bias"], o["y"], act=mhc.ACT_GELU, residual=c["residual"], z=o["z"],
                       workspace=o["ws"])
        mhc.mhc_linear_backward(c["x"], c["W"], o["z"], c["dy"], o["dx"], o["dW"], o["db"], o["wsb"],
                                act=mhc.ACT_GELU)
        torch.cuda.synchronize()
        assert all(guards_intact(b) for b in bufs)
        res.append(o)
    for k in ("y", "z", "dx", "dW", "db"):
        assert torch.equal(res[0][k], res[1][k]), k


def test_no_tokens():
    e = lambda *s: torch.empty(*s, device="cuda")
    mhc.mhc_linear(e(0, 8), e(16, 8), e(16), e(0, 16))
    dW, db = torch.ones(16, 8, device="cuda"), torch.ones(16, device="cuda")
    mhc.mhc_linear_backward(e(0, 8), e(16, 8), None, e(0, 16), e(0, 8), dW, db, None)
    assert not dW.any() and not db.any()


@pytest.mark.parametrize("T,K,N", [(1, 512, 264), (24, 1024, 256), (300, 256, 520), (70, 130, 66)])
def test_other_stream_and_captured_graph(T, K, N):
    c = _cuda(_case(T, K, N, BF, 6))
    y0, z0 = _fwd(c, "gelu")
    ref = _bwd(c, z0, "gelu")
    ws = _workspace(mhc.mhc_linear_workspace_bytes(T, K, N, BF))
    wsb = _workspace(mhc.mhc_linear_backward_workspace_bytes(T, K, N, BF))
    o = [torch.zeros_like(t) for t in (y0, z0, *ref)]

    def call(**kw):
        mhc.mhc_linear(c["x"], c["W"], c["bias"], o[0], act=mhc.ACT_GELU, residual=c["residual"], z=o[1],
                       workspace=ws, **kw)
        mhc.mhc_linear_backward(c["x"], c["W"], o[1], c["dy"], *o[2:], wsb, act=mhc.ACT_GELU, **kw)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    call(stream=side)
    side.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(o, (y0, z0, *ref)))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for s in (2.0, 0.25):
        c["x"].mul_(s)
        for t in o:
            t.zero_()
        g.replay()
        y1, z1 = _fwd(c, "gelu")
        assert all(torch.equal(p, q) for p, q in zip(o, (y1, z1, *_bwd(c, z1, "gelu"))))
