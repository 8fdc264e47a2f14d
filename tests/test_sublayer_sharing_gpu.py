"""The sub-layer operators where calls or buffers meet: calls on two streams at once, one buffer as
two inputs, a captured graph of the fp32 products, and arrays whose offsets pass 32 bits."""
import pytest

from _sublayer import HALF, U, act64, check, ln64, ln_bwd64, ln_bwd_tol, ln_tol, slope64, sum_tol

torch = pytest.importorskip("torch")
mhc = pytest.importorskip("mhc_hyper_connections_b200")

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def _bytes(n):
    return torch.empty(max(n, 1), dtype=torch.uint8, device="cuda")


class _Layer:
    """Layer norm and a projection with GELU, forward and backward, on buffers of its own."""

    def __init__(self, T, K, N, dt, seed):
        g = torch.Generator().manual_seed(seed)
        r = lambda *s: torch.randn(*s, generator=g)
        self.x, self.dy = r(T, K).to(dt).cuda(), r(T, N).to(dt).cuda()
        self.W = (r(N, K) / K ** 0.5).to(dt).cuda()
        self.w, self.b, self.c = (1 + 0.2 * r(K)).cuda(), r(K).cuda(), r(N).cuda()
        e = lambda *s, t=F32: torch.zeros(*s, dtype=t, device="cuda")
        self.xn, self.dxn, self.dx = (e(T, K, t=dt) for _ in range(3))
        self.y, self.z = e(T, N, t=dt), e(T, N, t=dt)
        self.mean, self.rstd = e(T), e(T)
        self.dW, self.dc, self.dw, self.db = e(N, K, t=dt), e(N), e(K), e(K)
        self.ws = [_bytes(mhc.mhc_linear_workspace_bytes(T, K, N, dt)),
                   _bytes(mhc.mhc_linear_backward_workspace_bytes(T, K, N, dt)),
                   _bytes(mhc.mhc_layer_norm_backward_workspace_bytes(T, K))]

    def outputs(self):
        return (self.xn, self.mean, self.rstd, self.y, self.z, self.dxn, self.dW, self.dc, self.dx, self.dw, self.db)

    def run(self, stream=None):
        mhc.mhc_layer_norm(self.x, self.w, self.b, 1e-5, self.xn, self.mean, self.rstd, stream=stream)
        mhc.mhc_linear(self.xn, self.W, self.c, self.y, act=mhc.ACT_GELU, z=self.z, workspace=self.ws[0],
                       stream=stream)
        mhc.mhc_linear_backward(self.xn, self.W, self.z, self.dy, self.dxn, self.dW, self.dc, self.ws[1],
                                act=mhc.ACT_GELU, stream=stream)
        mhc.mhc_layer_norm_backward(self.x, self.w, self.mean, self.rstd, self.dxn, self.dx, self.dw, self.db,
                                    self.ws[2], stream=stream)


@pytest.mark.parametrize("a,b", [((1, 1024, 512, BF), (300, 256, 520, BF)), ((40, 520, 264, BF), (40, 520, 264, BF)),
                                 ((2500, 256, 2056, BF), (1, 2048, 4096, BF)), ((1000, 1000, 1003, F32), (33, 130, 66, BF)),
                                 ((2400, 515, 200, BF), (2400, 512, 200, F32))])
def test_two_streams_at_once(a, b):
    layers = [_Layer(*a, seed=1), _Layer(*b, seed=2)]
    refs = []
    for m in layers:
        m.run()
        torch.cuda.synchronize()
        refs.append([t.clone() for t in m.outputs()])
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        for m in layers:
            for t in m.outputs():
                t.zero_()
        for s in streams:
            s.wait_stream(torch.cuda.current_stream())
        for _ in range(4):
            for m, s in zip(layers, streams):
                m.run(stream=s)
        torch.cuda.synchronize()
        for m, ref in zip(layers, refs):
            assert all(torch.equal(p, q) for p, q in zip(m.outputs(), ref))
    assert mhc.mhc_device_status() == 0


@pytest.mark.parametrize("T,K,N", [(5, 64, 72), (130, 520, 264), (1000, 1000, 1003)])
def test_captured_graph_in_fp32(T, K, N):
    m = _Layer(T, K, N, F32, seed=3)
    g = torch.cuda.CUDAGraph()
    m.run()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        m.run()
    for s in (2.0, 0.5):
        m.x.mul_(s)
        m.run()
        ref = [t.clone() for t in m.outputs()]
        for t in m.outputs():
            t.zero_()
        g.replay()
        assert all(torch.equal(p, q) for p, q in zip(m.outputs(), ref))


@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("n", [72, 300])
def test_one_buffer_as_several_inputs(n, dt):
    g = torch.Generator().manual_seed(n)
    x = torch.randn(n, n, generator=g).to(dt)
    d, xd = x.cuda(), x.double()
    y = torch.empty_like(d)
    s = xd.abs() @ xd.abs().T
    # x as activations, weights and residual: y = x x^T + x
    mhc.mhc_linear(d, d, None, y, residual=d, workspace=_bytes(mhc.mhc_linear_workspace_bytes(n, n, n, dt)))
    ref = xd @ xd.T + xd
    check(y, ref, HALF[dt] * ref.abs() + sum_tol(n) * s + 2 * U * (xd.abs() + s), "y")
    # and as upstream gradient too: dx = x x, dW = x^T x
    dx, dW = torch.empty_like(d), torch.empty_like(d)
    mhc.mhc_linear_backward(d, d, None, d, dx, dW, None,
                            _bytes(mhc.mhc_linear_backward_workspace_bytes(n, n, n, dt)))
    for got, a, b in ((dx, xd, xd), (dW, xd.T, xd)):
        ref = a @ b
        check(got, ref, HALF[dt] * ref.abs() + sum_tol(n) * (a.abs() @ b.abs()), "product")
    # layer norm's gradient with dy = x
    w = torch.ones(n)
    yn, mean, rstd = torch.empty_like(d), torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
    mhc.mhc_layer_norm(d, None, None, 1e-5, yn, mean, rstd)
    dw, db = torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
    mhc.mhc_layer_norm_backward(d, None, mean, rstd, d, dx, dw, db,
                                _bytes(mhc.mhc_layer_norm_backward_workspace_bytes(n, n)))
    m, r = mean.cpu(), rstd.cpu()
    for got, ref, tol, what in zip((dx, dw, db), ln_bwd64(x, w, m, r, x), ln_bwd_tol(x, w, m, r, x, dt),
                                   ("dx", "dweight", "dbias")):
        check(got, ref, tol, what)


def test_gelu_in_fp32_keeps_its_small_side():
    # x = 0, so z is the bias.  erfc's argument carries two roundings, which its slope turns into
    # 2 (z^2 + 1) u of the value; 8 u for the library function (4 ulp), 2 u for the products.
    z = torch.linspace(-12, 12, 4801)
    x, W = torch.zeros(3, 4, device="cuda"), torch.zeros(z.numel(), 4, device="cuda")
    y = torch.empty(3, z.numel(), device="cuda")
    mhc.mhc_linear(x, W, z.cuda(), y, act=mhc.ACT_GELU,
                   workspace=_bytes(mhc.mhc_linear_workspace_bytes(3, 4, z.numel(), F32)))
    ref = act64(z.double(), "gelu")
    check(y, ref.expand(3, -1), (ref.abs() * (2 * (z.double() ** 2 + 1) + 10) * U).expand(3, -1), "gelu")


def _long_rows(T, d, dt, seed):
    """[T, d] with the rows of one block of 4096 over and over: its oracle needs one block."""
    g = torch.Generator().manual_seed(seed)
    base = torch.randn(4096, d, generator=g).to(dt)
    out = torch.empty(T, d, dtype=dt, device="cuda")
    b = base.cuda()
    for t in range(0, T, 4096):
        out[t:t + 4096] = b[:min(4096, T - t)]
    return base, out


@pytest.mark.parametrize("d", [4096, 4095])
def test_layer_norm_past_32_bit_offsets(d):
    T = (1 << 31) // d + 2049                       # more than 2^31 elements; a last block cut short
    base, x = _long_rows(T, d, BF, d)
    g = torch.Generator().manual_seed(5)
    w, b = 1 + 0.2 * torch.randn(d, generator=g), torch.randn(d, generator=g)
    y, mean, rstd = torch.empty_like(x), torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    mhc.mhc_layer_norm(x, w.cuda(), b.cuda(), 1e-5, y, mean, rstd)
    ref, rm, rr, _ = ln64(base, w, b, 1e-5)
    ty, tm, tr = ln_tol(base, w, b, 1e-5, BF)
    last = (T - 1) // 4096 * 4096
    for got, r, tol in ((y, ref, ty), (mean, rm, tm), (rstd, rr, tr)):
        check(got[:4096], r, tol, "first")
        check(got[last:], r[:T - last], tol[:T - last], "last")
    assert all(torch.equal(y[t:t + 4096], y[:min(4096, T - t)]) for t in range(0, T, 4096))
    # backward with dy = x: every block of rows has the same dx, and the column sums are the block's, as
    # often as it occurs
    dx = y
    dw, db = torch.empty(d, device="cuda"), torch.empty(d, device="cuda")
    mhc.mhc_layer_norm_backward(x, w.cuda(), mean, rstd, x, dx, dw, db,
                                _bytes(mhc.mhc_layer_norm_backward_workspace_bytes(T, d)))
    m, r = mean[:4096].cpu(), rstd[:4096].cpu()
    rdx, _, _ = ln_bwd64(base, w, m, r, base)
    check(dx[last:], rdx[:T - last], ln_bwd_tol(base, w, m, r, base, BF)[0][:T - last], "dx")
    assert all(torch.equal(dx[t:t + 4096], dx[:min(4096, T - t)]) for t in range(0, T, 4096))
    xd = base.double()
    xh = (xd - m.double()[:, None]) * r.double()[:, None]
    n = torch.full((4096,), last // 4096, dtype=torch.float64)
    n[:T - last] += 1
    tol = (T + 76) * U
    check(dw, n @ (xd * xh), tol * (n @ (xd * xh).abs()), "dweight")
    check(db, n @ xd, tol * (n @ xd.abs()), "dbias")
    assert mhc.mhc_device_status() == 0


@pytest.mark.parametrize("N", [16384, 16381])
def test_linear_past_32_bit_offsets(N):
    K = 64
    T = (1 << 31) // N + 2049
    base, x = _long_rows(T, K, BF, N)
    g = torch.Generator().manual_seed(6)
    W, c = (torch.randn(N, K, generator=g) / 8).to(BF), torch.randn(N, generator=g)
    y, z = torch.empty(T, N, dtype=BF, device="cuda"), torch.empty(T, N, dtype=BF, device="cuda")
    mhc.mhc_linear(x, W.cuda(), c.cuda(), y, act=mhc.ACT_SILU, z=z,
                   workspace=_bytes(mhc.mhc_linear_workspace_bytes(T, K, N, BF)))
    last = (T - 1) // 4096 * 4096
    rows = T - 64                                   # the last rows, of the block that is cut short
    xr = base[rows - last:T - last].double()
    zr = xr @ W.double().T + c.double()
    tz = sum_tol(K) * (xr.abs() @ W.double().abs().T + c.double().abs())
    check(z[rows:], zr, HALF[BF] * zr.abs() + tz, "z")
    yr = act64(zr, "silu")
    check(y[rows:], yr, (HALF[BF] + 2.0 ** -16) * yr.abs() + 1.13 * tz + 8 * U * zr.abs(), "y")
    for t in (y, z):
        assert all(torch.equal(t[i:i + 4096], t[:min(4096, T - i)]) for i in range(0, T, 4096))
    # dx of the last rows, with y as the upstream gradient; the column sums count the blocks
    dx, db = torch.empty_like(x), torch.empty(N, device="cuda")
    mhc.mhc_linear_backward(x, W.cuda(), z, y, dx, None, db,
                            _bytes(mhc.mhc_linear_backward_workspace_bytes(T, K, N, BF)), act=mhc.ACT_SILU)
    dy, slope = y[:4096].double(), slope64(z[:4096].double(), "silu")
    dz = dy * slope
    e0 = 2.0 ** -16 * dy.abs()                      # the slope's short form
    d64, e = dz[rows - last:T - last].cpu(), (e0 + HALF[BF] * dz.abs())[rows - last:T - last].cpu()
    ref, Wd = d64 @ W.double(), W.double()
    check(dx[rows:], ref, HALF[BF] * ref.abs() + e @ Wd.abs() + sum_tol(N) * (d64.abs() @ Wd.abs()), "dx")
    assert all(torch.equal(dx[i:i + 4096], dx[:min(4096, T - i)]) for i in range(0, T, 4096))
    n = torch.full((4096,), last // 4096, dtype=torch.float64, device="cuda")
    n[:T - last] += 1
    check(db, (n @ dz).cpu(), (n @ e0 + (T + 80) * U * (n @ dz.abs())).cpu(), "dbias")
    assert mhc.mhc_device_status() == 0


def test_two_host_threads_at_once():
    # rows of many lengths that share kernels, each thread on a stream of its own
    import threading
    errors = []
    widths = ([2048, 1544, 2560, 4096, 520], [1800, 2048, 4000, 2112, 600])

    def work(k):
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                layers = [_Layer(600, d, 136, BF, seed=d) for d in widths[k]]
                s.synchronize()
                for _ in range(2):
                    for _ in range(30):
                        for m in layers:
                            m.run()
                    s.synchronize()
                    res = [[t.clone() for t in m.outputs()] for m in layers]
                    for m, ref in zip(layers, res):
                        m.run()
                        s.synchronize()
                        assert all(torch.equal(p, q) for p, q in zip(m.outputs(), ref))
        except BaseException as e:      # noqa: BLE001 -- reported by the main thread
            errors.append(e)

    threads = [threading.Thread(target=work, args=(k,)) for k in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    assert mhc.mhc_device_status() == 0
