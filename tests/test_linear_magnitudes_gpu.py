"""fp32 products over the whole range of fp32: operands too small or too large for bf16 parts as they lie,
sums past what scaled parts hold, and values of every magnitude side by side."""
import pytest

from _sublayer import U, check, sum_tol

torch = pytest.importorskip("torch")
mhc = pytest.importorskip("mhc_hyper_connections_b200")

pytestmark = pytest.mark.gpu
F32 = torch.float32
# half a step of fp32's subnormal numbers: what a result below 2^-126 may be off by per rounding, and at
# most 32 roundings there (parts of a tile, their sum, the product's own)
TINY = 32 * 2.0 ** -150


def _ws(n):
    return torch.empty(max(n, 1), dtype=torch.uint8, device="cuda")


def _linear(x, W):
    T, K, N = *x.shape, W.shape[0]
    y = torch.empty(T, N, device="cuda")
    mhc.mhc_linear(x.cuda(), W.cuda(), None, y, workspace=_ws(mhc.mhc_linear_workspace_bytes(T, K, N, F32)))
    return y.cpu()


def _backward(x, W, dy, want=(True, True)):
    T, K, N = *x.shape, W.shape[0]
    dx = torch.empty(T, K, device="cuda") if want[0] else None
    dW = torch.empty(N, K, device="cuda") if want[1] else None
    mhc.mhc_linear_backward(x.cuda(), W.cuda(), None, dy.cuda(), dx, dW, None,
                            _ws(mhc.mhc_linear_backward_workspace_bytes(T, K, N, F32)))
    return [None if t is None else t.cpu() for t in (dx, dW)]


def _case(T, K, N, seed):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*s, generator=g) for s in ((T, K), (N, K), (T, N)))


def _check(got, a, b, what):
    a, b = a.double(), b.double()
    ref = a @ b
    check(got, ref, U * ref.abs() + sum_tol(a.shape[1]) * (a.abs() @ b.abs()) + TINY, what)


# from bf16 parts, the last of them with tiles shared along K, and on CUDA cores
@pytest.mark.parametrize("T,K,N", [(600, 2048, 1030), (192, 4096, 1024), (20, 96, 40)])
@pytest.mark.parametrize("sx,sw", [(1e-34, 1), (1e-36, 1), (1, 1e-36), (1e-38, 1), (1e-36, 1e30), (1e-41, 1e10),
                                   (1e-20, 1e-17), (1e18, 1e17), (1e20, 1e14), (1e33, 1), (1, 1e34)])
def test_scaled_operands(T, K, N, sx, sw):
    x, W, dy = _case(T, K, N, 11)
    x, W = x * sx, W * sw
    _check(_linear(x, W), x, W.T, "y")
    # W's scale meets dy in dx, x's in dW
    dx, dW = _backward(x, W, dy)
    _check(dx, dy, W, "dx")
    _check(dW, dy.T, x, "dW")
    small = dy * min(sx, sw)
    dx, dW = _backward(x / sx, W / sw, small)
    _check(dx, small, W / sw, "dx of a small dy")
    _check(dW, small.T, x / sx, "dW of a small dy")


def _every_magnitude(shape, seed, top):
    """fp32 numbers of random significands, with exponents from the smallest subnormal to 2^top."""
    g = torch.Generator().manual_seed(seed)
    m = 1 + torch.rand(*shape, generator=g, dtype=torch.float64)
    e = torch.randint(-149, top, shape, generator=g).double()
    s = torch.randint(0, 2, shape, generator=g).double() * 2 - 1
    return (s * m * 2.0 ** e).float()


@pytest.mark.parametrize("top", [93, 127])      # 127: beyond the scaled parts too
def test_values_of_every_magnitude_pass_through_a_selection(top):
    # every output is one operand times 1 and zeros: it has to be that operand's bits, whatever else
    # stands in its row and column
    T, n = 600, 1024
    perm = torch.randperm(n, generator=torch.Generator().manual_seed(5))
    P = torch.zeros(n, n)
    P[torch.arange(n), perm] = 1.0
    a = _every_magnitude((T, n), 6, top)
    assert torch.equal(_linear(a, P), a[:, perm])                            # y[t][j] = a[t][perm[j]]
    W = a[:, perm].contiguous()
    assert torch.equal(_linear(P, W), W[:, perm].T)                          # y[i][t] = W[t][perm[i]]
    dx = _backward(a, P, a)[0]                                               # dx[t][perm[j]] = a[t][j]
    assert torch.equal(dx[:, perm], a)
    # dW = dz^T x with dz or x the selection: rows of the other in another order
    b = _every_magnitude((n, T), 7, top)
    assert torch.equal(_backward(b, torch.ones(n, T), P, (False, True))[1], b[torch.argsort(perm)])
    assert torch.equal(_backward(P, torch.ones(T, n), b, (False, True))[1], b.T[:, torch.argsort(perm)])


def test_a_call_with_large_sums_leaves_the_next_one_to_the_tensor_cores():
    # the words that send a product to the CUDA cores belong to a call: the same workspace, a call with
    # large sums and values without parts, then an ordinary one that has to give the bits it gave before
    T, K, N = 600, 2048, 1030
    x, W, dy = (t.cuda() for t in _case(T, K, N, 13))
    ws, wb = (_ws(f(T, K, N, F32)) for f in (mhc.mhc_linear_workspace_bytes, mhc.mhc_linear_backward_workspace_bytes))
    out = lambda: (torch.empty(T, N, device="cuda"), torch.empty(T, K, device="cuda"), torch.empty(N, K, device="cuda"))

    def call(x, W, dy):
        y, dx, dW = out()
        mhc.mhc_linear(x, W, None, y, workspace=ws)
        mhc.mhc_linear_backward(x, W, None, dy, dx, dW, None, wb)
        return y, dx, dW
    ref = call(x, W, dy)
    for sx, sw, sy in ((1e18, 1e18, 1.0), (1.0, 1e18, 1e18), (1e18, 1.0, 1e18), (1e34, 1.0, 1.0)):
        for g in call(x * sx, W * sw, dy * sy):
            assert torch.isfinite(g).all()
        assert all(torch.equal(p, q) for p, q in zip(call(x, W, dy), ref))
