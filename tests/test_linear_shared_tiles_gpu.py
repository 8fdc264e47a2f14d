"""mhc_linear and mhc_linear_backward where the tiles of the tensor-core kernels' last round are shared
along K: their parts go through the workspace and are joined by a second kernel.  Ragged in each
direction, rows of outputs that are not 16-byte aligned, every input of the epilogue, a workspace of
exactly the size asked for, and captured graphs that share one."""
import pytest

from _canary import guarded_empty, guards_intact
from test_linear_gpu import _bwd, _bwd_check, _case, _cuda, _fwd, _fwd_check, _workspace

torch = pytest.importorskip("torch")
mhc = pytest.importorskip("mhc_hyper_connections_b200")

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32

# (T, K, N, type): the forward product shares tiles in the first six, dx or dW in the others
SHAPES = [(700, 8192, 1100, BF), (2300, 8200, 1003, BF), (1030, 9001, 1300, BF), (250, 4096, 300, F32),
          (257, 2051, 1003, F32), (100, 4100, 1028, F32), (600, 1100, 8192, BF), (8190, 704, 1001, BF), (8190, 2500, 2100, BF),
          (1500, 1030, 130, F32), (2600, 520, 264, F32)]


@pytest.mark.parametrize("T,K,N,dt", SHAPES)
def test_forward_and_backward(T, K, N, dt):
    c = _case(T, K, N, dt, 11)
    y, z = _fwd(c, "gelu")
    _fwd_check(c, "gelu", (y, z))
    y2, z2 = _fwd(c, "gelu")
    assert torch.equal(y, y2) and torch.equal(z, z2) and torch.equal(_fwd(c, "gelu", z=False)[0], y)
    _fwd_check(c, "silu", _fwd(c, "silu", bias=False, residual=False), False, False)
    zc = z.cpu()
    got = _bwd(c, zc, "gelu")
    _bwd_check(c, zc, "gelu", got)
    for k in range(3):
        want = tuple(j == k for j in range(3))
        assert torch.equal(_bwd(c, zc, "gelu", want)[k], got[k])
    assert mhc.mhc_device_status() == 0


@pytest.mark.parametrize("T,K,N,dt", [(700, 8192, 1100, BF), (257, 2051, 1003, F32)])
def test_workspace_of_the_size_asked_for(T, K, N, dt):
    c = _cuda(_case(T, K, N, dt, 12))
    y0, _ = _fwd(c, "relu")
    guard, ws = guarded_empty((mhc.mhc_linear_workspace_bytes(T, K, N, dt),), torch.uint8, "cuda")
    gy, y = guarded_empty((T, N), dt, "cuda")
    mhc.mhc_linear(c["x"], c["W"], c["bias"], y, act=mhc.ACT_RELU, residual=c["residual"], workspace=ws)
    torch.cuda.synchronize()
    assert guards_intact(guard) and guards_intact(gy)
    assert torch.equal(y, y0)


@pytest.mark.parametrize("T,K,N,dt", [(700, 8192, 1100, BF), (250, 4096, 300, F32)])
def test_graphs_that_share_a_workspace(T, K, N, dt):
    ws = _workspace(mhc.mhc_linear_workspace_bytes(T, K, N, dt))
    cases = [_cuda(_case(T, K, N, dt, s)) for s in (13, 14)]
    refs = [_fwd(c, "none", z=False)[0] for c in cases]
    ys = [torch.zeros_like(r) for r in refs]
    graphs = []
    for c, y in zip(cases, ys):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            mhc.mhc_linear(c["x"], c["W"], c["bias"], y, residual=c["residual"], workspace=ws)
        graphs.append(g)
    for _ in range(5):
        for y in ys:
            y.zero_()
        for g in graphs:
            g.replay()
        assert all(torch.equal(y, r) for y, r in zip(ys, refs))


@pytest.mark.parametrize("T,K,N,dt", [(700, 8192, 1100, BF), (3000, 2056, 2100, BF), (257, 2056, 1003, F32),
                                      (2600, 264, 4000, F32)])
def test_equal_tokens_get_equal_bits(T, K, N, dt):
    c = _case(T, K, N, dt, 15)
    for k in ("x", "residual", "dy"):
        c[k] = c[k][:1].expand(T, -1).contiguous()
    y, z = _fwd(c, "gelu")
    assert torch.equal(y, y[:1].expand(T, -1)) and torch.equal(z, z[:1].expand(T, -1))
    dx, _, _ = _bwd(c, z.cpu(), "gelu")
    assert torch.equal(dx, dx[:1].expand(T, -1))
