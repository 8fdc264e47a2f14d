"""Sums so long that an accumulator takes longer than the limit of a single wait: the stages arrive in time, so
nothing has expired and the result is whole."""
import pytest

torch = pytest.importorskip("torch")
mhc = pytest.importorskip("mhc_hyper_connections_b200")

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture
def short_waits():
    # 5 ms per wait, where the sums below take 20 and more
    mhc.mhc_debug_sublayer_stop_after(-1, 5_000)
    yield
    mhc.mhc_debug_sublayer_stop_after(-1, 1_000_000)


@pytest.mark.parametrize("lg,K,N,dt", [(26, 8, 8, BF), (26, 8, 120, BF), (26, 120, 8, BF), (24, 8, 8, F32)])
def test_weight_gradient_of_many_tokens(lg, K, N, dt, short_waits):
    # sums of powers of two below 2^24 times their smallest term: exact in fp32 in any order
    T, every = 1 << lg, 1 << (lg - 16)
    x, dy = torch.zeros(T, K, dtype=dt, device="cuda"), torch.zeros(T, N, dtype=dt, device="cuda")
    x[::every] = torch.arange(1, K + 1, device="cuda").to(dt)
    dy[::every] = (torch.arange(N, device="cuda") % 4 - 1.5).to(dt)
    dW = torch.empty(N, K, dtype=dt, device="cuda")
    ws = torch.empty(mhc.mhc_linear_backward_workspace_bytes(T, K, N, dt), dtype=torch.uint8, device="cuda")
    mhc.mhc_linear_backward(x, torch.empty_like(dW), None, dy, None, dW, None, ws)
    assert mhc.mhc_device_status() == 0
    ref = (1 << 16) * (torch.arange(N) % 4 - 1.5)[:, None] * torch.arange(1, K + 1)[None, :]
    assert torch.equal(dW.cpu().float(), ref.to(dt).float())


def test_one_output_of_a_long_row(short_waits):
    K = 1 << 28
    x, W = torch.zeros(1, K, dtype=BF, device="cuda"), torch.zeros(3, K, dtype=BF, device="cuda")
    x[:, ::1 << 10] = 1.0
    W[:, ::1 << 10] = torch.tensor([1.0, -2.0, 0.5], device="cuda", dtype=BF)[:, None]
    y = torch.empty(1, 3, dtype=BF, device="cuda")
    ws = torch.empty(max(1, mhc.mhc_linear_workspace_bytes(1, K, 3, BF)), dtype=torch.uint8, device="cuda")
    mhc.mhc_linear(x, W, None, y, workspace=ws)
    assert mhc.mhc_device_status() == 0
    assert y.cpu().float().tolist() == [[2.0 ** 18, -2.0 ** 19, 2.0 ** 17]]
