"""Failure detection of the sub-layer operators, without a GPU fault: mhc_debug_sublayer_stop_after
makes their kernels stop loading at a stage boundary, so everything loaded before completes and the
waits for the rest run into a short limit.  The status word reports it, the context stays usable, and
the next normal call is right."""
import pytest

torch = pytest.importorskip("torch")
mhc = pytest.importorskip("mhc_hyper_connections_b200")

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture
def restore_hook():
    yield
    mhc.mhc_debug_sublayer_stop_after(-1, 1_000_000)


def _workspace(n):
    return torch.empty(max(n, 1), dtype=torch.uint8, device="cuda")


def _linear(T, K, N, dt):
    g = torch.Generator(device="cuda").manual_seed(T + K + N)
    x = torch.randn(T, K, generator=g, device="cuda").to(dt)
    W = (torch.randn(N, K, generator=g, device="cuda") / K ** 0.5).to(dt)
    ws = _workspace(mhc.mhc_linear_workspace_bytes(T, K, N, dt))

    def call():
        y = torch.zeros(T, N, dtype=dt, device="cuda")
        mhc.mhc_linear(x, W, None, y, workspace=ws)
        return (y,)
    return call


def _backward(T, K, N, dt):
    g = torch.Generator(device="cuda").manual_seed(T + K + N)
    x, W, dy = (torch.randn(*s, generator=g, device="cuda").to(dt) for s in ((T, K), (N, K), (T, N)))
    ws = _workspace(mhc.mhc_linear_backward_workspace_bytes(T, K, N, dt))

    def call():
        dx, dW = torch.zeros_like(x), torch.zeros_like(W)
        mhc.mhc_linear_backward(x, W, None, dy, dx, dW, None, ws)
        return dx, dW
    return call


def _norm(T, d, dt, backward):
    g = torch.Generator(device="cuda").manual_seed(T + d)
    x, dy = (torch.randn(T, d, generator=g, device="cuda").to(dt) for _ in range(2))
    w = torch.randn(d, generator=g, device="cuda")
    mean, rstd = x.float().mean(1), torch.ones(T, device="cuda")
    ws = _workspace(mhc.mhc_layer_norm_backward_workspace_bytes(T, d))

    def call():
        out = torch.zeros_like(x)
        if backward:
            dw, db = torch.zeros_like(w), torch.zeros_like(w)
            mhc.mhc_layer_norm_backward(x, w, mean, rstd, dy, out, dw, db, ws)
            return out, dw, db
        mhc.mhc_layer_norm(x, w, None, 1e-5, out)
        return (out,)
    return call


# kernels: pair 256 and 128 wide, split (narrow and wide, one CTA and a cluster), fp32 parts, and their
# layouts; layer norm by warp, by groups of lanes and by block.  Each has more stages than the stop.
CASES = {
    "pair256": lambda: _linear(4096, 1024, 4096, BF), "pair128": lambda: _linear(512, 1024, 1024, BF),
    "split16": lambda: _linear(3, 4096, 8192, BF), "split64": lambda: _linear(50, 4096, 1024, BF),
    "split128": lambda: _linear(100, 8192, 1024, BF), "f32": lambda: _linear(300, 2048, 2048, F32),
    "backward": lambda: _backward(2048, 1024, 2048, BF), "backward_f32": lambda: _backward(512, 2048, 1024, F32),
    "norm_warp": lambda: _norm(20000, 1024, BF, False), "norm_lanes": lambda: _norm(200000, 64, BF, False),
    "norm_block": lambda: _norm(6000, 4096, F32, False), "norm_backward_block": lambda: _norm(8000, 2560, BF, True),
    "norm_backward_lanes": lambda: _norm(200000, 64, BF, True),
}


@pytest.mark.parametrize("name", CASES)
def test_expired_waits_are_reported_and_the_next_call_is_clean(name, restore_hook):
    call = CASES[name]()
    good = call()
    torch.cuda.synchronize()
    assert mhc.mhc_device_status() == 0
    mhc.mhc_debug_sublayer_stop_after(2, 20_000)       # 2 stages, 20 ms waits
    call()
    torch.cuda.synchronize()                            # the kernels returned: the context is usable
    assert mhc.mhc_device_status() >> 29 != 0
    assert mhc.mhc_device_status() == 0                 # read-and-clear
    mhc.mhc_debug_sublayer_stop_after(-1, 1_000_000)
    assert all(torch.equal(a, b) for a, b in zip(call(), good))
    assert mhc.mhc_device_status() == 0


@pytest.mark.parametrize("name", ["pair256", "split64", "f32", "norm_warp", "norm_backward_block"])
def test_a_stop_past_the_last_stage_changes_nothing(name, restore_hook):
    call = CASES[name]()
    good = call()
    mhc.mhc_debug_sublayer_stop_after(1_000_000, 20_000)
    assert all(torch.equal(a, b) for a, b in zip(call(), good))
    assert mhc.mhc_device_status() == 0
