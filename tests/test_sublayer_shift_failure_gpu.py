"""The failure path of the layer norm kernels for rows that are not a multiple of 16 bytes: as
test_sublayer_failure_gpu.py does for the others, their bounded waits are made to run out."""
import pytest

from test_sublayer_failure_gpu import _norm, restore_hook  # noqa: F401

torch = pytest.importorskip("torch")
mhc = pytest.importorskip("mhc_hyper_connections_b200")

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32

# more rows per warp (forward) or block (backward) than the stop; the longest bf16 rows that these kernels take
CASES = [(T, d, dt, backward) for T, d, dt in ((20000, 1037, BF), (20000, 515, F32), (9000, 2563, BF))
         for backward in (False, True)] + [(20000, 8191, BF, False), (20000, 8177, BF, True)]


@pytest.mark.parametrize("T,d,dt,backward", CASES)
def test_expired_waits_are_reported_and_the_next_call_is_clean(T, d, dt, backward, restore_hook):  # noqa: F811
    call = _norm(T, d, dt, backward)
    good = call()
    torch.cuda.synchronize()
    assert mhc.mhc_device_status() == 0
    mhc.mhc_debug_sublayer_stop_after(1, 20_000)       # 1 row or batch, 20 ms waits
    call()
    torch.cuda.synchronize()                            # the kernels returned: the context is usable
    assert mhc.mhc_device_status() >> 29 != 0
    assert mhc.mhc_device_status() == 0
    mhc.mhc_debug_sublayer_stop_after(-1, 1_000_000)
    assert all(torch.equal(a, b) for a, b in zip(call(), good))
    mhc.mhc_debug_sublayer_stop_after(1_000_000, 20_000)
    assert all(torch.equal(a, b) for a, b in zip(call(), good))
    assert mhc.mhc_device_status() == 0
