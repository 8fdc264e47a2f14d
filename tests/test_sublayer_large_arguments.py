"""Arguments of the sub-layer operators that do not fit the C ABI's integers are refused, not cut down to ones
that do.  Runs without a GPU: meta tensors have shapes and no memory."""
import pytest

import mhc_hyper_connections_b200 as mhc

torch = pytest.importorskip("torch")

BF16, F32 = torch.bfloat16, torch.float32
BIG = 1 << 32


def _m(*shape, dtype=BF16):
    return torch.empty(*shape, dtype=dtype, device="meta")


f = lambda *s: _m(*s, dtype=F32)


def test_workspace_queries():
    assert mhc.mhc_linear_workspace_bytes(64, 1030, 64, BF16) > 0
    for T, K, N, dt in ((64, BIG + 1030, 64, BF16), (64, 1030, BIG + 64, BF16), (2 * BIG * BIG + 64, 1030, 64, BF16),
                        (64, 1030 - BIG, 64, BF16), (64, 1030, 64, BIG + 1)):
        assert mhc.mhc_linear_workspace_bytes(T, K, N, dt) == 0
        assert mhc.mhc_linear_backward_workspace_bytes(T, K, N, dt) == 0
    assert mhc.mhc_layer_norm_backward_workspace_bytes(4, 64) > 0
    for T, d in ((4, BIG + 64), (4, 64 - BIG), (2 * BIG * BIG + 4, 64)):
        assert mhc.mhc_layer_norm_backward_workspace_bytes(T, d) == 0


def test_layer_norm_of_rows_past_the_largest():
    d = BIG + 64
    with pytest.raises(mhc.MhcError, match="past the library's largest") as e:
        mhc.mhc_layer_norm(_m(1, d), f(d), f(d), 1e-5, _m(1, d))
    assert e.value.status == 2
    with pytest.raises(mhc.MhcError, match="x has shape"):
        mhc.mhc_layer_norm_backward(_m(1, d), f(d), f(1), f(1), _m(1, d), _m(1, d), f(d), f(d))


@pytest.mark.parametrize("K,N,name", [(BIG + 8, 8, "x"), (8, BIG + 8, "W")])
def test_linear_of_widths_past_the_largest(K, N, name):
    with pytest.raises(mhc.MhcError, match=f"{name} has shape"):
        mhc.mhc_linear(_m(1, K), _m(N, K), f(N), _m(1, N))
    with pytest.raises(mhc.MhcError, match=f"{name} has shape"):
        mhc.mhc_linear_backward(_m(1, K), _m(N, K), None, _m(1, N), _m(1, K), _m(N, K), f(N), None)


def test_many_tokens_are_not_past_the_largest():
    with pytest.raises(ValueError, match="must be a CUDA tensor"):
        mhc.mhc_linear(_m(BIG, 8), _m(8, 8), f(8), _m(BIG, 8))


def test_activations_past_the_largest(monkeypatch):
    # the value that reaches the C ABI, which refuses it
    assert [mhc._act(a) for a in range(5)] == [0, 1, 2, 3, 4]
    assert {mhc._act(a) for a in (5, -1, BIG, BIG + 2, -BIG)} == {-1}
    assert mhc.load_library().mhc_linear(1 << 20, 1 << 24, 0, 0, 1, 8, 8, mhc._act(BIG), 1, 1 << 28, 0, 0, 0, 0) == 5
