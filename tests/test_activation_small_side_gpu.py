"""The activations far on their small side, where the result is a normal number but a factor of it is not:
values of mhc_linear with x = 0, so that z is the bias."""
import math

import pytest

from _sublayer import U, check

torch = pytest.importorskip("torch")
mhc = pytest.importorskip("mhc_hyper_connections_b200")

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
TINY = 2.0 ** -126                     # below it a value may come out as 0


def _value64(z, name):
    """In 64 bits, with the small side as a quotient of small numbers: 1 + tanh(u) cancels there."""
    if name == "gelu":
        return 0.5 * z * torch.special.erfc(-z / math.sqrt(2.0))
    u = z if name == "silu" else 2 * math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3)
    e = torch.exp(-u.abs())
    return z * torch.where(u < 0, e, torch.ones_like(e)) / (1 + e)


def _exponent_error(z, name):
    """Roundings of the exponential's argument: v, formed in k steps, turns into k u |v| of the value."""
    if name == "gelu":
        return 4 * (z * z / 2 + 1) * U                # z / sqrt 2 with two, or z z / 2 with two, and log2(e)'s
    if name == "silu":
        return 2 * z.abs() * U                        # the product with log2(e), and that constant's own
    u = 2 * math.sqrt(2.0 / math.pi) * (z.abs() + 0.044715 * z.abs() ** 3)
    return 8 * u * U                                  # and the cubic's five


@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("name", ["gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("T", [3, 100, 300])      # the kernels of few, more and many tokens
def test_values_keep_their_relative_accuracy(name, dt, T):
    z = torch.linspace(-95, 10, 4096)
    x, W = torch.zeros(T, 64, dtype=dt, device="cuda"), torch.zeros(z.numel(), 64, dtype=dt, device="cuda")
    y = torch.empty(T, z.numel(), dtype=dt, device="cuda")
    ws = torch.empty(max(1, mhc.mhc_linear_workspace_bytes(T, 64, z.numel(), dt)), dtype=torch.uint8, device="cuda")
    mhc.mhc_linear(x, W, z.cuda(), y, act=getattr(mhc, "ACT_" + name.upper()), workspace=ws)
    zd = z.double()
    ref = _value64(zd, name)
    # 16 u for the library functions and products, or 2^-20 for the short form's (ex2 and 1/x to 2^-22, the
    # fitted polynomial to 2^-19.8); the storage's half step; results below the normal numbers flushed
    own = (16 * U if dt == F32 else 2.0 ** -19) + _exponent_error(zd, name)
    half = 2.0 ** -8 if dt == BF else U
    tol = ref.abs() * (own + half) + TINY * (ref.abs() < TINY) + 2.0 ** -149
    check(y, ref.expand(T, -1), tol.expand(T, -1), name)


@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "f32"])
def test_ends_of_the_range(dt):
    z = torch.tensor([0.0, -0.0, 1e30, -1e30, 3e38, -3e38, float("inf"), float("nan")])
    x, W = torch.zeros(2, 8, dtype=dt, device="cuda"), torch.zeros(8, 8, dtype=dt, device="cuda")
    y = torch.empty(2, 8, dtype=dt, device="cuda")
    ws = torch.empty(max(1, mhc.mhc_linear_workspace_bytes(2, 8, 8, dt)), dtype=torch.uint8, device="cuda")
    for name in ("gelu", "gelu_tanh", "silu"):
        mhc.mhc_linear(x, W, z.cuda(), y, act=getattr(mhc, "ACT_" + name.upper()), workspace=ws)
        got = y[0].float().cpu()
        want = torch.tensor([0.0, 0.0, 1e30, 0.0, 3e38, 0.0, float("inf"), float("nan")]).to(dt).float()
        assert torch.equal(torch.isnan(got), torch.isnan(want)), name
        assert torch.equal(got[:-1], want[:-1]), name
