"""A feed-forward layer wrapped by mHC, forward and backward, as a program runs it:

    mhc_pre_train -> mhc_layer_norm -> mhc_linear (activation) -> mhc_linear -> mhc_post
    mhc_backward (for dF_out) -> mhc_linear_backward x 2 -> mhc_layer_norm_backward -> mhc_backward

against 64-bit torch with autograd over the whole layer.  Every stored tensor adds one rounding of at
most half a step, h relative (rms h / sqrt(3)); about twelve lie on the longest path (x_in, the norm,
z and the activation, F_out, X'; dF_out, dz twice, dh, dx_norm, dx_in, dX), and a step of the layer
amplifies a relative error of its input by at most about 3 (the norm with its weights, the activation's
slope, sums of H).  So outputs and gradients have to agree to an rms of 3 sqrt(12) h / sqrt(3) = 6 h
relative; for fp32 storage, fp32 arithmetic takes h's place with K u-sized sums: 64 u."""
import math

import pytest

from mhc_hyper_connections_b200 import workloads as wl

from _parity import torch_inputs
from _sublayer import HALF, U

torch = pytest.importorskip("torch")
mhc = pytest.importorskip("mhc_hyper_connections_b200")

pytestmark = pytest.mark.gpu
EPS = 1e-5


def _layer64(p, t_max, eps, alphas):
    """The layer in 64 bits: (X', x_in) from the leaves p."""
    X = p["X"]
    T, n, d = X.shape
    v = X.reshape(T, n * d)
    h = (v / torch.sqrt((v * v).mean(1, keepdim=True) + eps)) @ p["phi"]
    a_pre, a_post, a_res = alphas
    Hpre = torch.sigmoid(a_pre * h[:, :n] + p["b_pre"])
    M = torch.exp(a_res * h[:, n:n + n * n].reshape(T, n, n) + p["b_res"])
    for _ in range(t_max):
        M = M / M.sum(1, keepdim=True)
        M = M / M.sum(2, keepdim=True)
    Hpost = 2 * torch.sigmoid(a_post * h[:, n + n * n:] + p["b_post"])
    x_in = torch.einsum("ti,tic->tc", Hpre, X)
    mean = x_in.mean(1, keepdim=True)
    var = ((x_in - mean) ** 2).mean(1, keepdim=True)
    y = (x_in - mean) / torch.sqrt(var + EPS) * p["ln_w"] + p["ln_b"]
    z = y @ p["W1"].T + p["c1"]
    u = 0.5 * z * torch.special.erfc(-z / math.sqrt(2.0))
    F = u @ p["W2"].T + p["c2"]
    return torch.einsum("tij,tjc->tic", M, X) + torch.einsum("ti,tc->tic", Hpost, F)


@pytest.mark.parametrize("T,n,d,hidden,dt", [(200, 4, 128, 512, "bf16"), (67, 2, 72, 200, "bf16"), (1, 4, 256, 1024, "bf16"),
                                             (700, 4, 256, 1024, "bf16"), (50, 3, 64, 96, "f32"),
                                             (520, 4, 512, 2048, "f32")])
def test_feed_forward_layer(T, n, d, hidden, dt):
    w = wl.make_inputs(T=T, n=n, d=d, dtype=dt, seed=5 * T + d, alpha=0.3)
    t, s, m = torch_inputs(w), w.scalars(), w.m
    X, st = t["X"], t["X"].dtype
    g = torch.Generator().manual_seed(T)
    r = lambda *sh: torch.randn(*sh, generator=g)
    par = dict(ln_w=1 + 0.1 * r(d), ln_b=0.1 * r(d), W1=(r(hidden, d) / d ** 0.5).to(st), c1=0.1 * r(hidden),
               W2=(r(d, hidden) / hidden ** 0.5).to(st), c2=0.1 * r(d))
    dY = r(T, n, d).to(st)
    q = {k: v.cuda() for k, v in par.items()}
    dYc = dY.cuda()
    e = lambda *sh, dtype=torch.float32: torch.empty(*sh, dtype=dtype, device="cuda")
    ws = lambda b: torch.empty(max(int(b), 1), dtype=torch.uint8, device="cuda")
    sa = (s["alpha_pre"], s["alpha_post"], s["alpha_res"], s["eps"], s["t_max"])
    pre = (t["phi"], t["b_pre"], t["b_post"], t["b_res"], *sa)
    # forward
    x_in, H, h = e(T, d, dtype=st), e(T, m), e(T, m)
    mhc.mhc_pre_train(X, *pre, x_in, H, h)
    xn, mean, rstd = e(T, d, dtype=st), e(T), e(T)
    mhc.mhc_layer_norm(x_in, q["ln_w"], q["ln_b"], EPS, xn, mean, rstd)
    u, z, F = e(T, hidden, dtype=st), e(T, hidden, dtype=st), e(T, d, dtype=st)
    wf = ws(max(mhc.mhc_linear_workspace_bytes(T, d, hidden, st), mhc.mhc_linear_workspace_bytes(T, hidden, d, st)))
    mhc.mhc_linear(xn, q["W1"], q["c1"], u, act=mhc.ACT_GELU, z=z, workspace=wf)
    mhc.mhc_linear(u, q["W2"], q["c2"], F, workspace=wf)
    Y = torch.empty_like(X)
    mhc.mhc_post(X, F, H, Y)
    # backward: dF_out does not depend on dx_in, so a first call of mhc_backward gives it
    out = dict(dX=torch.empty_like(X), dF=torch.empty_like(F), dphi=e(n * d, m), db_pre=e(n), db_post=e(n),
               db_res=e(n, n), dalpha=e(3))
    wb = ws(mhc.mhc_backward_workspace_bytes(T, n, d))
    back = lambda dx: mhc.mhc_backward(X, F, *pre, H, h, dYc, dx, out["dX"], out["dF"], out["dphi"], out["db_pre"],
                                       out["db_post"], out["db_res"], out["dalpha"], wb)
    back(torch.zeros_like(x_in))
    du, dxn, dx_in = torch.empty_like(u), torch.empty_like(xn), torch.empty_like(x_in)
    grads = {k: torch.empty_like(v) for k, v in q.items()}
    wl_ = ws(max(mhc.mhc_linear_backward_workspace_bytes(T, d, hidden, st),
                 mhc.mhc_linear_backward_workspace_bytes(T, hidden, d, st)))
    mhc.mhc_linear_backward(u, q["W2"], None, out["dF"], du, grads["W2"], grads["c2"], wl_)
    mhc.mhc_linear_backward(xn, q["W1"], z, du, dxn, grads["W1"], grads["c1"], wl_, act=mhc.ACT_GELU)
    mhc.mhc_layer_norm_backward(x_in, q["ln_w"], mean, rstd, dxn, dx_in, grads["ln_w"], grads["ln_b"],
                                ws(mhc.mhc_layer_norm_backward_workspace_bytes(T, d)))
    back(dx_in)
    torch.cuda.synchronize()
    assert mhc.mhc_device_status() == 0
    # the whole layer in 64 bits
    p = {k: v.double().cpu().requires_grad_() for k, v in
         dict(X=X, phi=t["phi"], b_pre=t["b_pre"], b_post=t["b_post"], b_res=t["b_res"].reshape(n, n), **q).items()}
    ref = _layer64(p, s["t_max"], s["eps"], sa[:3])
    (ref * dY.double()).sum().backward()
    bound = 6 * HALF[torch.bfloat16] if st == torch.bfloat16 else 64 * U
    got = dict(Y=Y, X=out["dX"], phi=out["dphi"], b_pre=out["db_pre"], b_post=out["db_post"], b_res=out["db_res"], **grads)
    want = dict(Y=ref.detach(), **{k: p[k].grad for k in got if k != "Y"})
    for k in got:
        a, b = got[k].double().cpu(), want[k]
        err = float((a - b).norm() / b.norm())
        assert err <= bound, (k, err)
