"""What is timed of the sub-layer operators: layer norm and the linear product with its
epilogue, forward and backward.

An mHC layer wraps a sub-layer F: pre gives x_in, F maps it, post merges F_out.  A feed-forward
F is a layer norm, an up projection with an activation and a down projection, so these four
calls are what a program runs between mhc_pre and mhc_post, and between mhc_backward's
dF_out and dx_in on the way back:

    layer_norm           y = (x - mean) rstd * weight + bias, and mean, rstd
    layer_norm_backward  dx, dweight, dbias
    linear               y = act(x W^T + bias) + residual, and z = x W^T + bias for training
    linear_backward      dx = dz W, dW = dz^T x, dbias = sum_t dz, with dz = dy act'(z)

``own`` chooses who computes in ``run``: plain torch operations in 32 bits (False), or the
package's calls on buffers that the caller keeps (True).  Activations and W are bf16 or fp32;
layer norm's parameters, biases and their gradients are fp32.
"""
import math

import torch

own = False

EPS = 1e-5
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")


def _ln(name, T, d, dt, train):
    return dict(name=name, op="layer_norm", T=T, d=d, dt=dt, train=train)


def _lnb(name, T, d, dt):
    return dict(name=name, op="layer_norm_backward", T=T, d=d, dt=dt)


def _lin(name, T, K, N, dt, act, residual, train):
    return dict(name=name, op="linear", T=T, K=K, N=N, dt=dt, act=act, residual=residual, train=train)


def _linb(name, T, K, N, dt, act):
    return dict(name=name, op="linear_backward", T=T, K=K, N=N, dt=dt, act=act)


def listed():
    return [
        # one token while generating: latency
        _ln("norm_one_token_d4096_bf16", 1, 4096, "bf16", False),
        # the headline batch of this repository's benchmark, in training
        _ln("norm_T16384_d4096_bf16_train", 16384, 4096, "bf16", True),
        # the backward at the other benchmark width
        _lnb("norm_backward_T16384_d2560_bf16", 16384, 2560, "bf16"),
        # a ragged fp32 batch with an odd width
        _lnb("norm_backward_T1001_d1037_f32", 1001, 1037, "f32"),
        # up projection of one generated token: the weights' bytes count
        _lin("linear_one_token_4096_to_16384_bf16_gelu", 1, 4096, 16384, "bf16", "gelu", False, False),
        # a few sequences generating together, down projection with a residual
        _lin("linear_T48_16384_to_4096_bf16_residual", 48, 16384, 4096, "bf16", "none", True, False),
        # a ragged prompt through odd widths
        _lin("linear_T777_1027_to_2565_bf16_silu", 777, 1027, 2565, "bf16", "silu", True, False),
        # training, up projection, the pre-activation kept
        _lin("linear_T16384_4096_to_16384_bf16_gelu_train", 16384, 4096, 16384, "bf16", "gelu", False, True),
        # training, down projection at d = 2560
        _lin("linear_T8192_10240_to_2560_bf16", 8192, 10240, 2560, "bf16", "none", False, False),
        # fp32 storage, the width of the small fp32 workload's streams side by side
        _lin("linear_T64_256_to_1024_f32_relu", 64, 256, 1024, "f32", "relu", False, True),
        # backward of the up projection at d = 1024
        _linb("linear_backward_T4096_1024_to_4096_bf16_gelu_tanh", 4096, 1024, 4096, "bf16", "gelu_tanh"),
        # backward of the up projection at the headline batch
        _linb("linear_backward_T16384_4096_to_16384_bf16_gelu", 16384, 4096, 16384, "bf16", "gelu"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("layer_norm", "layer_norm_backward", "linear", "linear_backward"))
    dt = rng.choice(("bf16", "bf16", "bf16", "f32"))
    T = _log(rng, 1, 16384)
    if op.startswith("layer_norm"):
        d = _log(rng, 64, 8192)
        if rng.random() < 0.6:
            d = (d + 63) // 64 * 64
        if T * d > 1 << 26:
            T = (1 << 26) // d
        if op == "layer_norm":
            return dict(op=op, T=T, d=d, dt=dt, train=rng.random() < 0.5)
        return dict(op=op, T=T, d=d, dt=dt)
    K, N = _log(rng, 64, 16384), _log(rng, 64, 16384)
    if rng.random() < 0.7:
        K, N = (K + 63) // 64 * 64, (N + 63) // 64 * 64
    # fp32 cases stay a quarter of the largest
    cap = 1 << 40 if dt == "bf16" else 1 << 38
    if T * K * N > cap:
        T = max(1, cap // (K * N))
    act = rng.choice(ACTS)
    if op == "linear":
        return dict(op=op, T=T, K=K, N=N, dt=dt, act=act, residual=rng.random() < 0.5, train=rng.random() < 0.5)
    return dict(op=op, T=T, K=K, N=N, dt=dt, act=act)


# ---- inputs

def _inputs(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt = DTYPES[case["dt"]]

    def normal(*shape, scale=1.0, dtype=torch.float32):
        # drawn in the storage type's own rows at most 2^27 at a time, to keep fp32 copies small
        out = torch.empty(shape, device="cuda", dtype=dtype)
        flat = out.view(-1)
        for i in range(0, flat.numel(), 1 << 27):
            part = flat[i:i + (1 << 27)]
            part.copy_(torch.randn(part.shape, generator=g, device="cuda").mul_(scale))
        return out

    def activations(T, d):
        # N(0, 1) with a common offset and one channel in a hundred 20 times as large, as the
        # streams of this repository's workloads have
        x = normal(T, d, dtype=dt)
        k = max(1, d // 100)
        cols = torch.randperm(d, generator=g, device="cuda")[:k]
        x[:, cols] = (x[:, cols].float() * 20.0 + 0.5).to(dt)
        return x

    T = case["T"]
    s = {}
    if case["op"].startswith("layer_norm"):
        d = case["d"]
        s["x"] = activations(T, d)
        s["weight"] = 1.0 + normal(d, scale=0.1)
        s["bias"] = normal(d, scale=0.1)
        if case["op"] == "layer_norm_backward":
            s["dy"] = normal(T, d, scale=0.02, dtype=dt)
            # mean and rstd as the forward saved them
            xd = s["x"].double()
            mean = xd.mean(dim=1)
            rstd = ((xd * xd).mean(dim=1) - mean * mean + EPS).rsqrt()
            s["mean"], s["rstd"] = mean.float(), rstd.float()
        return s
    K, N = case["K"], case["N"]
    s["W"] = normal(N, K, scale=K ** -0.5, dtype=dt)
    # normalised activations reach a projection without the outlier channels' factor
    s["x"] = normal(T, K, dtype=dt)
    if case["op"] == "linear":
        s["bias"] = normal(N, scale=0.1)
        s["residual"] = normal(T, N, dtype=dt) if case["residual"] else None
    else:
        # x W^T + bias of such inputs is N(0, 1)
        s["z"] = normal(T, N, dtype=dt) if case["act"] != "none" else None
        s["dy"] = normal(T, N, scale=0.02, dtype=dt)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    if not own:
        return s
    import mhc_hyper_connections_b200 as mhc
    T, dev, dt = case["T"], "cuda", DTYPES[case["dt"]]
    if case["op"] == "layer_norm":
        s["y"] = torch.empty_like(s["x"])
        s["mean"] = torch.empty(T, device=dev) if case["train"] else None
        s["rstd"] = torch.empty(T, device=dev) if case["train"] else None
    elif case["op"] == "layer_norm_backward":
        d = case["d"]
        s["dx"] = torch.empty_like(s["x"])
        s["dweight"], s["dbias"] = torch.empty(d, device=dev), torch.empty(d, device=dev)
        s["ws"] = torch.empty(mhc.mhc_layer_norm_backward_workspace_bytes(T, d), dtype=torch.uint8, device=dev)
    elif case["op"] == "linear":
        s["y"] = torch.empty(T, case["N"], dtype=dt, device=dev)
        s["z"] = torch.empty_like(s["y"]) if case["train"] else None
        s["act"] = getattr(mhc, "ACT_" + case["act"].upper())
        s["ws"] = torch.empty(mhc.mhc_linear_workspace_bytes(T, case["K"], case["N"], dt), dtype=torch.uint8,
                              device=dev)
    else:
        s["dx"], s["dW"] = torch.empty_like(s["x"]), torch.empty_like(s["W"])
        s["dbias"] = torch.empty(case["N"], device=dev)
        s["act"] = getattr(mhc, "ACT_" + case["act"].upper())
        s["ws"] = torch.empty(mhc.mhc_linear_backward_workspace_bytes(T, case["K"], case["N"], dt),
                              dtype=torch.uint8, device=dev)
    return s


# ---- the plain forms, in 32 bits

def _act(z, act):
    if act == "none":
        return z
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    return z / (1.0 + torch.exp(-z))


def _act_grad(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "gelu":
        cdf = 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5)))
        return cdf + z * torch.exp(-0.5 * z * z) * (1.0 / math.sqrt(2.0 * math.pi))
    if act == "gelu_tanh":
        c = math.sqrt(2.0 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z * z * z))
        return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * c * (1.0 + 3.0 * 0.044715 * z * z)
    s = 1.0 / (1.0 + torch.exp(-z))
    return s * (1.0 + z * (1.0 - s))


def _plain(s):
    case = s["case"]
    dt = DTYPES[case["dt"]]
    x = s["x"].float()
    if case["op"] == "layer_norm":
        mean = x.mean(dim=1, keepdim=True)
        c = x - mean
        rstd = 1.0 / torch.sqrt((c * c).mean(dim=1, keepdim=True) + EPS)
        y = (c * rstd * s["weight"] + s["bias"]).to(dt)
        return (y, mean[:, 0], rstd[:, 0]) if case["train"] else y
    if case["op"] == "layer_norm_backward":
        rstd = s["rstd"][:, None]
        xh = (x - s["mean"][:, None]) * rstd
        dy = s["dy"].float()
        g = dy * s["weight"]
        dx = rstd * (g - g.mean(dim=1, keepdim=True) - xh * (g * xh).mean(dim=1, keepdim=True))
        return dx.to(dt), (dy * xh).sum(dim=0), dy.sum(dim=0)
    W = s["W"].float()
    if case["op"] == "linear":
        z = x @ W.t() + s["bias"]
        y = _act(z, case["act"])
        if s["residual"] is not None:
            y = y + s["residual"].float()
        return (y.to(dt), z.to(dt)) if case["train"] else y.to(dt)
    dz = s["dy"].float()
    if case["act"] != "none":
        dz = dz * _act_grad(s["z"].float(), case["act"])
    return (dz @ W).to(dt), (dz.t() @ x).to(dt), dz.sum(dim=0)


def run(state):
    if not own:
        return _plain(state)
    import mhc_hyper_connections_b200 as mhc
    s, case = state, state["case"]
    if case["op"] == "layer_norm":
        mhc.mhc_layer_norm(s["x"], s["weight"], s["bias"], EPS, s["y"], s["mean"], s["rstd"])
        return (s["y"], s["mean"], s["rstd"]) if case["train"] else s["y"]
    if case["op"] == "layer_norm_backward":
        mhc.mhc_layer_norm_backward(s["x"], s["weight"], s["mean"], s["rstd"], s["dy"], s["dx"], s["dweight"],
                                    s["dbias"], s["ws"])
        return s["dx"], s["dweight"], s["dbias"]
    if case["op"] == "linear":
        mhc.mhc_linear(s["x"], s["W"], s["bias"], s["y"], act=s["act"], residual=s["residual"], z=s["z"],
                       workspace=s["ws"])
        return (s["y"], s["z"]) if case["train"] else s["y"]
    mhc.mhc_linear_backward(s["x"], s["W"], s["z"], s["dy"], s["dx"], s["dW"], s["dbias"], s["ws"], act=s["act"])
    return s["dx"], s["dW"], s["dbias"]


# ---- what one pass cannot do without

def work(case):
    es = 2 if case["dt"] == "bf16" else 4
    T = case["T"]
    if case["op"] == "layer_norm":
        d = case["d"]
        return {"bytes": 2 * T * d * es + 8 * d + (8 * T if case["train"] else 0), "flops": 8 * T * d}
    if case["op"] == "layer_norm_backward":
        d = case["d"]
        return {"bytes": 3 * T * d * es + 12 * d + 8 * T, "flops": 16 * T * d}
    K, N = case["K"], case["N"]
    if case["op"] == "linear":
        rows = 1 + int(case["residual"]) + int(case["train"])
        return {"bytes": (T * K + N * K + rows * T * N) * es + 4 * N, "flops": 2 * T * K * N}
    rows = 1 if case["act"] == "none" else 2
    return {"bytes": (2 * T * K + 2 * N * K + rows * T * N) * es + 4 * N, "flops": 4 * T * K * N}


# ---- the definitions in 64 bits

def exact(case, seed):
    s = _inputs(case, seed)
    d64 = {k: v.double() for k, v in s.items() if v is not None}
    del s
    if case["op"] == "layer_norm":
        x, w, b = d64["x"], d64["weight"], d64["bias"]
        var, mean = torch.var_mean(x, dim=1, correction=0)
        rstd = (var + EPS).pow(-0.5)
        y = x.sub(mean.unsqueeze(1)).mul_(rstd.unsqueeze(1)).mul_(w).add_(b)
        return (y, mean, rstd) if case["train"] else y
    if case["op"] == "layer_norm_backward":
        x, w, mean, rstd, dy = (d64[k] for k in ("x", "weight", "mean", "rstd", "dy"))
        d = x.shape[1]
        xh = x.sub(mean.unsqueeze(1)).mul_(rstd.unsqueeze(1))
        dweight = torch.einsum("td,td->d", dy, xh)
        dbias = dy.sum(0)
        a = torch.mv(dy, w) / d
        c = torch.einsum("td,td,d->t", dy, xh, w) / d
        dx = dy.mul(w).sub_(a.unsqueeze(1)).sub_(xh.mul(c.unsqueeze(1))).mul_(rstd.unsqueeze(1))
        return dx, dweight, dbias
    act = case["act"]

    def value_and_slope(z):
        if act == "none":
            return z, torch.ones_like(z)
        if act == "relu":
            return z.clamp_min(0.0), torch.sign(z).clamp_min(0.0)
        if act == "gelu":        # z Phi(z), and Phi(z) + z phi(z)
            cdf = torch.special.ndtr(z)
            return z * cdf, cdf + z * torch.exp(z.square() * -0.5) / math.sqrt(2 * math.pi)
        if act == "silu":
            sg = torch.sigmoid(z)
            return z * sg, sg + z * sg * torch.sigmoid(-z)
        # gelu_tanh: (1 + tanh u) / 2 = sigmoid(2 u)
        u2 = math.sqrt(8.0 / math.pi) * (z + 0.044715 * z.pow(3))
        sg = torch.sigmoid(u2)
        return z * sg, sg + z * sg * torch.sigmoid(-u2) * math.sqrt(8.0 / math.pi) * (1 + 0.134145 * z.square())

    if case["op"] == "linear":
        z = torch.addmm(d64["bias"], d64["x"], d64["W"].T)
        y = value_and_slope(z)[0]
        if "residual" in d64:
            y = y + d64["residual"]
        return (y, z) if case["train"] else y
    dz = d64["dy"]
    if act != "none":
        dz = dz.mul_(value_and_slope(d64.pop("z"))[1])
    return torch.mm(dz, d64["W"]), torch.mm(dz.T, d64["x"]), torch.einsum("tn->n", dz)
