"""The layer function's operators, as cases that can be timed and compared.

An mHC stack wraps a layer function F; the one these operators make is a layer
norm followed by a gated feed-forward block.  Both have a forward and a
backward pass:

    norm       y = (x - mean) / sqrt(var + eps) * weight + bias      per token
    norm_grad  grad_x, grad_weight, grad_bias of it, statistics recomputed
    ffn        y = (act(x w_gate^T) * (x w_up^T)) w_down^T
    ffn_grad   grad_x, grad_w_gate, grad_w_up, grad_w_down of it, with the two
               projections recomputed from x

``run`` computes them in plain fp32 torch where ``own`` is false and calls the
library where it is true; ``exact`` computes them in fp64, token block by token
block.  x, y and their gradients are [T, C] and the weights of the block [F, C]
and [C, F], of one type (bf16 or fp32); the norm's weight and bias and their
gradients are fp32.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6


def listed():
    """Twelve cases: each operator in each direction and both types, from one token to a
    training batch, at the channel counts of this repository's workloads."""
    return [
        # one token being generated: nothing but latency
        dict(name="norm_token", op="norm", T=1, C=7168, dtype="bf16", bias=True),
        # one layer's batch in training, the size of the benchmark's layer
        dict(name="norm_train", op="norm", T=16384, C=7168, dtype="bf16", bias=True),
        # a small model's gradient step: few rows, so latency and the reduction count
        dict(name="norm_grad_small", op="norm_grad", T=130, C=512, dtype="bf16", bias=True),
        # the training batch's gradient
        dict(name="norm_grad_train", op="norm_grad", T=16384, C=7168, dtype="bf16", bias=True),
        # fp32 activations, a row count and a width that no tile divides
        dict(name="norm_grad_f32", op="norm_grad", T=2049, C=4104, dtype="f32", bias=False),
        # one token being generated: the three weights are read once
        dict(name="ffn_token", op="ffn", T=1, C=7168, F=14336, dtype="bf16", act="silu"),
        # a batch of sequences being generated together, one token each
        dict(name="ffn_batch", op="ffn", T=48, C=4096, F=16384, dtype="bf16", act="silu"),
        # a prompt of odd length through a block of odd width
        dict(name="ffn_ragged", op="ffn", T=777, C=4096, F=10952, dtype="bf16", act="gelu"),
        # one layer's batch in training
        dict(name="ffn_train", op="ffn", T=8192, C=7168, F=14336, dtype="bf16", act="silu"),
        # a small model's gradient step
        dict(name="ffn_grad_small", op="ffn_grad", T=130, C=512, F=1368, dtype="bf16",
             act="silu"),
        # the training batch's gradient
        dict(name="ffn_grad_train", op="ffn_grad", T=8192, C=7168, F=14336, dtype="bf16",
             act="silu"),
        # fp32 activations and weights, odd sizes
        dict(name="ffn_grad_f32", op="ffn_grad", T=1023, C=1024, F=2728, dtype="f32",
             act="gelu"),
    ]


MOST = 8192 * 7168 * 14336      # T * C * F of the largest listed block
MOST_F32 = MOST // 16           # fp32 blocks of the same range, kept smaller


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _eights(rng, lo, hi):
    """A multiple of 8 in [lo, hi], spread over the logarithm."""
    return min(hi, max(lo, 8 * int(round(_log(rng, lo, hi) / 8))))


def draw(rng):
    """A case of the same ranges: 1 to 16384 tokens, 8 to 7168 channels, 8 to 16384 hidden
    units, both types, either activation, with and without a bias."""
    op = rng.choice(["norm", "norm_grad", "ffn", "ffn_grad", "ffn", "ffn_grad"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op.startswith("norm"):
        return dict(op=op, T=_log(rng, 1, 16384), C=_eights(rng, 8, 7168), dtype=dtype,
                    bias=rng.random() < 0.7)
    most = MOST if dtype == "bf16" else MOST_F32
    while True:
        case = dict(op=op, T=_log(rng, 1, 8192), C=_eights(rng, 64, 7168),
                    F=_eights(rng, 64, 16384), dtype=dtype, act=rng.choice(["silu", "gelu"]))
        if case["T"] * case["C"] * case["F"] <= most:
            return case


def work(case):
    """Bytes: every input read once, every output written once.  Operations: the matrix
    products (two per multiply-add), or about eight and sixteen per element of a norm."""
    T, C = case["T"], case["C"]
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "norm":
        return {"bytes": 2 * T * C * e + (8 if case["bias"] else 4) * C, "flops": 8 * T * C}
    if case["op"] == "norm_grad":
        return {"bytes": 3 * T * C * e + 12 * C, "flops": 16 * T * C}
    F = case["F"]
    if case["op"] == "ffn":
        return {"bytes": (2 * T * C + 3 * C * F) * e, "flops": 6 * T * C * F}
    return {"bytes": (3 * T * C + 6 * C * F) * e, "flops": 16 * T * C * F}


def prepare(case, seed):
    """Inputs of the layer function on the GPU: activations and gradients of unit variance
    (the norm's own rows with a mean and a scale of their own), weights at the usual
    1/sqrt(fan-in), a norm's gain around one."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    T, C = case["T"], case["C"]

    def normal(*shape, std=1.0, dtype=dt):
        t = torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)
        return t.mul_(std).to(dtype)

    s = dict(case=case)
    if case["op"].startswith("norm"):
        scale = torch.rand(T, 1, generator=g, device="cuda") * 2 + 0.5
        shift = torch.randn(T, 1, generator=g, device="cuda") * 0.5
        s["x"] = (normal(T, C, dtype=torch.float32) * scale + shift).to(dt)
        s["weight"] = 1 + normal(C, std=0.1, dtype=torch.float32)
        s["bias"] = normal(C, std=0.1, dtype=torch.float32) if case["bias"] else None
        if case["op"] == "norm_grad":
            s["grad_y"] = normal(T, C)
    else:
        F = case["F"]
        s["x"] = normal(T, C)
        s["w_gate"] = normal(F, C, std=C ** -0.5)
        s["w_up"] = normal(F, C, std=C ** -0.5)
        s["w_down"] = normal(C, F, std=F ** -0.5)
        if case["op"] == "ffn_grad":
            s["grad_y"] = normal(T, C)
    if own:
        import manifold_constrained_hyper_token_b200 as mhc
        s["mhc"] = mhc
        n = 0
        if case["op"] == "norm_grad":
            n = mhc.mhc_layer_norm_backward_workspace_size(T, C, dt)
        elif case["op"] == "ffn":
            n = mhc.mhc_ffn_workspace_size(T, C, case["F"], dt)
        elif case["op"] == "ffn_grad":
            n = mhc.mhc_ffn_backward_workspace_size(T, C, case["F"], dt)
        s["workspace"] = torch.empty(n, dtype=torch.uint8, device="cuda") if n else None
    return s


# ---------------------------------------------------------------- plain forms
def _act(g, name):
    if name == "silu":
        return g / (1 + torch.exp(-g))
    return 0.5 * g * (1 + torch.erf(g * 2 ** -0.5))


def _act_grad(g, name):
    if name == "silu":
        sg = 1 / (1 + torch.exp(-g))
        return sg * (1 + g * (1 - sg))
    return 0.5 * (1 + torch.erf(g * 2 ** -0.5)) + g * torch.exp(-0.5 * g * g) * (
        2 * math.pi) ** -0.5


def _plain_norm(s):
    x = s["x"].float()
    d = x - x.mean(1, keepdim=True)
    xh = d / torch.sqrt((d * d).mean(1, keepdim=True) + EPS)
    y = xh * s["weight"]
    if s["bias"] is not None:
        y = y + s["bias"]
    return y.to(s["x"].dtype)


def _plain_norm_grad(s):
    x, gy = s["x"].float(), s["grad_y"].float()
    d = x - x.mean(1, keepdim=True)
    r = 1 / torch.sqrt((d * d).mean(1, keepdim=True) + EPS)
    xh = d * r
    a = gy * s["weight"]
    gx = r * (a - a.mean(1, keepdim=True) - xh * (a * xh).mean(1, keepdim=True))
    return gx.to(s["x"].dtype), (gy * xh).sum(0), gy.sum(0)


def _plain_ffn(s):
    x, act = s["x"].float(), s["case"]["act"]
    a = _act(x @ s["w_gate"].float().T, act) * (x @ s["w_up"].float().T)
    return (a @ s["w_down"].float().T).to(s["x"].dtype)


def _plain_ffn_grad(s):
    x, gy, act = s["x"].float(), s["grad_y"].float(), s["case"]["act"]
    wg, wu, wd = s["w_gate"].float(), s["w_up"].float(), s["w_down"].float()
    g, u = x @ wg.T, x @ wu.T
    h = _act(g, act)
    da = gy @ wd
    du = da * h
    dg = da * u * _act_grad(g, act)
    dt = s["x"].dtype
    return ((dg @ wg + du @ wu).to(dt), (dg.T @ x).to(dt), (du.T @ x).to(dt),
            (gy.T @ (h * u)).to(dt))


PLAIN = dict(norm=_plain_norm, norm_grad=_plain_norm_grad, ffn=_plain_ffn,
             ffn_grad=_plain_ffn_grad)


def run(s):
    """One pass through the operator."""
    case = s["case"]
    op = case["op"]
    if not own:
        return PLAIN[op](s)
    mhc = s["mhc"]
    if op == "norm":
        return mhc.mhc_layer_norm(s["x"], s["weight"], s["bias"], eps=EPS)
    if op == "norm_grad":
        return mhc.mhc_layer_norm_backward(s["x"], s["weight"], s["grad_y"], eps=EPS,
                                           workspace=s["workspace"])
    if op == "ffn":
        return mhc.mhc_ffn(s["x"], s["w_gate"], s["w_up"], s["w_down"], act=case["act"],
                           workspace=s["workspace"])
    return mhc.mhc_ffn_backward(s["x"], s["w_gate"], s["w_up"], s["w_down"], s["grad_y"],
                                act=case["act"], workspace=s["workspace"])


# ------------------------------------------------------------------- in fp64
BLOCK = 2048


def _sigmoid64(g):
    # 1/(1 + e^-|g|) on either side of zero: no overflow
    e = torch.exp(-g.abs())
    return torch.where(g >= 0, 1 / (1 + e), e / (1 + e))


def _gate64(g, name):
    """act(g) and act'(g)."""
    if name == "silu":
        p = _sigmoid64(g)
        return g * p, p + g * p * (1 - p)
    cdf = torch.special.ndtr(g)
    pdf = torch.exp(g.square() / -2) / math.sqrt(2 * math.pi)
    return g * cdf, cdf + g * pdf


def exact(case, seed):
    """``run``'s outputs from the definition in fp64."""
    s = prepare(case, seed)
    T, C = case["T"], case["C"]
    if case["op"].startswith("norm"):
        w = s["weight"].double()
        rows, gw, gb = [], 0, 0
        for t in range(0, T, BLOCK):
            x = s["x"][t:t + BLOCK].double()
            var, mean = torch.var_mean(x, 1, correction=0, keepdim=True)
            r = (var + EPS).rsqrt()
            xh = (x - mean) * r
            if case["op"] == "norm":
                rows.append(xh * w + (s["bias"].double() if case["bias"] else 0))
                continue
            gy = s["grad_y"][t:t + BLOCK].double()
            a = gy * w
            rows.append((a - a.sum(1, keepdim=True) / C
                         - xh * ((a * xh).sum(1, keepdim=True) / C)) * r)
            gw = gw + torch.einsum("tc,tc->c", gy, xh)
            gb = gb + gy.sum(0)
        out = torch.cat(rows)
        return out if case["op"] == "norm" else (out, gw, gb)
    wg, wu, wd = (s[k].double() for k in ("w_gate", "w_up", "w_down"))
    rows = []
    if case["op"] == "ffn_grad":
        gwg, gwu, gwd = torch.zeros_like(wg), torch.zeros_like(wu), torch.zeros_like(wd)
    for t in range(0, T, BLOCK):
        x = s["x"][t:t + BLOCK].double()
        h, dh = _gate64(torch.matmul(x, wg.t()), case["act"])
        u = torch.matmul(x, wu.t())
        if case["op"] == "ffn":
            rows.append(torch.matmul(h * u, wd.t()))
            continue
        gy = s["grad_y"][t:t + BLOCK].double()
        da = torch.matmul(gy, wd)
        dg, du = da * (u * dh), da * h
        rows.append(torch.matmul(dg, wg) + torch.matmul(du, wu))
        gwg.addmm_(dg.t(), x)
        gwu.addmm_(du.t(), x)
        gwd.addmm_(gy.t(), h * u)
    return torch.cat(rows) if case["op"] == "ffn" else (torch.cat(rows), gwg, gwu, gwd)
