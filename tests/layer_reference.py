"""Layer norm and the gated feed-forward block in fp64, with a bound on how far a
kernel's result may be from it.

Every bound is propagated through the operator step by step in absolute values:

* u = 2^-24: one fp32 rounding, relative.  A tensor-core sum may cut instead of
  round; that is one step, 2u, but it adds 16 products at a time, so (k + 16) u
  times the sum of absolute products covers a sum of k terms either way (fp32
  operands are split in three bf16 parts by cutting and take six passes: 6 k / 16
  additions of 2u each, 0.75 k u; the parts are below 2^-7 and 2^-15 of the whole, so the
  three products left out are below 2 2^-22 + 2^-30 = 8u of a product: inside the 16 u).
* GRID = 2^-133: bf16's smallest step.  The last of an fp32 operand's three bf16 parts is
  cut to it, so an operand is off by up to GRID absolutely: |x| = 3.3e38 against a weight
  of 1e-39 makes that 3.3e38 2^-133 = 0.03 of a product of 0.3, and nothing otherwise.
* r: the rounding of a stored value, half a step of its type: 2^-8 relative for
  bf16, u for fp32.
* the norm's row sums run over at most 32 values per thread in order, five
  exchanges per warp and five across warps: fewer than 64 roundings.
* SiLU and GELU change by at most 1.2 per unit of g and their derivatives by at
  most 0.8; a few roundings of the function itself are counted as ``fn``.
"""
import math

import torch

U = 2.0 ** -24
GRID = 2.0 ** -133
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: U}


# --------------------------------------------------------------------- norm
def norm(x, w, b, eps):
    x = x.double()
    m = x.mean(1, keepdim=True)
    s = 1 / torch.sqrt(((x - m) ** 2).mean(1, keepdim=True) + eps)
    y = (x - m) * s * w.double()
    return y if b is None else y + b.double()


def _norm_parts(x, eps):
    """mean, s, xh and a bound on xh's error."""
    g = 64 * U
    m = x.mean(1, keepdim=True)
    v = ((x - m) ** 2).mean(1, keepdim=True)
    s = 1 / torch.sqrt(v + eps)
    xh = (x - m) * s
    dm = g * x.abs().mean(1, keepdim=True)
    return m, s, xh, s * dm + (g + s * s * dm * dm) * xh.abs() + 4 * U * s * x.abs()


def norm_bound(x, w, b, eps, dtype):
    """Bound on |y - exact|."""
    x, w = x.double(), w.double()
    _, _, xh, dxh = _norm_parts(x, eps)
    y = xh * w
    ab = 0.0 if b is None else b.double().abs()
    d = w.abs() * dxh + 4 * U * (y.abs() + ab)
    return d + HALF_STEP[dtype] * ((y if b is None else y + b.double()).abs() + d)


def norm_grad(x, w, gy, eps):
    x, w, gy = x.double(), w.double(), gy.double()
    m = x.mean(1, keepdim=True)
    s = 1 / torch.sqrt(((x - m) ** 2).mean(1, keepdim=True) + eps)
    xh = (x - m) * s
    a = gy * w
    gx = s * (a - a.mean(1, keepdim=True) - xh * (a * xh).mean(1, keepdim=True))
    return gx, (gy * xh).sum(0), gy.sum(0)


def norm_grad_bound(x, w, gy, eps, dtype):
    """Bounds on grad_x, grad_weight, grad_bias."""
    T = x.shape[0]
    x, w, gy = x.double(), w.double(), gy.double()
    g = 64 * U
    _, s, xh, dxh = _norm_parts(x, eps)
    a = gy * w
    c1, c2 = a.mean(1, keepdim=True), (a * xh).mean(1, keepdim=True)
    dc1 = g * a.abs().mean(1, keepdim=True)
    dc2 = (g * (a * xh).abs() + a.abs() * dxh).mean(1, keepdim=True)
    terms = a.abs() + c1.abs() + (xh * c2).abs()
    d = s * (dc1 + xh.abs() * dc2 + c2.abs() * dxh + g * terms)
    gx = s * (a - c1 - xh * c2)
    d = d + HALF_STEP[dtype] * (gx.abs() + d)
    dw = (gy.abs() * dxh).sum(0) + (T + 16) * U * (gy * xh).abs().sum(0)
    return d, dw, (T + 16) * U * gy.abs().sum(0)


# ---------------------------------------------------------------------- ffn
def gate(g, act):
    """act(g), act'(g) in fp64."""
    if act == "silu":
        p = torch.sigmoid(g)
        return g * p, p * (1 + g * (1 - p))
    c = 0.5 * torch.erfc(-g / math.sqrt(2.0))
    return g * c, c + g * torch.exp(-0.5 * g * g) / math.sqrt(2 * math.pi)


def ffn(x, wg, wu, wd, act):
    x, wg, wu, wd = (t.double() for t in (x, wg, wu, wd))
    return (gate(x @ wg.T, act)[0] * (x @ wu.T)) @ wd.T


def ffn_grad(x, wg, wu, wd, gy, act):
    x, wg, wu, wd, gy = (t.double() for t in (x, wg, wu, wd, gy))
    g, u = x @ wg.T, x @ wu.T
    h, dh = gate(g, act)
    da = gy @ wd
    dg, du = da * u * dh, da * h
    return dg @ wg + du @ wu, dg.T @ x, du.T @ x, gy.T @ (h * u)


def _sum_err(a, b, dtype, terms=None):
    """Bound on the error of a kernel's a @ b, given a and b exactly; terms: the sum's length
    where it goes on beyond a and b."""
    a, b = a.abs(), b.abs()
    e = ((terms or a.shape[1]) + 16) * U * (a @ b)
    if dtype == torch.float32:
        e = e + GRID * (a.sum(1, keepdim=True) + b.sum(0, keepdim=True))
    return e


def _inner(x, wg, wu, act, dtype, store):
    """g, u, h, dh and bounds on them; store: g and u are kept in the call's type."""
    fn = 16 * U if dtype == torch.float32 else 2.0 ** -18
    r = HALF_STEP[dtype] if store else 0.0
    g, u = x @ wg.T, x @ wu.T
    dg = _sum_err(x, wg.T, dtype)
    du = _sum_err(x, wu.T, dtype)
    dg, du = dg + r * (g.abs() + dg), du + r * (u.abs() + du)
    h, dh = gate(g, act)
    eh = 1.2 * dg + fn * g.abs()
    edh = 0.8 * dg + fn * (1 + g.abs())
    return g, u, h, dh, du, eh, edh


def ffn_bound(x, wg, wu, wd, act, dtype):
    r = HALF_STEP[dtype]
    x, wg, wu, wd = (t.double() for t in (x, wg, wu, wd))
    g, u, h, _, eu, eh, _ = _inner(x, wg, wu, act, dtype, False)
    a = h * u
    ea = eh * (u.abs() + eu) + h.abs() * eu
    ea = ea + r * (a.abs() + ea) + 2 * U * a.abs()
    d = ea @ wd.abs().T + _sum_err(a, wd.T, dtype)
    return d + r * ((a @ wd.T).abs() + d)


def ffn_grad_bound(x, wg, wu, wd, gy, act, dtype):
    r = HALF_STEP[dtype]
    x, wg, wu, wd, gy = (t.double() for t in (x, wg, wu, wd, gy))
    F = wg.shape[0]
    # a may come from the unrounded or from the stored g and u: the larger bound
    g, u, h, dh, eu, eh, edh = _inner(x, wg, wu, act, dtype, True)
    a = h * u
    ea = eh * (u.abs() + eu) + h.abs() * eu
    ea = ea + (r + 2 * U) * (a.abs() + ea)
    da = gy @ wd
    eda = _sum_err(gy, wd, dtype)
    dg, du = da * u * dh, da * h
    edu = eda * (h.abs() + eh) + da.abs() * eh
    edu = edu + (r + 2 * U) * (du.abs() + edu)
    edg = eda * ((u.abs() + eu) * (dh.abs() + edh)) + da.abs() * (eu * (dh.abs() + edh)
                                                                  + u.abs() * edh)
    edg = edg + (r + 3 * U) * (dg.abs() + edg)
    ex = (edg @ wg.abs() + edu @ wu.abs() + _sum_err(dg, wg, dtype, 2 * F)
          + _sum_err(du, wu, dtype, 2 * F))
    egw = edg.T @ x.abs() + _sum_err(dg.T, x, dtype)
    euw = edu.T @ x.abs() + _sum_err(du.T, x, dtype)
    edw = gy.abs().T @ ea + _sum_err(gy.T, a, dtype)
    outs = (dg @ wg + du @ wu, dg.T @ x, du.T @ x, gy.T @ a)
    return tuple(e + r * (o.abs() + e) for e, o in zip((ex, egw, euw, edw), outs))


def assert_within(got, ref, bound, name):
    """Every element of got within its bound of ref (got in any dtype)."""
    got = got.detach().double().cpu()
    ref, bound = ref.cpu(), bound.cpu()
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    # a result below fp32's normal range may be flushed: 2^-126 absolute
    over = (got - ref).abs() - (bound + 2.0 ** -126)
    bad = ~(over <= 0)  # NaN counts
    if bad.any():
        i = int(torch.where(bad.flatten())[0][0])
        raise AssertionError(
            f"{name}: {int(bad.sum())} of {bad.numel()} elements out of bound, first at flat "
            f"index {i}: got {got.flatten()[i]:.9g}, ref {ref.flatten()[i]:.9g}, bound "
            f"{bound.flatten()[i]:.3g}")


def norm_rel(got, ref):
    """|got - ref| / |ref| in the 2-norm."""
    got, ref = got.detach().double().cpu(), ref.cpu()
    n = float(ref.norm())
    return float((got - ref).norm()) / n if n > 0 else float((got - ref).norm())
