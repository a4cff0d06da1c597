"""The layer norm and feed-forward entry points without a GPU: their argument checks in
the C ABI and in the binding, and the fp64 formulas that the GPU tests compare against,
held to differences of the forward."""
import ctypes

import pytest
import torch

import layer_reference as R
from manifold_constrained_hyper_token_b200 import _lib, build

F32, BF16 = torch.float32, torch.bfloat16
FAKE = [ctypes.c_void_p(0x10000000 * (i + 1)) for i in range(12)]  # far apart, never followed
ODD = ctypes.c_void_p(0x10000004)
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


@pytest.fixture(scope="module")
def mhc():
    build.build()
    import manifold_constrained_hyper_token_b200 as m
    return m


def _np(**kw):
    d = dict(T=16, C=64, eps=1e-6, dtype=1)
    d.update(kw)
    return ctypes.byref(_lib.NormParams(**d))


def _fp(**kw):
    d = dict(T=16, C=64, F=96, dtype=1, act=0, wait_ns=0)
    d.update(kw)
    return ctypes.byref(_lib.FfnParams(**d))


def test_struct_layouts():
    assert ctypes.sizeof(_lib.NormParams) == 24 and _lib.NormParams.eps.offset == 16
    assert ctypes.sizeof(_lib.FfnParams) == 40 and _lib.FfnParams.wait_ns.offset == 32


BAD_NORM = [(dict(T=0), 1), (dict(T=-1), 1), (dict(T=2**31 - 256), 1), (dict(C=0), 1),
            (dict(C=12), 1), (dict(C=2**24 + 8), 1), (dict(eps=-1.0), 1),
            (dict(eps=float("nan")), 1), (dict(eps=float("inf")), 1), (dict(dtype=2), 2)]


@pytest.mark.parametrize("kw,code", BAD_NORM)
def test_norm_params_refused(lib, kw, code):
    p = _np(**kw)
    assert lib.mhc_layer_norm(p, FAKE[0], FAKE[1], FAKE[2], FAKE[3], None, None) == code
    assert lib.mhc_layer_norm_backward(p, *FAKE[:6], FAKE[6], BIG, None, None) == code
    assert lib.mhc_layer_norm_backward_workspace_size(p) == 0


BAD_FFN = [(dict(T=0), 1), (dict(T=2**31 - 256), 1), (dict(C=4), 1), (dict(C=60), 1),
           (dict(F=0), 1), (dict(F=36), 1), (dict(F=2**24 + 8), 1), (dict(wait_ns=-1), 1),
           (dict(dtype=9), 2), (dict(act=2), 2), (dict(act=-1), 2)]


@pytest.mark.parametrize("kw,code", BAD_FFN)
def test_ffn_params_refused(lib, kw, code):
    p = _fp(**kw)
    assert lib.mhc_ffn(p, *FAKE[:5], FAKE[5], BIG, None, None) == code
    assert lib.mhc_ffn_backward(p, *FAKE[:9], FAKE[9], BIG, None, None) == code
    assert lib.mhc_ffn_workspace_size(p) == 0
    assert lib.mhc_ffn_backward_workspace_size(p) == 0


def test_null_params_refused(lib):
    assert lib.mhc_layer_norm(None, *FAKE[:4], None, None) == 1
    assert lib.mhc_ffn(None, *FAKE[:5], FAKE[5], BIG, None, None) == 1


# which positions may be left out: the norm's bias and grad_bias
CALLS = {
    "mhc_layer_norm": (_np, 4, {2}, False, {3}),
    "mhc_layer_norm_backward": (_np, 6, {5}, True, {3, 4, 5}),
    "mhc_ffn": (_fp, 5, set(), True, {4}),
    "mhc_ffn_backward": (_fp, 9, set(), True, {5, 6, 7, 8}),
}


def _call(lib, name, ptrs, ws=FAKE[10], wsb=BIG):
    mk, _, _, has_ws, _ = CALLS[name]
    tail = (ws, wsb) if has_ws else ()
    return getattr(lib, name)(mk(), *ptrs, *tail, None, None)


@pytest.mark.parametrize("name", CALLS)
def test_null_misaligned_and_overlapping_arrays_refused(lib, name):
    _, k, optional, _, outs = CALLS[name]
    for i in range(k):
        ptrs = list(FAKE[:k])
        if i not in optional:
            ptrs[i] = None
            assert _call(lib, name, ptrs) == 1, (i, "null")
        ptrs[i] = ODD
        assert _call(lib, name, ptrs) == 1, (i, "misaligned")
    for o in outs:
        for i in range(k):
            if i != o:
                ptrs = list(FAKE[:k])
                ptrs[o] = ptrs[i]
                assert _call(lib, name, ptrs) == 1, (o, i, "same array")
                ptrs[o] = ctypes.c_void_p(FAKE[i].value + 16)
                assert _call(lib, name, ptrs) == 1, (o, i, "overlap")


@pytest.mark.parametrize("name", [n for n in CALLS if CALLS[n][3]])
def test_workspace_refused(lib, name):
    mk, k, _, _, outs = CALLS[name]
    need = getattr(lib, name + "_workspace_size")(mk())
    assert need > 0 and need % 256 == 0
    ptrs = FAKE[:k]
    assert _call(lib, name, ptrs, None, 0) == 6
    assert _call(lib, name, ptrs, FAKE[10], need - 1) == 6
    assert _call(lib, name, ptrs, ctypes.c_void_p(FAKE[10].value + 16), need) == 6
    for i in range(k):  # over an input or an output
        assert _call(lib, name, ptrs, FAKE[i], need) == 1, i


# ------------------------------------------------------------------- binding
T, C, FH = 5, 16, 24


def _args(dtype):
    z = lambda *s: torch.zeros(*s, dtype=dtype)
    return dict(x=z(T, C), weight=torch.ones(C), bias=torch.zeros(C), grad_y=z(T, C),
                w_gate=z(FH, C), w_up=z(FH, C), w_down=z(C, FH))


def _bind(mhc):
    return {
        "norm": lambda a, **k: mhc.mhc_layer_norm(a["x"], a["weight"], a["bias"], **k),
        "norm_bwd": lambda a, **k: mhc.mhc_layer_norm_backward(a["x"], a["weight"], a["grad_y"],
                                                               **k),
        "ffn": lambda a, **k: mhc.mhc_ffn(a["x"], a["w_gate"], a["w_up"], a["w_down"], **k),
        "ffn_bwd": lambda a, **k: mhc.mhc_ffn_backward(a["x"], a["w_gate"], a["w_up"],
                                                       a["w_down"], a["grad_y"], **k),
    }


USES = {"norm": ("x", "weight", "bias"), "norm_bwd": ("x", "weight", "grad_y"),
        "ffn": ("x", "w_gate", "w_up", "w_down"),
        "ffn_bwd": ("x", "w_gate", "w_up", "w_down", "grad_y")}


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("call", USES)
def test_well_formed_calls_reach_the_device_guard(mhc, call, dtype):
    with pytest.raises(ValueError, match="CUDA tensors only"):
        _bind(mhc)[call](_args(dtype))
    a = _args(dtype)
    a["bias"] = None
    with pytest.raises(ValueError, match="CUDA tensors only"):
        _bind(mhc)[call](a)


def _spoils(t):
    yield "short", t[:-1].clone() if t.dim() == 1 else t[:, :-1].clone()
    yield "long", torch.cat([t, t])
    yield "type", t.to(BF16 if t.dtype == F32 else F32)
    yield "half", t.to(torch.float16)
    yield "meta", t.to("meta")
    if t.dim() == 2:
        yield "strided", torch.zeros(t.shape[0], 2 * t.shape[1], dtype=t.dtype)[:, ::2]
        yield "transposed", torch.zeros(t.shape[1], t.shape[0], dtype=t.dtype).T
        yield "batched", t[None]
    else:
        yield "strided", torch.zeros(2 * t.shape[0])[::2]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("call", USES)
def test_spoiled_tensors_refused_by_name(mhc, call, dtype):
    for arg in USES[call]:
        for how, bad in _spoils(_args(dtype)[arg]):
            if arg == "x" and (call, how) in (("norm", "long"), ("norm", "type"), ("ffn", "long")):
                continue  # another row count, or the norm's other type: a call of its own
            a = _args(dtype)
            a[arg] = bad
            with pytest.raises(ValueError) as e:
                _bind(mhc)[call](a)
            assert "CUDA tensors only" not in str(e.value), (arg, how)


def test_outputs_checked(mhc):
    a = _args(BF16)
    b = _bind(mhc)
    with pytest.raises(ValueError, match="^out: shape"):
        b["norm"](a, out=torch.zeros(T, C + 8, dtype=BF16))
    with pytest.raises(ValueError, match="^out: dtype"):
        b["ffn"](a, out=torch.zeros(T, C))
    good = [torch.zeros(T, C, dtype=BF16), torch.zeros(C), torch.zeros(C)]
    for i, n in enumerate(("grad_x", "grad_weight", "grad_bias")):
        o = list(good)
        o[i] = o[i].double()
        with pytest.raises(ValueError, match=f"^{n}: dtype"):
            b["norm_bwd"](a, out=tuple(o))
    good = [torch.zeros_like(a[k]) for k in ("x", "w_gate", "w_up", "w_down")]
    for i, n in enumerate(("grad_x", "grad_w_gate", "grad_w_up", "grad_w_down")):
        o = list(good)
        o[i] = o[i][1:]
        with pytest.raises(ValueError, match=f"^{n}: shape"):
            b["ffn_bwd"](a, out=tuple(o))


def test_other_arguments_checked(mhc):
    a, b = _args(BF16), _bind(mhc)
    for call in ("ffn", "ffn_bwd"):
        with pytest.raises(ValueError, match="^act: "):
            b[call](a, act="relu")
    for call in USES:
        with pytest.raises(ValueError, match="^dev_status: "):
            b[call](a, dev_status=torch.zeros(1))
    with pytest.raises(ValueError, match="^workspace: on meta"):
        b["ffn"](a, workspace=torch.empty(8, dtype=torch.uint8, device="meta"))
    for call in ("ffn", "ffn_bwd", "norm_bwd"):
        with pytest.raises(ValueError, match="^workspace: "):
            b[call](a, workspace=torch.empty(1, dtype=torch.uint8).expand(1 << 20))
    for f in (mhc.mhc_ffn_workspace_size, mhc.mhc_ffn_backward_workspace_size):
        with pytest.raises(ValueError):
            f(4, 8, 8, torch.float16)
    with pytest.raises(ValueError):
        mhc.mhc_layer_norm_backward_workspace_size(4, 8, torch.float64)


def test_feedforward_layers_checked():
    from manifold_constrained_hyper_token_b200.feedforward import FeedForward
    p = dict(weight=None, w_gate=None, w_up=None, w_down=None)
    assert FeedForward([p]).grads == [None]
    for k in p:
        with pytest.raises(ValueError, match=f"layer 1: no {k}"):
            FeedForward([p, {j: v for j, v in p.items() if j != k}])


# ------------------------------------------------- the formulas themselves
def _gen(seed):
    g = torch.Generator().manual_seed(seed)
    return lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)


def _hold_to_differences(f, args, grads, gy, h=1e-5):
    """grad . d against the central difference of sum(gy . f) along random d: its error is
    h^2 times a third derivative (1e-10 here) and 1e-16 / h of the values (1e-11)."""
    for i, (a, g) in enumerate(zip(args, grads)):
        d = _gen(90 + i)(*a.shape)
        up, dn = list(args), list(args)
        up[i], dn[i] = a + h * d, a - h * d
        diff = float(((f(*up) - f(*dn)) * gy).sum()) / (2 * h)
        want = float((g * d).sum())
        scale = float(gy.norm()) * float(d.norm())
        assert abs(diff - want) <= 1e-7 * scale, (i, diff, want)


def test_norm_formula_matches_differences():
    n = _gen(1)
    x, w, b, gy = n(5, 24) * 2 + 1, n(24), n(24), n(5, 24)
    grads = R.norm_grad(x, w, gy, 1e-3)
    _hold_to_differences(lambda x, w, b: R.norm(x, w, b, 1e-3), (x, w, b), grads, gy)


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_ffn_formula_matches_differences(act):
    n = _gen(2)
    x, wg, wu, wd, gy = n(6, 8), n(12, 8) / 3, n(12, 8) / 3, n(8, 12) / 4, n(6, 8)
    grads = R.ffn_grad(x, wg, wu, wd, gy, act)
    _hold_to_differences(lambda *a: R.ffn(*a, act), (x, wg, wu, wd), grads, gy)
