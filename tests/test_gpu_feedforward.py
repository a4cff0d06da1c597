"""The feed-forward layer function inside the stack: DepthStack with FeedForward, forward and
backward, against an fp64 chain (the oracle's mHC layer around the fp64 norm and block)."""
import numpy as np
import pytest
import torch

import layer_reference as R
from conftest import assert_close

pytestmark = pytest.mark.gpu

L, N, EPS = 3, 4, 1e-6
# fp32: the framework's parity tolerance for one layer, times the layers that a value passes.
# bf16: a layer stores five tensors on the way up (h_in, the norm's y, a, f_out, x_next) and
# five on the way down (grad_f_out, dg or du, grad_y, grad_h_in, grad_x), and each storing
# moves a value by up to 2^-8 of itself: at most 10 L 2^-8 (here 0.117) of an element when all
# fall the same way.  In a tensor's 2-norm the storings are independent, sqrt(10 L) 2^-8, and
# the mHC layers around F, themselves held to 2e-2 by their own tests, pass a value 2 L times:
# sqrt(10 L 2^-16 + 2 L 2e-2^2) = 0.0534.
# (2e-2 L, the same product over layers as for fp32, counts only five storings per layer:
# the chain has ten.)  The 2-norm bound is for tensors whose elements carry the storings'
# relative errors; grad_phi = x dz does not: dz is a difference of sums over C whose terms
# cancel, so with a single token its one relative error can exceed any of theirs.
TOL = {torch.float32: 1e-5 * L, torch.bfloat16: 10 * L * 2.0 ** -8}
REL = {torch.float32: 1e-5 * L, torch.bfloat16: (10 * L * 2.0 ** -16 + 2 * L * 2e-2 ** 2) ** 0.5}


@pytest.fixture(scope="module")
def mhc():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from manifold_constrained_hyper_token_b200 import build
    build.build()
    import manifold_constrained_hyper_token_b200 as m
    return m


def _params(C, F, dtype):
    from manifold_constrained_hyper_token_b200 import synth
    layers, ffs = [], []
    for l in range(L):
        layers.append(synth.layer_params(N, C, seed=l))
        g = torch.Generator().manual_seed(100 + l)
        n = lambda *s: torch.randn(*s, generator=g)
        ffs.append(dict(weight=1 + 0.1 * n(C), bias=0.1 * n(C) if l else None,
                        w_gate=(n(F, C) * C ** -0.5).to(dtype),
                        w_up=(n(F, C) * C ** -0.5).to(dtype),
                        w_down=(n(C, F) * F ** -0.5).to(dtype)))
    return layers, ffs


def _cuda(ps):
    return [{k: None if v is None else v.cuda() for k, v in p.items()} for p in ps]


def _t(a):
    return torch.from_numpy(np.asarray(a, dtype=np.float64))


def _chain(oracle, layers, ffs, x0, G, act):
    """x_L, grad_x0, per layer (grad_phi, F's gradients) in fp64."""
    x, saved = x0.double(), []
    for p, f in zip(layers, ffs):
        m = oracle.pre(x.numpy(), p["phi"], p["b"], float(p["alpha"][0]))
        h = _t(m["h_in"])
        y = R.norm(h, f["weight"], f["bias"], EPS)
        fo = R.ffn(y, f["w_gate"], f["w_up"], f["w_down"], act)
        saved.append((x, h, y, fo, m))
        x = _t(oracle.post(x.numpy(), fo.numpy(), m["H_post"], m["H_res"]))
    xL, G, out = x, G.double(), [None] * L
    for l in reversed(range(L)):
        x, h, y, fo, m = saved[l]
        p, f = layers[l], ffs[l]
        a = float(p["alpha"][0])
        # the merge's gradient with respect to f_out, then F's backward, then the layer's
        gf = torch.einsum("ti,tic->tc", _t(m["H_post"]), G)
        gy, gwg, gwu, gwd = R.ffn_grad(y, f["w_gate"], f["w_up"], f["w_down"], gf, act)
        gh, gw, gb = R.norm_grad(h, f["weight"], gy, EPS)
        r = oracle.backward(x.numpy(), p["phi"], p["b"], a, fo.numpy(), G.numpy(), gh.numpy())
        out[l] = (_t(r["grad_phi"]), dict(weight=gw, bias=gb, w_gate=gwg, w_up=gwu, w_down=gwd))
        G = _t(r["grad_x"]).reshape(x.shape)
    return xL, G, out


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,C,F,act", [(1, 64, 96, "silu"), (37, 72, 200, "silu"),
                                       (300, 128, 264, "gelu")])
def test_stack_of_feed_forward_layers(mhc, oracle_mod, T, C, F, act, dtype):
    from manifold_constrained_hyper_token_b200.depth import DepthStack
    from manifold_constrained_hyper_token_b200.feedforward import FeedForward
    layers, ffs = _params(C, F, dtype)
    g = torch.Generator().manual_seed(T)
    x0, G = (torch.randn(T, N, C, generator=g).to(dtype) for _ in range(2))
    xL, gx0, want = _chain(oracle_mod, layers, ffs, x0, G, act)
    tol, runs = TOL[dtype], []
    for block in (1, 2, L):
        ff = FeedForward(_cuda(ffs), act=act, eps=EPS)
        st = DepthStack(_cuda(layers), ff.F, ff.F_backward, n=N, block=block)
        got = st.forward(x0.cuda())
        ggx, ggrads = st.backward(G.cuda())
        runs.append([got, ggx, *[gr[0] for gr in ggrads],
                     *[ff.grads[l][k] for l in range(L) for k in sorted(ff.grads[l])]])
        for l in range(L):
            assert ("bias" in ff.grads[l]) == (ffs[l]["bias"] is not None)
    def hold(got, ref, name, rel=REL[dtype]):
        got, ref = got.detach().double().cpu(), ref.reshape(got.shape)
        assert_close(got.numpy(), ref.numpy(), tol, name)
        assert rel is None or R.norm_rel(got, ref) < rel, name

    hold(got, xL, "x_L")
    hold(ggx, gx0, "grad_x0")
    for l in range(L):
        hold(ggrads[l][0], want[l][0], f"grad_phi {l}", rel=None)
        for k, v in ff.grads[l].items():
            hold(v, want[l][1][k], f"{k} {l}")
    for r in runs[1:]:  # recompute changes no bit
        assert all(torch.equal(a, b) for a, b in zip(runs[0], r))
