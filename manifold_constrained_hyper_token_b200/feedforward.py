"""The feed-forward layer function of an mHC stack: F(h) = ffn(layer_norm(h)).

``DepthStack`` wraps a layer function F and its backward.  ``FeedForward``
gives it both, from the library's layer norm and gated feed-forward block:

    stack = DepthStack(layers, ff.F, ff.F_backward, n=4)
    xL = stack.forward(x0)
    grad_x0, grads = stack.backward(grad_xL)     # phi, b, alpha per layer
    ff.grads[l]                                  # F's own parameters' gradients

Like the stack's layers it keeps no activation: the backward takes h_in and
recomputes the norm and the two projections from it.
"""
from __future__ import annotations

from typing import Sequence

from .api import mhc_ffn, mhc_ffn_backward, mhc_layer_norm, mhc_layer_norm_backward

PARAMS = ("weight", "bias", "w_gate", "w_up", "w_down")


class FeedForward:
    """Layer norm and gated feed-forward block for every layer of a stack.

    layers : per layer a dict with CUDA tensors ``weight`` [C] fp32, ``bias`` [C] fp32 or
             None, and ``w_gate``, ``w_up`` [F,C], ``w_down`` [C,F] of the activations' dtype
    act    : "silu" or "gelu"
    eps    : the norm's epsilon

    ``grads[l]`` holds layer l's parameter gradients of the last ``F_backward`` call, in a
    dict with the parameters' names (``bias`` only where the layer has one).
    """

    def __init__(self, layers: Sequence[dict], act: str = "silu", eps: float = 1e-6):
        self.layers = list(layers)
        self.act, self.eps = act, eps
        for l, p in enumerate(self.layers):
            missing = [k for k in PARAMS if k not in p and k != "bias"]
            if missing:
                raise ValueError(f"layer {l}: no {', '.join(missing)}")
        self.grads: list = [None] * len(self.layers)

    def _norm(self, l, h_in):
        p = self.layers[l]
        return mhc_layer_norm(h_in, p["weight"], p.get("bias"), eps=self.eps)

    def F(self, l, h_in):
        """f_out [T,C] of layer l."""
        p = self.layers[l]
        return mhc_ffn(self._norm(l, h_in), p["w_gate"], p["w_up"], p["w_down"], act=self.act)

    def F_backward(self, l, h_in, f_out, grad_f_out):
        """grad_h_in [T,C] of layer l; its parameters' gradients go to ``grads[l]``.  f_out is
        not read (the backward recomputes from h_in)."""
        p = self.layers[l]
        y = self._norm(l, h_in)
        gy, gwg, gwu, gwd = mhc_ffn_backward(y, p["w_gate"], p["w_up"], p["w_down"], grad_f_out,
                                             act=self.act)
        gh, gw, gb = mhc_layer_norm_backward(h_in, p["weight"], gy, eps=self.eps)
        g = dict(weight=gw, w_gate=gwg, w_up=gwu, w_down=gwd)
        if p.get("bias") is not None:
            g["bias"] = gb
        self.grads[l] = g
        return gh
