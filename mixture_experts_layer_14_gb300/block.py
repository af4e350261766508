"""A pre-norm residual block around the MoE layer, through forward, backward and optimiser step.

    h = x + residual;  u = RMSNorm(h);  block output: MoE(u) and the new residual h

(the block's output is added to h by the next block's norm).  The training step adds the router's
balance and z losses; ``train_block.py`` beside this file clips the gradients by their common norm and
applies AdamW.
"""

import torch

from . import (MOK_MXFP8, MoELayer, balance_loss, balance_loss_workspace_size, prepare_weights,
               prepare_weights_bwd, rms_norm, rms_norm_backward, rms_norm_workspace_size)

__all__ = ["MoEBlock"]

EXPERT_WEIGHTS = ("W_router", "W_gate", "W_up", "W_down", "Ws_gate", "Ws_up", "Ws_down")


class MoEBlock:
    """Holds the norm weight and the layer of one block.  ``W``: the layer's weights (see
    :class:`MoELayer`) plus "norm" [d], bf16 or fp32.  For MOK_MXFP8 layers the norm writes the
    experts' codes and scales itself."""

    def __init__(self, D, W, eps=1e-6, alpha=0.0, z_coef=0.0):
        self.D, self.W, self.eps, self.alpha, self.z_coef = D, W, eps, alpha, z_coef
        self.mx = D.dtype == MOK_MXFP8
        if self.mx and W.get("prepared") is None:
            W["prepared"] = prepare_weights(D, W)
        if self.mx and W.get("prepared_bwd") is None:
            W["prepared_bwd"] = prepare_weights_bwd(D, W)
        self.layer = MoELayer(D, W)
        self.aux = None
        self._trained = None  # u, h and the losses' gradient of the pass that backward belongs to
        self._ws = {}

    def requantise(self):
        """MXFP8: quantise the weights again, after an optimiser step changed them."""
        if self.mx:
            self.W["prepared"] = prepare_weights(self.D, self.W)
            self.W["prepared_bwd"] = prepare_weights_bwd(self.D, self.W)

    def _workspace(self, key, size):
        if key not in self._ws or self._ws[key].numel() < size:
            self._ws[key] = torch.zeros(size, dtype=torch.uint8, device=self.W["norm"].device)
        return self._ws[key]

    def forward(self, x, residual=None, training=False, seq_offsets=None, token_mask=None):
        """(y, h): the block's output [T,d] bf16 and the new residual (x itself without one).  In
        training the balance and z losses are in ``self.aux`` (a dict, see
        :func:`balance_loss`)."""
        if training:
            self.aux = self._trained = None
        n = rms_norm(x, self.W["norm"], self.eps, residual=residual, mx="atoms" if self.mx else None)
        self.u, self.h = n["y"], n.get("residual", x)
        y = self.layer.forward(self.u, training=training, want_logits=training,
                               x_mx=(n["codes"], n["scales"]) if self.mx else None)
        if training:
            S = 1 if seq_offsets is None else seq_offsets.numel() - 1
            self.aux = balance_loss(self.D, self.layer.logits, self.layer.routing["topk_idx"],
                                    self._workspace("balance", balance_loss_workspace_size(self.D, S)),
                                    self.alpha, z_coef=self.z_coef, seq_offsets=seq_offsets,
                                    token_mask=token_mask)
            self._trained = self.u, self.h, self.aux["dlogits"]
        return y, self.h

    def backward(self, dy, dh=None):
        """Gradients of the last forward with training=True (whatever ran for inference since) for
        upstream dy of the output and dh of the new residual (or None): the layer's dict plus "norm" (dweight, fp32), "dinput" (the gradient of x, bf16, and of a bf16
        residual) and, for an fp32 residual, "dresidual".  The gradient of the losses in
        ``self.aux`` is included."""
        if self._trained is None:
            raise RuntimeError("backward needs a forward with training=True")
        u, h, dlogits = self._trained
        g = self.layer.backward(u, dy, dlogits_aux=dlogits)
        ws = self._workspace("norm", rms_norm_workspace_size(self.D.T, self.D.d))
        n = rms_norm_backward(g["dX"], h, self.W["norm"], self.eps, dres=dh, ws=ws)
        g["norm"] = n["dweight"]
        g["dinput"] = n["dx"]
        if "dresidual" in n:
            g["dresidual"] = n["dresidual"]
        return g

    def parameters(self):
        """Names and weights, in the order of :meth:`gradients`.  The router's "bias" is not among them:
        it enters the logits, but the layer has no gradient for it (a program that has one moves it
        by the counts in ``self.aux``)."""
        names = [k for k in EXPERT_WEIGHTS if self.W.get(k) is not None] + ["norm"]
        return names, [self.W[k] for k in names]

    def gradients(self, g):
        """The gradients of :meth:`backward` in the order of :meth:`parameters`."""
        return [g["norm"] if k == "norm" else g["d" + k] for k in self.parameters()[0]]
