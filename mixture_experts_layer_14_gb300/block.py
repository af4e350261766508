"""A residual block around the MoE layer, through forward, backward and optimiser step.

    h = x + residual;  u = RMSNorm(h);  block output: MoE(u) and the new residual h

(the block's output is added to h by the next block's norm).  With norms on both sides of every
branch, x is normed and gated on its way into the residual:

    h = res_scale residual + token_gate post_gate RMSNorm(x)

The training step adds the router's balance and z losses; ``train_block.py`` beside this file clips
the gradients by their common norm and applies AdamW.
"""

import torch

from . import (MOK_MXFP8, MoELayer, activation_pack, activation_unpack, balance_loss, balance_loss_workspace_size,
               prepare_weights, prepare_weights_bwd, rms_norm, rms_norm_backward, rms_norm_workspace_size,
               sandwich_norm, sandwich_norm_backward, sandwich_norm_workspace_size)

__all__ = ["MoEBlock"]

EXPERT_WEIGHTS = ("W_router", "W_gate", "W_up", "W_down", "Ws_gate", "Ws_up", "Ws_down")
NORMS = ("norm", "post_norm", "post_gate")


class MoEBlock:
    """Holds the norm weight and the layer of one block.  ``W``: the layer's weights (see
    :class:`MoELayer`) plus "norm" [d], bf16 or fp32.  For MOK_MXFP8 layers the norm writes the
    experts' codes and scales itself.  With "post_norm" [d] in W (and "post_gate" [d], if there is
    one) the block's input x is normed, gated and added to ``res_scale`` times the residual, which
    is then required.  ``selection``, ``saved``: see :class:`MoELayer`.  ``checkpoint`` "mxfp8": the
    layer's saved activations, u, h and x are kept in 8 bits between forward and backward, whose
    gradients are those at the values that these hold (for MOK_MXFP8 layers u is what the experts
    read)."""

    def __init__(self, D, W, eps=1e-6, alpha=0.0, z_coef=0.0, selection=None, res_scale=1.0, checkpoint=None, saved=None):
        self.D, self.W, self.eps, self.alpha, self.z_coef = D, W, eps, alpha, z_coef
        self.res_scale, self.checkpoint = res_scale, checkpoint
        self.post = W.get("post_norm") is not None
        if not self.post and (W.get("post_gate") is not None or res_scale != 1.0):
            raise ValueError("post_gate and res_scale need post_norm")
        self.mx = D.dtype == MOK_MXFP8
        if self.mx and W.get("prepared") is None:
            W["prepared"] = prepare_weights(D, W)
        if self.mx and W.get("prepared_bwd") is None:
            W["prepared_bwd"] = prepare_weights_bwd(D, W)
        self.layer = MoELayer(D, W, selection=selection, checkpoint=checkpoint, saved=saved)
        self.aux = None
        self._trained = None  # what the pass that backward belongs to left for it
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

    def _norm(self, x, residual, token_gate, mx, save):
        if not self.post:
            if token_gate is not None:
                raise ValueError("token_gate needs post_norm")
            return rms_norm(x, self.W["norm"], self.eps, residual=residual, mx=mx)
        if residual is None:
            raise ValueError("post_norm needs a residual")
        return sandwich_norm(x, residual, self.W["post_norm"], weight=self.W["norm"], gate=self.W.get("post_gate"),
                             token_gate=token_gate, res_scale=self.res_scale, eps=self.eps, mx=mx,
                             save="mxfp8" if save else None)

    def forward(self, x, residual=None, training=False, seq_offsets=None, token_mask=None, token_gate=None):
        """(y, h): the block's output [T,d] bf16 and the new residual (x itself without one).  In
        training the balance and z losses are in ``self.aux`` (a dict, see
        :func:`balance_loss`).  ``token_gate`` fp32 [T] (with post_norm): the branch's gate by token."""
        if training:
            self.aux = self._trained = None
        save = training and self.checkpoint is not None
        n = self._norm(x, residual, token_gate, "atoms" if self.mx else "rows" if save else None, save)
        self.u, self.h = n["y"], n.get("residual", x)
        y = self.layer.forward(self.u, training=training, want_logits=training,
                               x_mx=(n["codes"], n["scales"]) if self.mx else None)
        h = self.h
        if training:
            S = 1 if seq_offsets is None else seq_offsets.numel() - 1
            self.aux = balance_loss(self.D, self.layer.logits, self.layer.routing["topk_idx"],
                                    self._workspace("balance", balance_loss_workspace_size(self.D, S)),
                                    self.alpha, z_coef=self.z_coef, seq_offsets=seq_offsets,
                                    token_mask=token_mask)
            kept = [self.u, h, x if self.post else None]
            if save:
                kept[0] = n["codes"], n["scales"]
                kept[1] = (n["h_codes"], n["h_scales"]) if self.post else activation_pack(h)
                kept[2] = (n["x_codes"], n["x_scales"]) if self.post else None
                self.u = self.h = None
            self._trained = (*kept, h.dtype, token_gate, self.aux["dlogits"])
        return y, h

    def backward(self, dy, dh=None):
        """Gradients of the last forward with training=True (whatever ran for inference since) for
        upstream dy of the output and dh of the new residual (or None): the layer's dict plus "norm" (dweight, fp32), "dinput" (the gradient of x, bf16, and without
        post_norm of a bf16 residual) and, for an fp32 residual, "dresidual"; with post_norm
        "dresidual" always, "post_norm" and, where they are, "post_gate" and "token_gate" (fp32).  The
        gradient of the losses in ``self.aux`` is included."""
        if self._trained is None:
            raise RuntimeError("backward needs a forward with training=True")
        u, h, x, kind, token_gate, dlogits = self._trained
        if self.checkpoint:
            u = activation_unpack(*u, layout="atoms" if self.mx else "rows")
        g = self.layer.backward(u, dy, dlogits_aux=dlogits)
        if self.post:
            ws = self._workspace("norm", sandwich_norm_workspace_size(self.D.T, self.D.d))
            n = sandwich_norm_backward(x, h, self.W["post_norm"], dy=g["dX"], dres=dh, weight=self.W["norm"],
                                       gate=self.W.get("post_gate"), token_gate=token_gate, res_scale=self.res_scale,
                                       eps=self.eps, residual_dtype=kind, ws=ws)
            g["post_norm"] = n["dpost_weight"]
            for k in ("gate", "token_gate"):
                if "d" + k in n:
                    g["post_gate" if k == "gate" else k] = n["d" + k]
        else:
            if self.checkpoint:
                h = activation_unpack(*h, dtype=kind)
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
        by the counts in ``self.aux``, and so does one that has a "balance_bias" for its selection)."""
        names = [k for k in EXPERT_WEIGHTS + NORMS if self.W.get(k) is not None]
        return names, [self.W[k] for k in names]

    def gradients(self, g):
        """The gradients of :meth:`backward` in the order of :meth:`parameters`."""
        return [g[k] if k in NORMS else g["d" + k] for k in self.parameters()[0]]
