"""Gradient norm with clipping, and AdamW over all weights in one launch.

Argument marshalling for mok_grad_norm and mok_adamw_step (declared in ``include/mok.h``); like the
rest of the binding there is no path without the compiled library.
"""

import ctypes

import numpy as np
import torch

from . import _ELEM, AdamWArgs, AdamWTensor, MokError, _check, _elem, _ptr, _stream, _want_ws, lib

__all__ = ["TensorList", "grad_norm", "grad_norm_workspace_size", "AdamW"]

# AdamWTensor as a numpy record, so that a step writes all gradient addresses at once
_TABLE = np.dtype([(n, np.uint64) for n in ("param", "grad", "master", "exp_avg", "exp_avg_sq", "exp_avg_scale",
                                            "exp_avg_sq_scale")]
                  + [("numel", np.int64), ("weight_decay", np.float64), ("param_type", np.int32),
                     ("grad_type", np.int32)])
assert _TABLE.itemsize == ctypes.sizeof(AdamWTensor)

STATE_FORMATS = {"f32": 0, "mxfp8": 1}   # mok_state_format
STATE_KEYS = ("master", "exp_avg", "exp_avg_sq", "exp_avg_scale", "exp_avg_sq_scale")


class TensorList:
    """bf16 and fp32 CUDA tensors checked once and held with their addresses, for
    :func:`grad_norm` and :meth:`AdamW.step`.  A program whose gradients live in the same buffers
    every step makes one and keeps it; the values are read at each call.  The tensors must not be
    resized or given other storage while the list is in use."""

    def __init__(self, tensors):
        self.tensors = list(tensors)
        n = len(self.tensors)
        self.device = self.tensors[0].device if n else torch.device("cuda", torch.cuda.current_device())
        types = [_ELEM.get(t.dtype, -1) for t in self.tensors]
        for i, t in enumerate(self.tensors):
            if types[i] < 0:
                _elem(t, f"tensor {i}")
            if not t.is_contiguous():
                raise ValueError(f"tensor {i} must be contiguous")
            if not t.is_cuda or t.device != self.device:
                raise ValueError(f"tensor {i} must live on one CUDA device with the others")
        self.view_pointers = np.array([t.data_ptr() for t in self.tensors], dtype=np.uint64)
        self.view_numel = np.array([t.numel() for t in self.tensors], dtype=np.int64)
        self.view_types = np.array(types, dtype=np.int32)
        # the same arrays as C pointers
        self.pointers, self.numel, self.types = (
            a.ctypes.data for a in (self.view_pointers, self.view_numel, self.view_types))

    def __len__(self):
        return len(self.tensors)


def _as_list(tensors):
    return tensors if isinstance(tensors, TensorList) else TensorList(tensors)


def grad_norm_workspace_size(grads):
    g = _as_list(grads)
    n = lib().mok_grad_norm_workspace_size(len(g), g.numel)
    if n == 0:
        raise MokError("unsupported tensor sizes")
    return n


def grad_norm(grads, max_norm=0.0, ws=None):
    """Norm of all gradients together and the factor that clips it: fp32 [2] on the device,
    {norm, min(1, max_norm / norm)}; the factor is 1 without a positive max_norm and NaN when the
    norm is not finite.  ``grads``: a list of bf16 / fp32 tensors or a :class:`TensorList`;
    ``ws``: grad_norm_workspace_size(grads) bytes (allocated per call when None)."""
    g = _as_list(grads)
    if ws is None:
        ws = torch.empty(grad_norm_workspace_size(g), dtype=torch.uint8, device=g.device)
    _want_ws(ws, g.device)
    out = torch.empty(2, dtype=torch.float32, device=g.device)
    _check(lib().mok_grad_norm(len(g), g.pointers, g.numel, g.types, max_norm, _ptr(out), _ptr(ws),
                               ws.numel(), _stream()))
    return out


class AdamW:
    """AdamW over a list of weights, one launch per step (up to 384 tensors; more take several).

    ``params``: bf16 or fp32 CUDA tensors, updated in place (held, with their addresses: they must
    not be given other storage), no two of them on the same memory.  The learning rate and the step's number are constants of the
    launch, in a captured CUDA graph too.  A bf16 weight has an fp32 master that
    the steps accumulate in.  ``states``: "f32", or "mxfp8" for E4M3 codes with one power-of-two
    scale per 32 elements and dithered rounding (1.03 bytes per state and element; mok.h,
    mok_state_format: elements whose gradients are some 400 times smaller than the largest of their 32
    neighbours take smaller steps than they should, so that weights like W_router [d, E] under a
    very uneven load belong to an optimiser with "f32").  ``weight_decay``: one value, or one per tensor.  ``state``: buffers to use
    (and resume from) instead of new ones, a dict of lists like :meth:`state_dict` returns."""

    def __init__(self, params, betas=(0.9, 0.95), eps=1e-8, weight_decay=0.0, states="f32", state=None,
                 step=0):
        if states not in STATE_FORMATS:
            raise ValueError(f"states must be one of {sorted(STATE_FORMATS)}")
        self.params = list(params)
        self.states = states
        self.args = AdamWArgs(0.0, betas[0], betas[1], eps, step, STATE_FORMATS[states])
        n = len(self.params)
        decay = list(weight_decay) if isinstance(weight_decay, (list, tuple)) else [weight_decay] * n
        if len(decay) != n:
            raise ValueError(f"weight_decay: {len(decay)} values for {n} tensors")
        checked = TensorList(self.params)
        self.device = checked.device
        self.table = (AdamWTensor * n)()
        self._view = np.frombuffer(self.table, dtype=_TABLE) if n else np.zeros(0, dtype=_TABLE)
        self._view["param"], self._view["param_type"] = checked.view_pointers, checked.view_types
        self._view["numel"], self._view["weight_decay"] = checked.view_numel, decay
        self.state = {}
        for key in STATE_KEYS:
            buffers = self.state[key] = self._buffers(key, checked.view_numel.tolist(), state)
            self._view[key] = [0 if t is None else t.data_ptr() for t in buffers]
        self._check_disjoint()

    def _check_disjoint(self):
        """One launch updates everything, so no element may be reached twice (tied weights are one
        entry, with the sum of their gradients)."""
        v = self._view
        n = v["numel"]
        state = n if self.states == "mxfp8" else 4 * n
        scale = (n + 31) // 32
        size = np.concatenate([n * np.where(v["param_type"] == 0, 2, 4), 4 * n, state, state, scale, scale])
        start = np.concatenate([v[key] for key in ("param", *STATE_KEYS)])
        there = (start != 0) & (size != 0)
        start, size = start[there], size[there].astype(np.uint64)
        order = np.argsort(start)
        start, end = start[order], (start + size)[order]
        if (start[1:] < end[:-1]).any():
            raise ValueError("weights and states must not share memory")

    def _buffers(self, key, sizes, state):
        """The tensors of one kind of state, None where a weight has none: new ones, or the given
        ones checked."""
        mx, master, scale = self.states == "mxfp8", key == "master", key.endswith("scale")
        if scale and not mx:
            return [None] * len(sizes)
        given = None if state is None else state.get(key) or [None] * len(sizes)
        if given is not None and len(given) != len(sizes):
            raise ValueError(f"state[{key!r}]: {len(given)} entries for {len(sizes)} tensors")
        dtype = torch.uint8 if mx and not master else torch.float32
        out = []
        for i, (p, n) in enumerate(zip(self.params, sizes)):
            n = (n + 31) // 32 if scale else n
            if master and p.dtype == torch.float32:
                t = None
            elif given is not None:
                t = given[i]
                if t is None or t.dtype != dtype or t.numel() != n or not t.is_contiguous() or t.device != self.device:
                    raise ValueError(f"state[{key!r}][{i}] must be {n} contiguous {dtype} elements on {self.device}")
            elif master:
                t = p.detach().to(torch.float32).reshape(-1)
            else:
                t = torch.zeros(n, dtype=dtype, device=self.device)
            out.append(t)
        return out

    @property
    def steps(self):
        """Steps taken so far."""
        return self.args.step

    def step(self, grads, lr, clip=None):
        """One step with gradients ``grads`` (a list in the order of the weights, or a
        :class:`TensorList`) and learning rate ``lr``.  ``clip``: the tensor that
        :func:`grad_norm` returned; its factor scales the gradients, and a factor that is NaN
        leaves every weight and state unchanged (the step still counts)."""
        g = _as_list(grads)
        if len(g) != len(self.params):
            raise ValueError(f"{len(g)} gradients for {len(self.params)} tensors")
        if not np.array_equal(self._view["numel"], g.view_numel):
            i = int(np.nonzero(self._view["numel"] != g.view_numel)[0][0])
            raise ValueError(f"gradient {i}: {g.view_numel[i]} elements, the weight has {self.params[i].numel()}")
        if len(g) and g.device != self.device:
            raise ValueError(f"gradients must live on {self.device}")
        self._view["grad"], self._view["grad_type"] = g.view_pointers, g.view_types
        if clip is not None and (clip.dtype != torch.float32 or clip.numel() != 2 or clip.device != self.device
                                 or not clip.is_contiguous()):
            raise ValueError(f"clip must be 2 fp32 values on {self.device}")
        args = self.args
        args.lr = lr
        args.step += 1
        rc = lib().mok_adamw_step(ctypes.byref(args), self.table, len(self.params), _ptr(clip), _stream())
        if rc != 0:
            args.step -= 1
            _check(rc)

    def state_dict(self):
        """The states (not copied) and the number of steps: AdamW(params, ..., **state_dict()) goes on
        from them."""
        return {"state": dict(self.state), "step": int(self.args.step), "states": self.states}
