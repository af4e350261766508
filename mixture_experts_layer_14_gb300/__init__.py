"""GB300-native (sm_103a) DeepSeek-V3-style MoE layer — Python binding of the C-ABI library.

This module only marshals arguments: it checks tensor shapes, dtypes, devices and contiguity,
allocates outputs with PyTorch and passes raw device pointers and the current CUDA stream to
``libmok.so`` (declared in ``include/mok.h``).  Every step of the layer runs in that library's
kernels.  There is no fallback: without the compiled library every call raises.

Entry points mirror the C ABI: :func:`route`, :func:`dispatch_index`, :func:`moe_forward`,
:func:`moe_backward`, :func:`layer_forward_host`, plus :class:`MoELayer`, a small convenience
holder of weights and workspaces.  Around the layer: :func:`rms_norm`, :func:`balance_loss`,
:func:`grad_norm` and :class:`AdamW`, and :class:`MoEBlock`, which runs them together.
"""

import ctypes
import os

import torch

__all__ = [
    "MokError", "Dims", "Weights", "lib", "lib_path", "dims", "route", "dispatch_index",
    "moe_forward", "moe_backward", "layer_forward_host", "workspace_size", "saved_size",
    "read_status", "clear_status", "last_launch_count", "MoELayer", "EXPORTED_SYMBOLS",
    "MOK_BF16", "MOK_MXFP8", "MOK_NVFP4", "prepare_weights", "prepare_weights_bwd",
    "mx_quantize_rows", "nvfp4_set_activation_amax",
    "rms_norm", "rms_norm_backward", "rms_norm_workspace_size", "balance_loss",
    "balance_loss_workspace_size", "TensorList", "grad_norm", "grad_norm_workspace_size", "AdamW",
    "MoEBlock",
]

MOK_BF16, MOK_MXFP8, MOK_NVFP4 = 0, 1, 2
PASS_FORWARD, PASS_BACKWARD = 0, 1

EXPORTED_SYMBOLS = [
    "mok_workspace_size", "mok_saved_size", "mok_prepared_size", "mok_prepare_weights",
    "mok_route", "mok_dispatch_index", "mok_moe_forward", "mok_moe_backward",
    "mok_layer_host_extra_size", "mok_layer_forward_host", "mok_status_string",
    "mok_read_device_status", "mok_clear_device_status", "mok_last_launch_count",
    "mok_timing_enable", "mok_timing_collect", "mok_dispatch_index_noalloc",
    "mok_mx_quantize_rows", "mok_selftest_bounded_wait", "mok_prepared_bwd_size",
    "mok_prepare_weights_bwd", "mok_set_forward_schedule", "mok_nvfp4_set_activation_amax",
    "mok_rms_norm", "mok_rms_norm_workspace_size", "mok_rms_norm_backward",
    "mok_balance_loss_workspace_size", "mok_balance_loss", "mok_grad_norm_workspace_size",
    "mok_grad_norm", "mok_adamw_step", "mok_moe_forward_mx", "mok_moe_backward_aux",
]


class MokError(RuntimeError):
    pass


class Dims(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("d", ctypes.c_int32), ("E", ctypes.c_int32),
                ("k", ctypes.c_int32), ("F", ctypes.c_int32), ("F_shared", ctypes.c_int32),
                ("n_shared", ctypes.c_int32), ("dtype", ctypes.c_int32)]


class Weights(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in (
        "W_router", "router_bias", "W_gate", "W_up", "W_down", "Ws_gate", "Ws_up", "Ws_down",
        "prepared", "prepared_bwd")]


class AdamWTensor(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in (
        "param", "grad", "master", "exp_avg", "exp_avg_sq", "exp_avg_scale", "exp_avg_sq_scale")] + [
        ("numel", ctypes.c_int64), ("weight_decay", ctypes.c_double),
        ("param_type", ctypes.c_int32), ("grad_type", ctypes.c_int32)]


class AdamWArgs(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_double), ("beta1", ctypes.c_double), ("beta2", ctypes.c_double),
                ("eps", ctypes.c_double), ("step", ctypes.c_int64), ("state_format", ctypes.c_int32)]


_LIB = None
_VP = ctypes.c_void_p
_SZ = ctypes.c_size_t
_I64, _INT, _F = ctypes.c_int64, ctypes.c_int, ctypes.c_float
_DP = ctypes.POINTER(Dims)
_WP = ctypes.POINTER(Weights)


def lib_path():
    return os.path.join(os.path.dirname(os.path.abspath(__file__)), "libmok.so")


def lib():
    """The loaded libmok.so (raises if it has not been built)."""
    global _LIB
    if _LIB is None:
        path = lib_path()
        if not os.path.exists(path):
            raise MokError(f"{path} is missing; build it with `python -m mixture_experts_layer_14_gb300.build`")
        L = ctypes.CDLL(path)
        sig = {
            "mok_workspace_size": (_SZ, [_DP, ctypes.c_int]),
            "mok_saved_size": (_SZ, [_DP]),
            "mok_prepared_size": (_SZ, [_DP]),
            "mok_prepared_bwd_size": (_SZ, [_DP]),
            "mok_prepare_weights_bwd": (ctypes.c_int, [_DP, _WP, _VP, _VP]),
            "mok_layer_host_extra_size": (_SZ, [_DP]),
            "mok_prepare_weights": (ctypes.c_int, [_DP, _WP, _VP, _VP]),
            "mok_route": (ctypes.c_int, [_DP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _SZ, _VP]),
            "mok_dispatch_index": (ctypes.c_int, [_DP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _SZ, _VP]),
            "mok_moe_forward": (ctypes.c_int, [_DP, _WP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _SZ, _VP]),
            "mok_moe_backward": (ctypes.c_int, [_DP, _WP] + [_VP] * 19 + [_SZ, _VP]),
            "mok_layer_forward_host": (ctypes.c_int, [_DP, _WP, _VP, _VP, _VP, _SZ, _VP]),
            "mok_status_string": (ctypes.c_char_p, [ctypes.c_int]),
            "mok_read_device_status": (ctypes.c_int, [_VP, ctypes.POINTER(ctypes.c_int), _VP]),
            "mok_clear_device_status": (ctypes.c_int, [_VP, _VP]),
            "mok_last_launch_count": (ctypes.c_int, []),
            "mok_timing_enable": (ctypes.c_int, [ctypes.c_int]),
            "mok_selftest_bounded_wait": (ctypes.c_int, [_VP, ctypes.c_int64, _VP]),
            "mok_mx_quantize_rows": (ctypes.c_int, [ctypes.c_int64, ctypes.c_int, _VP, _VP, _VP, _VP]),
            "mok_dispatch_index_noalloc": (ctypes.c_int, [_DP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP]),
            "mok_set_forward_schedule": (ctypes.c_int, [ctypes.c_int, ctypes.POINTER(ctypes.c_int)]),
            "mok_nvfp4_set_activation_amax": (ctypes.c_int, [_DP, _VP, ctypes.c_float, ctypes.c_float, _VP]),
            "mok_rms_norm": (ctypes.c_int, [_I64, _INT, _F, _VP, _VP, _INT, _VP, _INT, _VP, _VP, _VP, _VP, _INT, _VP]),
            "mok_rms_norm_workspace_size": (_SZ, [_I64, _INT]),
            "mok_rms_norm_backward": (ctypes.c_int, [_I64, _INT, _F, _VP, _VP, _INT, _VP, _INT] + [_VP] * 5 + [_SZ, _VP]),
            "mok_balance_loss_workspace_size": (_SZ, [_DP, _I64]),
            "mok_balance_loss": (ctypes.c_int, [_DP, _VP, _VP, _VP, _I64, _VP, _F, _F] + [_VP] * 5 + [_SZ, _VP]),
            "mok_grad_norm_workspace_size": (_SZ, [_INT, _VP]),
            "mok_grad_norm": (ctypes.c_int, [_INT, _VP, _VP, _VP, _F, _VP, _VP, _SZ, _VP]),
            "mok_adamw_step": (ctypes.c_int, [ctypes.POINTER(AdamWArgs), ctypes.POINTER(AdamWTensor), _INT, _VP, _VP]),
            "mok_moe_forward_mx": (ctypes.c_int, [_DP, _WP] + [_VP] * 10 + [_SZ, _VP]),
            "mok_moe_backward_aux": (ctypes.c_int, [_DP, _WP] + [_VP] * 20 + [_SZ, _VP]),
            "mok_timing_collect": (ctypes.c_int, [ctypes.c_char_p, ctypes.POINTER(ctypes.c_int),
                                                  ctypes.POINTER(ctypes.c_double), ctypes.c_int,
                                                  ctypes.POINTER(ctypes.c_int)]),
        }
        for name, (res, args) in sig.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _LIB = L
    return _LIB


def _check(rc):
    if rc != 0:
        raise MokError(lib().mok_status_string(rc).decode())


def _ptr(t):
    return None if t is None else t.data_ptr()


# The current stream's handle of a device, without a Stream object around it (a sixth of a small
# call's time on the host) where this PyTorch has it.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream():
    if _raw_stream is not None:
        return _raw_stream(torch.cuda.current_device())
    return torch.cuda.current_stream().cuda_stream


def _want(t, name, shape, dtype, device, check_device=True):
    if t is not None and t.shape == shape and t.dtype == dtype and t.is_contiguous() and (
            not check_device or (t.is_cuda and (device is None or t.device == device))):
        return t
    if t is None:
        raise ValueError(f"{name} is required")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)} != {tuple(shape)}")
    if t.dtype != dtype:
        raise ValueError(f"{name}: dtype {t.dtype} != {dtype}")
    if check_device and (not t.is_cuda or (device is not None and t.device != device)):
        raise ValueError(f"{name} must live on {device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _want_ws(ws, device):
    if ws.dtype != torch.uint8 or ws.device != device or not ws.is_cuda or not ws.is_contiguous():
        raise ValueError(f"ws must be a contiguous uint8 tensor on {device}")


def dims(T, d, E, k, F, F_shared=0, n_shared=1, dtype=MOK_BF16):
    return Dims(T, d, E, k, F, F_shared if n_shared else 0, n_shared, dtype)


def workspace_size(D, backward=False):
    n = lib().mok_workspace_size(ctypes.byref(D), PASS_BACKWARD if backward else PASS_FORWARD)
    if n == 0:
        raise MokError("unsupported layer dimensions")
    return n


def saved_size(D):
    return lib().mok_saved_size(ctypes.byref(D))


def read_status(ws):
    v = ctypes.c_int(0)
    _check(lib().mok_read_device_status(_ptr(ws), ctypes.byref(v), _stream()))
    return v.value


def clear_status(ws):
    _check(lib().mok_clear_device_status(_ptr(ws), _stream()))


def last_launch_count():
    return lib().mok_last_launch_count()


def selftest_bounded_wait(ws, budget_ns=50_000_000):
    """Runs a kernel whose bounded wait must run out; the status word of ws then reads
    MOK_ERR_TIMEOUT (-5)."""
    _check(lib().mok_selftest_bounded_wait(_ptr(ws), int(budget_ns), _stream()))


SCHEDULE_TWO_LAUNCHES, SCHEDULE_FUSED = 0, 1


def set_forward_schedule(schedule):
    """Process-wide schedule of the bf16 forward's expert GEMMs (SCHEDULE_TWO_LAUNCHES, the
    default, or SCHEDULE_FUSED: one persistent launch fed by a device work counter); returns the
    previous one.  Results are bit-identical under both."""
    prev = ctypes.c_int(0)
    _check(lib().mok_set_forward_schedule(int(schedule), ctypes.byref(prev)))
    return prev.value


def timing_enable(on=True):
    """Record a CUDA event pair around every kernel the library launches on this thread."""
    _check(lib().mok_timing_enable(1 if on else 0))


def timing_collect(max_kernels=64):
    """{kernel name: (launches, summed device ms)} of the recorded launches; clears them."""
    names = ctypes.create_string_buffer(32 * max_kernels)
    launches = (ctypes.c_int * max_kernels)()
    ms = (ctypes.c_double * max_kernels)()
    n = ctypes.c_int(0)
    _check(lib().mok_timing_collect(names, launches, ms, max_kernels, ctypes.byref(n)))
    out = {}
    for i in range(n.value):
        name = names.raw[32 * i:32 * i + 32].split(b"\0", 1)[0].decode()
        out[name] = (launches[i], ms[i])
    return out


def _weights_struct(D, W):
    dev = W["W_gate"].device
    bf = torch.bfloat16
    _want(W["W_router"], "W_router", (D.d, D.E), bf, dev)
    _want(W["W_gate"], "W_gate", (D.E, D.d, D.F), bf, dev)
    _want(W["W_up"], "W_up", (D.E, D.d, D.F), bf, dev)
    _want(W["W_down"], "W_down", (D.E, D.F, D.d), bf, dev)
    if W.get("bias") is not None:
        _want(W["bias"], "bias", (D.E,), torch.float32, dev)
    if D.n_shared:
        _want(W["Ws_gate"], "Ws_gate", (D.d, D.F_shared), bf, dev)
        _want(W["Ws_up"], "Ws_up", (D.d, D.F_shared), bf, dev)
        _want(W["Ws_down"], "Ws_down", (D.F_shared, D.d), bf, dev)
    if D.dtype != MOK_BF16 and W.get("prepared") is not None:
        _want(W["prepared"], "prepared", (prepared_size(D),), torch.uint8, dev)
    if D.dtype == MOK_MXFP8 and W.get("prepared_bwd") is not None:
        _want(W["prepared_bwd"], "prepared_bwd", (lib().mok_prepared_bwd_size(ctypes.byref(D)),), torch.uint8, dev)
    return Weights(
        W["W_router"].data_ptr(), W["bias"].data_ptr() if W.get("bias") is not None else None,
        W["W_gate"].data_ptr(), W["W_up"].data_ptr(), W["W_down"].data_ptr(),
        W["Ws_gate"].data_ptr() if D.n_shared else None,
        W["Ws_up"].data_ptr() if D.n_shared else None,
        W["Ws_down"].data_ptr() if D.n_shared else None,
        W["prepared"].data_ptr() if W.get("prepared") is not None else None,
        W["prepared_bwd"].data_ptr() if W.get("prepared_bwd") is not None else None)


def route(D, x, W_router, bias, ws, want_logits=False):
    """Returns (topk_idx[T,k] int32, topk_w[T,k] fp32, logits[T,E] fp32 or None)."""
    dev = x.device
    _want(x, "x", (D.T, D.d), torch.bfloat16, dev)
    _want(W_router, "W_router", (D.d, D.E), torch.bfloat16, dev)
    if bias is not None:
        _want(bias, "bias", (D.E,), torch.float32, dev)
    idx = torch.empty((D.T, D.k), dtype=torch.int32, device=dev)
    w = torch.empty((D.T, D.k), dtype=torch.float32, device=dev)
    logits = torch.empty((D.T, D.E), dtype=torch.float32, device=dev) if want_logits else None
    _check(lib().mok_route(ctypes.byref(D), _ptr(x), _ptr(W_router), _ptr(bias), _ptr(idx), _ptr(w),
                           _ptr(logits), _ptr(ws), ws.numel(), _stream()))
    return idx, w, logits


def dispatch_index(D, topk_idx, topk_w, ws):
    """Returns a dict with counts[E], offsets[E+1], sorted_tok[T*k], sorted_w[T*k], inv_pos[T,k]."""
    dev = topk_idx.device
    _want(topk_idx, "topk_idx", (D.T, D.k), torch.int32, dev)
    _want(topk_w, "topk_w", (D.T, D.k), torch.float32, dev)
    R = D.T * D.k
    out = {
        "topk_idx": topk_idx, "topk_w": topk_w,
        "counts": torch.empty((D.E,), dtype=torch.int32, device=dev),
        "offsets": torch.empty((D.E + 1,), dtype=torch.int32, device=dev),
        "sorted_tok": torch.empty((R,), dtype=torch.int32, device=dev),
        "sorted_w": torch.empty((R,), dtype=torch.float32, device=dev),
        "inv_pos": torch.empty((D.T, D.k), dtype=torch.int32, device=dev),
    }
    _check(lib().mok_dispatch_index(
        ctypes.byref(D), _ptr(topk_idx), _ptr(topk_w), _ptr(out["counts"]), _ptr(out["offsets"]),
        _ptr(out["sorted_tok"]), _ptr(out["sorted_w"]), _ptr(out["inv_pos"]), _ptr(ws), ws.numel(),
        _stream()))
    return out


def dispatch_index_noalloc(D, topk_idx, topk_w, out):
    """Pull schedule into the caller's preallocated tensors ``out`` (same keys as the dict of
    :func:`dispatch_index`) without a workspace: for callers that may not allocate device memory
    while routing.  The library keeps its scratch in a fixed device array (1 MiB of histogram),
    looked up for the current device, so every tensor must live there."""
    dev = torch.device("cuda", torch.cuda.current_device()) if torch.cuda.is_available() else "cuda"
    R = D.T * D.k
    specs = [(topk_idx, "topk_idx", (D.T, D.k), torch.int32), (topk_w, "topk_w", (D.T, D.k), torch.float32)]
    for key, shape, dtype in (("counts", (D.E,), torch.int32), ("offsets", (D.E + 1,), torch.int32),
                              ("sorted_tok", (R,), torch.int32), ("sorted_w", (R,), torch.float32),
                              ("inv_pos", (D.T, D.k), torch.int32)):
        specs.append((out.get(key), f"out[{key!r}]", shape, dtype))
    for t, name, shape, dtype in specs:      # every shape and dtype first, then the devices
        _want(t, name, shape, dtype, None, check_device=False)
    for t, name, shape, dtype in specs:
        _want(t, name, shape, dtype, dev)
    _check(lib().mok_dispatch_index_noalloc(
        ctypes.byref(D), _ptr(topk_idx), _ptr(topk_w), _ptr(out["counts"]), _ptr(out["offsets"]),
        _ptr(out["sorted_tok"]), _ptr(out["sorted_w"]), _ptr(out["inv_pos"]), _stream()))
    return out


def mx_quantize_rows(src):
    """MXFP8 quantisation of a [rows, K] bf16 CUDA tensor along K: (codes uint8 [rows, K],
    UE8M0 scale bytes uint8 [rows, K/32])."""
    if src.dtype != torch.bfloat16 or not src.is_cuda or not src.is_contiguous() or src.dim() != 2:
        raise ValueError("src must be a contiguous 2-D bf16 CUDA tensor")
    rows, K = src.shape
    q = torch.empty((rows, K), dtype=torch.uint8, device=src.device)
    sc = torch.empty((rows, K // 32), dtype=torch.uint8, device=src.device)
    _check(lib().mok_mx_quantize_rows(rows, K, _ptr(src), _ptr(q), _ptr(sc), _stream()))
    return q, sc


_ELEM = {torch.bfloat16: 0, torch.float32: 1}   # mok_elem


def _elem(t, name):
    if t.dtype not in _ELEM:
        raise ValueError(f"{name}: dtype {t.dtype} is neither bfloat16 nor float32")
    return _ELEM[t.dtype]


def _scale_bytes(rows, K, layout):
    return (rows + 127) // 128 * 128 * (K // 32) if layout == "atoms" else rows * (K // 32)


def rms_norm(x, weight, eps=1e-6, residual=None, mx=None, want_y=True):
    """RMS norm of the rows of x [T,d] bf16, with the residual's addition: h = x + residual,
    v = h / sqrt(mean(h^2) + eps) * weight, in fp32.  residual [T,d] and weight [d] are bf16 or
    fp32.  Returns a dict: "y" (v in bf16; not with want_y=False), "residual" (h in residual's
    type, when there is one) and, with mx="rows" or "atoms", the MXFP8 form of v: "codes" uint8
    [T,d] and "scales" uint8 ([T,d/32], or the flat scale atoms that
    ``moe_forward(..., x_mx=(codes, scales))`` takes)."""
    if x.dim() != 2:
        raise ValueError("x must be 2-D")
    shape, dev = x.shape, x.device
    T, d = shape
    _want(x, "x", shape, torch.bfloat16, dev)
    _want(weight, "weight", (d,), weight.dtype, dev)
    y = torch.empty_like(x) if want_y else None
    h = codes = scales = None
    rt = 0
    if residual is not None:
        rt = _elem(residual, "residual")
        _want(residual, "residual", shape, residual.dtype, dev)
        h = torch.empty_like(residual)
    if mx is not None:
        if mx not in ("rows", "atoms"):
            raise ValueError("mx must be None, 'rows' or 'atoms'")
        codes = torch.empty(shape, dtype=torch.uint8, device=dev)
        scales = torch.empty((T, d // 32) if mx == "rows" else (_scale_bytes(T, d, mx),), dtype=torch.uint8,
                             device=dev)
    _check(lib().mok_rms_norm(T, d, eps, x.data_ptr(), _ptr(residual), rt, weight.data_ptr(), _elem(weight, "weight"),
                              _ptr(y), _ptr(h), _ptr(codes), _ptr(scales), 1 if mx == "atoms" else 0, _stream()))
    out = {}
    if want_y:
        out["y"] = y
    if h is not None:
        out["residual"] = h
    if codes is not None:
        out["codes"], out["scales"] = codes, scales
    return out


def rms_norm_workspace_size(T, d):
    n = lib().mok_rms_norm_workspace_size(T, d)
    if n == 0:
        raise MokError("unsupported norm dimensions")
    return n


def rms_norm_backward(dy, s, weight, eps=1e-6, dres=None, ws=None):
    """Gradients of :func:`rms_norm`: dy [T,d] bf16 of "y"; s the rows that were normalised (its
    "residual", or x when there was none); dres the gradient that arrives through "residual" (of
    s's type) or None.  Returns a dict: "dx" [T,d] bf16 (the gradient of x, and of a bf16
    residual), "dresidual" [T,d] fp32 when s is fp32, "dweight" [d] fp32.  ``ws``: at least
    rms_norm_workspace_size(T, d) bytes (allocated per call when None)."""
    if s.dim() != 2:
        raise ValueError("s must be 2-D")
    shape, dev = s.shape, s.device
    T, d = shape
    st = _elem(s, "s")
    _want(s, "s", shape, s.dtype, dev)
    _want(dy, "dy", shape, torch.bfloat16, dev)
    _want(weight, "weight", (d,), weight.dtype, dev)
    if dres is not None:
        _want(dres, "dres", shape, s.dtype, dev)
    if ws is None:
        ws = torch.empty(rms_norm_workspace_size(T, d), dtype=torch.uint8, device=dev)
    _want_ws(ws, dev)
    dx = torch.empty_like(dy)
    dweight = torch.empty((d,), dtype=torch.float32, device=dev)
    ds = torch.empty_like(s) if st else None
    _check(lib().mok_rms_norm_backward(T, d, eps, dy.data_ptr(), s.data_ptr(), st, weight.data_ptr(),
                                       _elem(weight, "weight"), _ptr(dres), dx.data_ptr(), _ptr(ds),
                                       dweight.data_ptr(), ws.data_ptr(), ws.numel(), _stream()))
    out = {"dx": dx, "dweight": dweight}
    if st:
        out["dresidual"] = ds
    return out


def balance_loss_workspace_size(D, n_seqs=1):
    n = lib().mok_balance_loss_workspace_size(ctypes.byref(D), n_seqs)
    if n == 0:
        raise MokError("unsupported layer dimensions")
    return n


def balance_loss(D, logits, topk_idx, ws, alpha, z_coef=0.0, seq_offsets=None, token_mask=None,
                 grad=None, want_dlogits=True):
    """Balance loss and z loss of the router (formulas in mok.h, mok_balance_loss) for logits
    [T,E] fp32 and topk_idx [T,k] int32 of :func:`route`.  ``seq_offsets`` int32 [S+1]: packed
    sequences, each balanced by itself (None: one); ``token_mask`` bool [T]: tokens that count;
    ``grad`` fp32 [1]: the upstream gradient (None: 1); ``ws``: a zeroed workspace of at least
    balance_loss_workspace_size(D, S) bytes, whose status word reports an index outside [0,E).
    Returns a dict: "loss" fp32 [2] (balance, z), "counts" int32 [S,E] and "dlogits" fp32 [T,E],
    which goes into ``moe_backward(..., dlogits_aux=...)``."""
    dev = logits.device
    _want(logits, "logits", (D.T, D.E), torch.float32, dev)
    _want(topk_idx, "topk_idx", (D.T, D.k), torch.int32, dev)
    S = 1
    if seq_offsets is not None:
        S = seq_offsets.numel() - 1
        _want(seq_offsets, "seq_offsets", (max(S, 1) + 1,), torch.int32, dev)
    if token_mask is not None:
        _want(token_mask, "token_mask", (D.T,), torch.bool, dev)
    if grad is not None:
        _want(grad, "grad", (1,), torch.float32, dev)
    _want_ws(ws, dev)
    loss = torch.empty((2,), dtype=torch.float32, device=dev)
    counts = torch.empty((S, D.E), dtype=torch.int32, device=dev)
    dlogits = torch.empty_like(logits) if want_dlogits else None
    _check(lib().mok_balance_loss(ctypes.byref(D), logits.data_ptr(), topk_idx.data_ptr(), _ptr(seq_offsets), S,
                                  _ptr(token_mask), alpha, z_coef, _ptr(grad), counts.data_ptr(), loss.data_ptr(),
                                  _ptr(dlogits), ws.data_ptr(), ws.numel(), _stream()))
    out = {"loss": loss, "counts": counts}
    if want_dlogits:
        out["dlogits"] = dlogits
    return out


def prepared_size(D):
    return lib().mok_prepared_size(ctypes.byref(D))


def prepare_weights(D, W):
    """MXFP8 / NVFP4: quantised copy of the expert weights in the layout of mok_prepare_weights
    (uint8 CUDA tensor); returns None for bf16.  Pass it as W["prepared"].  NVFP4: set the
    calibrated activation amaxes with :func:`nvfp4_set_activation_amax` afterwards."""
    n = prepared_size(D)
    if n == 0:
        return None
    buf = torch.empty(n, dtype=torch.uint8, device=W["W_gate"].device)
    Wd = dict(W)
    Wd["prepared"] = None
    Wd["prepared_bwd"] = None
    st = _weights_struct(D, Wd)
    _check(lib().mok_prepare_weights(ctypes.byref(D), ctypes.byref(st), _ptr(buf), _stream()))
    return buf


def nvfp4_set_activation_amax(D, prepared, amax_x, amax_h):
    """NVFP4: the calibrated tensor amaxes of x and h, written into ``prepared``."""
    _want(prepared, "prepared", (prepared_size(D),), torch.uint8, prepared.device)
    _check(lib().mok_nvfp4_set_activation_amax(ctypes.byref(D), _ptr(prepared), float(amax_x),
                                                float(amax_h), _stream()))


def prepare_weights_bwd(D, W):
    """MXFP8: the expert weights quantised along the backward GEMMs' reduction dimensions (uint8
    CUDA tensor); returns None for bf16.  Pass it as W["prepared_bwd"] for the MXFP8 backward."""
    n = lib().mok_prepared_bwd_size(ctypes.byref(D))
    if n == 0:
        return None
    buf = torch.empty(n, dtype=torch.uint8, device=W["W_gate"].device)
    Wd = dict(W)
    Wd["prepared"] = None
    Wd["prepared_bwd"] = None
    st = _weights_struct(D, Wd)
    _check(lib().mok_prepare_weights_bwd(ctypes.byref(D), ctypes.byref(st), _ptr(buf), _stream()))
    return buf


def moe_forward(D, W, x, routing, ws, saved=None, y=None, x_mx=None):
    """y[T,d] bf16 of the expert part for a routing from :func:`dispatch_index`.  ``x_mx``
    (MOK_MXFP8): x already quantised, (codes uint8 [T,d], scale atoms) as :func:`rms_norm` gives
    them with ``mx="atoms"``; the experts then read these instead of quantising x."""
    dev = x.device
    _want(x, "x", (D.T, D.d), torch.bfloat16, dev)
    ws_struct = _weights_struct(D, W)
    if y is None:
        y = torch.empty((D.T, D.d), dtype=torch.bfloat16, device=dev)
    if x_mx is not None:
        codes, atoms = x_mx
        _want(codes, "x_mx codes", (D.T, D.d), torch.uint8, dev)
        _want(atoms, "x_mx scales", (_scale_bytes(D.T, D.d, "atoms"),), torch.uint8, dev)
        _check(lib().mok_moe_forward_mx(
            ctypes.byref(D), ctypes.byref(ws_struct), _ptr(codes), _ptr(atoms),
            _ptr(routing["topk_idx"]), _ptr(routing["offsets"]), _ptr(routing["sorted_tok"]),
            _ptr(routing["sorted_w"]), _ptr(routing["inv_pos"]), _ptr(y), _ptr(saved), _ptr(ws),
            ws.numel(), _stream()))
        return y
    _check(lib().mok_moe_forward(
        ctypes.byref(D), ctypes.byref(ws_struct), _ptr(x), _ptr(routing["topk_idx"]),
        _ptr(routing["offsets"]), _ptr(routing["sorted_tok"]), _ptr(routing["sorted_w"]),
        _ptr(routing["inv_pos"]), _ptr(y), _ptr(saved), _ptr(ws), ws.numel(), _stream()))
    return y


def moe_backward(D, W, x, dY, saved, routing, ws, want_dW_router=True, dlogits_aux=None):
    """Gradients of the layer for upstream dY (selection held constant).  Returns a dict.
    ``dlogits_aux`` [T,E] fp32: a further gradient of the logits (from :func:`balance_loss`),
    included in dX, dW_router and dlogits."""
    dev = x.device
    bf = torch.bfloat16
    _want(dY, "dY", (D.T, D.d), bf, dev)
    if dlogits_aux is not None:
        _want(dlogits_aux, "dlogits_aux", (D.T, D.E), torch.float32, dev)
    ws_struct = _weights_struct(D, W)
    g = {
        "dX": torch.empty((D.T, D.d), dtype=bf, device=dev),
        "dW_gate": torch.empty((D.E, D.d, D.F), dtype=bf, device=dev),
        "dW_up": torch.empty((D.E, D.d, D.F), dtype=bf, device=dev),
        "dW_down": torch.empty((D.E, D.F, D.d), dtype=bf, device=dev),
        "dWs_gate": torch.empty((D.d, D.F_shared), dtype=bf, device=dev) if D.n_shared else None,
        "dWs_up": torch.empty((D.d, D.F_shared), dtype=bf, device=dev) if D.n_shared else None,
        "dWs_down": torch.empty((D.F_shared, D.d), dtype=bf, device=dev) if D.n_shared else None,
        "dlogits": torch.empty((D.T, D.E), dtype=torch.float32, device=dev),
        "dW_router": torch.empty((D.d, D.E), dtype=bf, device=dev) if want_dW_router else None,
    }
    r = routing
    _check(lib().mok_moe_backward_aux(
        ctypes.byref(D), ctypes.byref(ws_struct), _ptr(x), _ptr(dY), _ptr(saved), _ptr(r["topk_idx"]),
        _ptr(r["topk_w"]), _ptr(r["offsets"]), _ptr(r["sorted_tok"]), _ptr(r["sorted_w"]),
        _ptr(r["inv_pos"]), _ptr(dlogits_aux), _ptr(g["dX"]), _ptr(g["dW_gate"]), _ptr(g["dW_up"]), _ptr(g["dW_down"]),
        _ptr(g["dWs_gate"]), _ptr(g["dWs_up"]), _ptr(g["dWs_down"]), _ptr(g["dlogits"]),
        _ptr(g["dW_router"]), _ptr(ws), ws.numel(), _stream()))
    return g


def layer_forward_host(D, W, x_host, y_host, ws):
    """Whole-layer forward with x and y in (pinned) host memory; asynchronous on the current
    stream.  ``ws`` must hold workspace_size(D) + host_extra_size(D) bytes."""
    if x_host.is_cuda or y_host.is_cuda:
        raise ValueError("x_host and y_host must be host tensors")
    ws_struct = _weights_struct(D, W)
    _check(lib().mok_layer_forward_host(ctypes.byref(D), ctypes.byref(ws_struct), _ptr(x_host),
                                        _ptr(y_host), _ptr(ws), ws.numel(), _stream()))


def host_extra_size(D):
    return lib().mok_layer_host_extra_size(ctypes.byref(D))


class MoELayer:
    """Holds the weights of one layer and its workspaces; calls the C ABI in sequence.  ``backward``
    belongs to the last forward with training=True, whatever ran for inference since."""

    def __init__(self, D, W, device=None):
        self.D = D
        self.W = W
        dev = device or W["W_gate"].device
        self.ws = torch.zeros(workspace_size(D), dtype=torch.uint8, device=dev)
        self.saved = None
        self._trained = None  # the routing that ``saved`` belongs to
        self._ws_bwd = None

    def forward(self, x, training=False, x_mx=None, want_logits=False):
        idx, w, self.logits = route(self.D, x, self.W["W_router"], self.W.get("bias"), self.ws,
                                    want_logits)
        n = last_launch_count()
        routing = dispatch_index(self.D, idx, w, self.ws)
        n += last_launch_count()
        if training and self.saved is None:
            self.saved = torch.empty(saved_size(self.D), dtype=torch.uint8, device=x.device)
        if training:
            self._trained = None
        y = moe_forward(self.D, self.W, x, routing, self.ws, saved=self.saved if training else None,
                        x_mx=x_mx)
        self.last_launches = n + last_launch_count()  # kernels this call enqueued
        self.routing = routing
        if training:
            self._trained = routing
        return y

    def backward(self, x, dY, dlogits_aux=None):
        if self._trained is None:
            raise MokError("backward needs a forward with training=True")
        if self._ws_bwd is None:
            self._ws_bwd = torch.zeros(workspace_size(self.D, backward=True), dtype=torch.uint8,
                                       device=x.device)
        g = moe_backward(self.D, self.W, x, dY, self.saved, self._trained, self._ws_bwd,
                         dlogits_aux=dlogits_aux)
        self.last_launches = last_launch_count()
        return g


from .block import MoEBlock  # noqa: E402
from .optim import AdamW, TensorList, grad_norm, grad_norm_workspace_size  # noqa: E402
