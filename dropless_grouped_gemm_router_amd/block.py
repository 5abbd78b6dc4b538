"""Operators around the MoE layer (``include/moe_block.h``): layer norm, the
dense gated feed-forward block, products with 8-bit integer weights, products
with bias, activation and residual, the norms, gate and residual between two
blocks, and the router's balance loss; forward and, where they train, backward.

The ``moe_*`` functions have the C entry points' names and only marshal
arguments, as in ``binding``. The functions without that prefix take tensors:
they check shapes, types, contiguity and device on the host, launch on the
tensors' own device (its current stream unless one is given) and write into
buffers that were allocated once (``allocate_norm``, ``allocate_ffn``,
``allocate_linear_i8``, ``allocate_linear``, ``allocate_residual_norm``,
``allocate_balance_loss``). Tensors used on a stream other than their own have to
be ordered by the caller, as for every call of the library.
"""

from __future__ import annotations

import ctypes
from dataclasses import dataclass
from functools import cached_property, lru_cache
from typing import Dict, Optional

import torch

from . import binding
from .binding import (DTYPES, MOE_BF16, MOE_FP32, _check, _ptr, _stream, load as _load_library,
                      moe_routing, routing_struct)

MOE_I8 = 2
ACTS = {"silu": 0, "gelu": 1, "gelu_tanh": 2, "relu": 3}
LINEAR_ACTS = dict(ACTS, none=4)
NORM_KINDS = {"layer": 0, "rms": 1}
NORM_PARAMS = ("post_weight", "post_bias", "gate", "pre_weight", "pre_bias")

EXPORTED = ["moe_layer_norm", "moe_layer_norm_workspace_bytes", "moe_layer_norm_bwd",
            "moe_gated_ffn_workspace_bytes", "moe_gated_ffn_saved_bytes", "moe_gated_ffn",
            "moe_gated_ffn_bwd", "moe_i8_pitch", "moe_quantize_rows", "moe_quantize_weight",
            "moe_linear_i8_workspace_bytes", "moe_linear_i8",
            "moe_linear_workspace_bytes", "moe_linear_saved_bytes", "moe_linear_fwd", "moe_linear_bwd",
            "moe_residual_norm_fwd", "moe_residual_norm_workspace_bytes", "moe_residual_norm_bwd",
            "moe_balance_workspace_bytes", "moe_balance_saved_bytes", "moe_balance_loss",
            "moe_balance_loss_bwd"]


class moe_norm(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("width", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("eps", ctypes.c_float), ("ld_x", ctypes.c_int64), ("ld_y", ctypes.c_int64),
                ("ld_grad_out", ctypes.c_int64), ("ld_grad_x", ctypes.c_int64)]


class moe_ffn(ctypes.Structure):
    _fields_ = [("tokens", ctypes.c_int64), ("d_model", ctypes.c_int32),
                ("d_hidden", ctypes.c_int32), ("dtype", ctypes.c_int32), ("act", ctypes.c_int32),
                ("grad_dtype", ctypes.c_int32)]


class moe_i8_linear(ctypes.Structure):
    _fields_ = [("tokens", ctypes.c_int64)] + [(n, ctypes.c_int32) for n in (
        "inputs", "outputs", "x_dtype", "dtype", "groups", "top_k", "gather", "gated", "capacity")]


class moe_linear(ctypes.Structure):
    _fields_ = [("tokens", ctypes.c_int64)] + [(n, ctypes.c_int32) for n in (
        "inputs", "outputs", "dtype", "act", "grad_dtype")]


class moe_residual_norm(ctypes.Structure):
    _fields_ = ([("rows", ctypes.c_int64)]
                + [(n, ctypes.c_int32) for n in ("width", "dtype", "kind", "post", "pre")]
                + [("eps", ctypes.c_float), ("scale", ctypes.c_float)]
                + [("ld_" + n, ctypes.c_int64) for n in (
                    "z", "res", "out", "y", "grad_out", "grad_y", "grad_z", "grad_res")])


class moe_norm_params(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in NORM_PARAMS]


class moe_norm_grads(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in NORM_PARAMS]


class moe_balance(ctypes.Structure):
    _fields_ = ([("tokens", ctypes.c_int64)]
                + [(n, ctypes.c_int32) for n in ("experts", "top_k", "d_model", "dtype")]
                + [("balance", ctypes.c_float), ("z", ctypes.c_float)])


_lib = None


def load():
    """libmoe.so with the signatures of this header's entry points."""
    global _lib
    if _lib is not None:
        return _lib
    lib = _load_library()
    P, i32, i64, size = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    N, F, L = (ctypes.POINTER(t) for t in (moe_norm, moe_ffn, moe_i8_linear))
    D, R, S = (ctypes.POINTER(t) for t in (moe_linear, moe_residual_norm, moe_balance))
    W, G = ctypes.POINTER(moe_norm_params), ctypes.POINTER(moe_norm_grads)
    sig = {
        "moe_layer_norm": (ctypes.c_int, [N] + [P] * 7),
        "moe_layer_norm_workspace_bytes": (size, [N]),
        "moe_layer_norm_bwd": (ctypes.c_int, [N] + [P] * 9 + [size, P]),
        "moe_gated_ffn_workspace_bytes": (size, [F, ctypes.c_int]),
        "moe_gated_ffn_saved_bytes": (size, [F]),
        "moe_gated_ffn": (ctypes.c_int, [F] + [P] * 7 + [size, P]),
        "moe_gated_ffn_bwd": (ctypes.c_int, [F] + [P] * 11 + [size, P]),
        "moe_i8_pitch": (i64, [i32]),
        "moe_quantize_rows": (ctypes.c_int, [i64, i32, i32, P, i64, P, P, P]),
        "moe_quantize_weight": (ctypes.c_int, [i32, i32, i32, i32, P, i64, P, P, P]),
        "moe_linear_i8_workspace_bytes": (size, [L]),
        "moe_linear_i8": (ctypes.c_int, [L, P, P, P, P, P, ctypes.POINTER(moe_routing), P, P, size, P]),
        "moe_linear_workspace_bytes": (size, [D, ctypes.c_int]),
        "moe_linear_saved_bytes": (size, [D]),
        "moe_linear_fwd": (ctypes.c_int, [D] + [P] * 7 + [size, P]),
        "moe_linear_bwd": (ctypes.c_int, [D] + [P] * 8 + [size, P]),
        "moe_residual_norm_fwd": (ctypes.c_int, [R, P, P, W, P, P, P, P]),
        "moe_residual_norm_workspace_bytes": (size, [R]),
        "moe_residual_norm_bwd": (ctypes.c_int, [R, P, P, W] + [P] * 5 + [G, P, size, P]),
        "moe_balance_workspace_bytes": (size, [S]),
        "moe_balance_saved_bytes": (size, [S]),
        "moe_balance_loss": (ctypes.c_int, [S] + [P] * 9 + [size, P]),
        "moe_balance_loss_bwd": (ctypes.c_int, [S] + [P] * 4 + [ctypes.c_int] + [P] * 3 + [size, P]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


# ---------------------------------------------------------- C entry points

def _dtype(d) -> int:
    return DTYPES[d] if isinstance(d, str) else int(d)


def _nbytes(workspace, given: Optional[int]) -> int:
    if given is not None:
        return given
    return 0 if workspace is None else workspace.numel() * workspace.element_size()


def moe_layer_norm(n: moe_norm, x, weight, bias, y, mean, rstd, stream=None):
    _check(load().moe_layer_norm(ctypes.byref(n), _ptr(x), _ptr(weight), _ptr(bias), _ptr(y),
                                 _ptr(mean), _ptr(rstd), _stream(stream)), "moe_layer_norm")


def moe_layer_norm_workspace_bytes(n: moe_norm) -> int:
    return int(load().moe_layer_norm_workspace_bytes(ctypes.byref(n)))


def moe_layer_norm_bwd(n: moe_norm, x, weight, mean, rstd, grad_out, grad_x, grad_weight, grad_bias,
                       workspace, workspace_bytes: Optional[int] = None, stream=None):
    _check(load().moe_layer_norm_bwd(ctypes.byref(n), _ptr(x), _ptr(weight), _ptr(mean), _ptr(rstd),
                                     _ptr(grad_out), _ptr(grad_x), _ptr(grad_weight),
                                     _ptr(grad_bias), _ptr(workspace),
                                     _nbytes(workspace, workspace_bytes), _stream(stream)),
           "moe_layer_norm_bwd")


def moe_gated_ffn_workspace_bytes(f: moe_ffn, training: bool = False) -> int:
    return int(load().moe_gated_ffn_workspace_bytes(ctypes.byref(f), int(training)))


def moe_gated_ffn_saved_bytes(f: moe_ffn) -> int:
    return int(load().moe_gated_ffn_saved_bytes(ctypes.byref(f)))


def moe_gated_ffn(f: moe_ffn, x, w_gate, w_up, w_down, saved, out, workspace,
                  workspace_bytes: Optional[int] = None, stream=None):
    _check(load().moe_gated_ffn(ctypes.byref(f), _ptr(x), _ptr(w_gate), _ptr(w_up), _ptr(w_down),
                                _ptr(saved), _ptr(out), _ptr(workspace),
                                _nbytes(workspace, workspace_bytes), _stream(stream)), "moe_gated_ffn")


def moe_gated_ffn_bwd(f: moe_ffn, x, w_gate, w_up, w_down, saved, grad_out, grad_x, grad_gate,
                      grad_up, grad_down, workspace, workspace_bytes: Optional[int] = None,
                      stream=None):
    _check(load().moe_gated_ffn_bwd(ctypes.byref(f), _ptr(x), _ptr(w_gate), _ptr(w_up),
                                    _ptr(w_down), _ptr(saved), _ptr(grad_out), _ptr(grad_x),
                                    _ptr(grad_gate), _ptr(grad_up), _ptr(grad_down),
                                    _ptr(workspace), _nbytes(workspace, workspace_bytes),
                                    _stream(stream)), "moe_gated_ffn_bwd")


def moe_i8_pitch(width: int) -> int:
    return int(load().moe_i8_pitch(int(width)))


def moe_quantize_rows(rows: int, width: int, dtype, x, ld_x: int, q, scale, stream=None):
    _check(load().moe_quantize_rows(rows, width, _dtype(dtype), _ptr(x), ld_x, _ptr(q),
                                    _ptr(scale), _stream(stream)), "moe_quantize_rows")


def moe_quantize_weight(groups: int, width: int, outputs: int, dtype, w, q_rows: int, q, scale,
                        stream=None):
    _check(load().moe_quantize_weight(groups, width, outputs, _dtype(dtype), _ptr(w), q_rows,
                                      _ptr(q), _ptr(scale), _stream(stream)), "moe_quantize_weight")


def moe_linear_i8_workspace_bytes(l: moe_i8_linear) -> int:
    return int(load().moe_linear_i8_workspace_bytes(ctypes.byref(l)))


def moe_linear_i8(l: moe_i8_linear, x, x_scale, wq, w_scale, bias, routing: Optional[Dict], y,
                  workspace, workspace_bytes: Optional[int] = None, stream=None):
    r = None if routing is None else ctypes.byref(routing_struct(routing))
    _check(load().moe_linear_i8(ctypes.byref(l), _ptr(x), _ptr(x_scale), _ptr(wq), _ptr(w_scale),
                                _ptr(bias), r, _ptr(y), _ptr(workspace),
                                _nbytes(workspace, workspace_bytes), _stream(stream)),
           "moe_linear_i8")


def moe_linear_workspace_bytes(l: moe_linear, training: bool = False) -> int:
    return int(load().moe_linear_workspace_bytes(ctypes.byref(l), int(training)))


def moe_linear_saved_bytes(l: moe_linear) -> int:
    return int(load().moe_linear_saved_bytes(ctypes.byref(l)))


def moe_linear_fwd(l: moe_linear, x, w, bias, residual, saved, y, workspace,
                   workspace_bytes: Optional[int] = None, stream=None):
    _check(load().moe_linear_fwd(ctypes.byref(l), _ptr(x), _ptr(w), _ptr(bias), _ptr(residual),
                                 _ptr(saved), _ptr(y), _ptr(workspace),
                                 _nbytes(workspace, workspace_bytes), _stream(stream)),
           "moe_linear_fwd")


def moe_linear_bwd(l: moe_linear, x, w, saved, grad_out, grad_x, grad_w, grad_bias, workspace,
                   workspace_bytes: Optional[int] = None, stream=None):
    _check(load().moe_linear_bwd(ctypes.byref(l), _ptr(x), _ptr(w), _ptr(saved), _ptr(grad_out),
                                 _ptr(grad_x), _ptr(grad_w), _ptr(grad_bias), _ptr(workspace),
                                 _nbytes(workspace, workspace_bytes), _stream(stream)),
           "moe_linear_bwd")


def norm_params_struct(params: Dict) -> moe_norm_params:
    return moe_norm_params(*[_ptr(params.get(n)) for n in NORM_PARAMS])


def norm_grads_struct(grads: Dict) -> moe_norm_grads:
    return moe_norm_grads(*[_ptr(grads.get(n)) for n in NORM_PARAMS])


def moe_residual_norm_fwd(n: moe_residual_norm, z, res, params: Dict, out, y, stats, stream=None):
    p = norm_params_struct(params)
    _check(load().moe_residual_norm_fwd(ctypes.byref(n), _ptr(z), _ptr(res), ctypes.byref(p),
                                        _ptr(out), _ptr(y), _ptr(stats), _stream(stream)),
           "moe_residual_norm_fwd")


def moe_residual_norm_workspace_bytes(n: moe_residual_norm) -> int:
    return int(load().moe_residual_norm_workspace_bytes(ctypes.byref(n)))


def moe_residual_norm_bwd(n: moe_residual_norm, z, res, params: Dict, stats, grad_out, grad_y, grad_z,
                          grad_res, grads: Dict, workspace, workspace_bytes: Optional[int] = None,
                          stream=None):
    p, g = norm_params_struct(params), norm_grads_struct(grads)
    _check(load().moe_residual_norm_bwd(ctypes.byref(n), _ptr(z), _ptr(res), ctypes.byref(p),
                                        _ptr(stats), _ptr(grad_out), _ptr(grad_y), _ptr(grad_z),
                                        _ptr(grad_res), ctypes.byref(g), _ptr(workspace),
                                        _nbytes(workspace, workspace_bytes), _stream(stream)),
           "moe_residual_norm_bwd")


def moe_balance_workspace_bytes(b: moe_balance) -> int:
    return int(load().moe_balance_workspace_bytes(ctypes.byref(b)))


def moe_balance_saved_bytes(b: moe_balance) -> int:
    return int(load().moe_balance_saved_bytes(ctypes.byref(b)))


def moe_balance_loss(b: moe_balance, x, w_router, topk_idx, mask, counts, mean_prob, loss, saved,
                     workspace, workspace_bytes: Optional[int] = None, stream=None):
    _check(load().moe_balance_loss(ctypes.byref(b), _ptr(x), _ptr(w_router), _ptr(topk_idx),
                                   _ptr(mask), _ptr(counts), _ptr(mean_prob), _ptr(loss), _ptr(saved),
                                   _ptr(workspace), _nbytes(workspace, workspace_bytes),
                                   _stream(stream)), "moe_balance_loss")


def moe_balance_loss_bwd(b: moe_balance, x, mask, saved, grad_loss, add: bool, grad_x, grad_router,
                         workspace, workspace_bytes: Optional[int] = None, stream=None):
    _check(load().moe_balance_loss_bwd(ctypes.byref(b), _ptr(x), _ptr(mask), _ptr(saved),
                                       _ptr(grad_loss), int(add), _ptr(grad_x), _ptr(grad_router),
                                       _ptr(workspace), _nbytes(workspace, workspace_bytes),
                                       _stream(stream)),
           "moe_balance_loss_bwd")


# ------------------------------------------------------------ tensor checks
#
# These run on every call, in front of kernels that take a few microseconds:
# a tensor that fits costs one expression, and the problem structs of the C
# calls are kept by their values.

_TORCH = {"fp32": torch.float32, "bf16": torch.bfloat16, MOE_FP32: torch.float32,
          MOE_BF16: torch.bfloat16}
_CODE = {torch.float32: MOE_FP32, torch.bfloat16: MOE_BF16}


def _refuse(name, t, shape, dtype, device, strided=False):
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype != dtype:
        raise ValueError(f"{name}: {t.dtype}, expected {dtype}")
    if t.device != device:
        raise ValueError(f"{name}: on {t.device}, expected {device}")
    if strided:
        raise ValueError(f"{name}: rows have to be contiguous and apart, strides {t.stride()}")
    raise ValueError(f"{name}: has to be contiguous")


def _want(name, t, shape, dtype, device):
    """``t`` is a contiguous tensor of this shape, type and device."""
    if t.shape != shape or t.dtype is not dtype or t.device != device or not t.is_contiguous():
        _refuse(name, t, shape, dtype, device)


def _want_rows(name, t, shape, dtype, device) -> int:
    """``t`` is a matrix of this shape, type and device whose rows are
    contiguous and do not overlap; returns the elements between rows."""
    if t.shape != shape or t.dtype is not dtype or t.device != device:
        _refuse(name, t, shape, dtype, device)
    if t.is_contiguous():
        return shape[1]
    row, col = t.stride()
    if shape[1] > 1 and col != 1 or shape[0] > 1 and row < shape[1]:
        _refuse(name, t, shape, dtype, device, strided=True)
    return row if shape[0] > 1 else shape[1]


def _want_bytes(name, t, least, device):
    """``t`` is a contiguous buffer of bytes on this device, of ``least`` or more."""
    if t.dtype is torch.uint8 and t.device == device and t.numel() >= least and t.is_contiguous():
        return
    if t.numel() < least:
        raise ValueError(f"{name}: {t.numel()} bytes, {least} are needed: allocated for another problem?")
    _refuse(name, t, t.shape, torch.uint8, device)


def _code(t) -> int:
    if t.dtype not in _CODE:
        raise ValueError(f"{t.dtype}: float32 or bfloat16 is supported")
    return _CODE[t.dtype]


def _want_gpu(device):
    if device.type != "cuda":
        raise ValueError(f"tensors have to be on a GPU, not on {device}")


def _run(where, device, stream, fn, *args):
    """fn(*args, stream) on the tensors' device."""
    index = device.index
    if index is None:  # a GPU's tensors have one
        _want_gpu(device)
    # the raw handles: a tenth of the time of making a torch.cuda.Stream, half of asking
    # torch.cuda for the current device
    s = torch._C._cuda_getCurrentRawStream(index) if stream is None else _stream(stream)
    if torch._C._cuda_getDevice() != index:
        with torch.cuda.device(device):
            status = fn(*args, s)
    else:
        status = fn(*args, s)
    if status:
        _check(status, where)


def _device(device):
    d = torch.device(device)
    if d.type == "cuda" and d.index is None:
        d = torch.device("cuda", torch.cuda.current_device())
    return d


# ---------------------------------------------------------------- layer norm

@dataclass
class NormBuffers:
    """Device buffers of one layer norm, allocated once."""

    y: object
    mean: object
    rstd: object
    grad_x: Optional[object] = None
    grad_weight: Optional[object] = None
    grad_bias: Optional[object] = None
    workspace: Optional[object] = None
    # what allocate_norm made, with its shape, type and device: tensors put in
    # their place are checked on every call, these are known to fit
    made: Optional[tuple] = None


@lru_cache(maxsize=256)
def _norm(*fields):
    n = moe_norm(*fields)
    return n, ctypes.byref(n)


def allocate_norm(rows: int, width: int, dtype, device="cuda", training: bool = False) -> NormBuffers:
    dt, device = _TORCH[dtype], _device(device)
    f32 = dict(dtype=torch.float32, device=device)
    b = NormBuffers(y=torch.empty((rows, width), dtype=dt, device=device),
                    mean=torch.empty(rows, **f32), rstd=torch.empty(rows, **f32))
    if training:
        nws = moe_layer_norm_workspace_bytes(moe_norm(rows, width, _dtype(dtype), 0.0, 0, 0, 0, 0))
        b.grad_x = torch.empty((rows, width), dtype=dt, device=device)
        b.grad_weight, b.grad_bias = torch.empty(width, **f32), torch.empty(width, **f32)
        b.workspace = torch.empty(nws, dtype=torch.uint8, device=device)
    b.made = (b.y.shape, dt, device, b.y, b.mean, b.rstd, b.grad_x, b.grad_weight, b.grad_bias, b.workspace)
    return b


def layer_norm(x, weight, bias, eps: float, buf: NormBuffers, stream=None):
    """Layer norm over the rows of x [rows, width] (rows may be strided);
    weight and bias are fp32 or None. Returns buf.y, with buf.mean and
    buf.rstd kept for the backward pass."""
    if x.dim() != 2:
        raise ValueError(f"x: a matrix is expected, not {x.dim()} dimensions")
    shape, dt, dev, f32 = x.shape, x.dtype, x.device, torch.float32
    rows, width = shape
    ld_x = _want_rows("x", x, shape, dt, dev)
    if weight is not None:
        _want("weight", weight, (width,), f32, dev)
    if bias is not None:
        _want("bias", bias, (width,), f32, dev)
    y, mean, rstd, m = buf.y, buf.mean, buf.rstd, buf.made
    if m and y is m[3] and mean is m[4] and rstd is m[5] and m[0] == shape and m[1] is dt and m[2] == dev:
        ld_y = width
    else:
        ld_y = _want_rows("y", y, shape, dt, dev)
        _want("mean", mean, (rows,), f32, dev)
        _want("rstd", rstd, (rows,), f32, dev)
    n = _norm(rows, width, _code(x), eps, ld_x, ld_y, 0, 0)
    _run("moe_layer_norm", dev, stream, load().moe_layer_norm, n[1], x.data_ptr(),
         None if weight is None else weight.data_ptr(), None if bias is None else bias.data_ptr(),
         y.data_ptr(), mean.data_ptr(), rstd.data_ptr())
    return y


def layer_norm_backward(x, weight, grad_out, buf: NormBuffers, stream=None):
    """Gradients of sum(y * grad_out) after ``layer_norm`` with the same
    buffers: (grad_x, grad_weight, grad_bias), the last two in fp32."""
    shape, dt, dev, f32 = x.shape, x.dtype, x.device, torch.float32
    rows, width = shape
    gx, gw, gb = buf.grad_x, buf.grad_weight, buf.grad_bias
    if gx is None:
        raise ValueError("the buffers were allocated without training=True")
    ld_x = _want_rows("x", x, shape, dt, dev)
    ld_go = _want_rows("grad_out", grad_out, shape, dt, dev)
    if weight is not None:
        _want("weight", weight, (width,), f32, dev)
    m = buf.made
    if (m and gx is m[6] and gw is m[7] and gb is m[8] and buf.mean is m[4] and buf.rstd is m[5]
            and buf.workspace is m[9] and m[0] == shape and m[1] is dt and m[2] == dev):
        ld_gx = width
    else:
        ld_gx = _want_rows("grad_x", gx, shape, dt, dev)
        _want("mean", buf.mean, (rows,), f32, dev)
        _want("rstd", buf.rstd, (rows,), f32, dev)
        _want("grad_weight", gw, (width,), f32, dev)
        _want("grad_bias", gb, (width,), f32, dev)
        _want_bytes("workspace", buf.workspace, 0, dev)
    n = _norm(rows, width, _code(x), 0.0, ld_x, 0, ld_go, ld_gx)
    _run("moe_layer_norm_bwd", dev, stream, load().moe_layer_norm_bwd, n[1], x.data_ptr(),
         None if weight is None else weight.data_ptr(), buf.mean.data_ptr(), buf.rstd.data_ptr(), grad_out.data_ptr(), gx.data_ptr(),
         gw.data_ptr(), gb.data_ptr(), buf.workspace.data_ptr(), buf.workspace.numel())
    return gx, gw, gb


# -------------------------------------------------- gated feed-forward block

@dataclass(frozen=True)
class GatedFfn:
    """A dense gated feed-forward block: out = (act(x W_gate) * (x W_up)) W_down."""

    tokens: int
    d_model: int
    d_hidden: int
    dtype: str = "bf16"
    act: str = "silu"
    grad_dtype: str = "fp32"  # of the weight gradients: fp32, or dtype

    @property
    def _fields(self):
        return (self.tokens, self.d_model, self.d_hidden, DTYPES[self.dtype], ACTS[self.act],
                DTYPES[self.grad_dtype])

    def struct(self) -> moe_ffn:
        """The C problem, the caller's own to change."""
        return moe_ffn(*self._fields)


@lru_cache(maxsize=256)
def _ffn(*fields):
    f = moe_ffn(*fields)
    return f, ctypes.byref(f), moe_gated_ffn_saved_bytes(f)


@dataclass
class FfnBuffers:
    """Device buffers of one block, allocated once."""

    out: object
    workspace: object
    saved: Optional[object] = None
    grad_x: Optional[object] = None
    grads: Optional[Dict] = None


def allocate_ffn(f: GatedFfn, device="cuda", training: bool = False) -> FfnBuffers:
    dt, device, c = _TORCH[f.dtype], _device(device), f.struct()
    nws, nsv = moe_gated_ffn_workspace_bytes(c, training), moe_gated_ffn_saved_bytes(c)
    if nws == 0:
        raise ValueError(f"unsupported problem {f}")
    b = FfnBuffers(out=torch.empty((f.tokens, f.d_model), dtype=dt, device=device),
                   workspace=torch.empty(nws, dtype=torch.uint8, device=device))
    if training:
        g = dict(dtype=_TORCH[f.grad_dtype], device=device)
        b.saved = torch.empty(nsv, dtype=torch.uint8, device=device)
        b.grad_x = torch.empty((f.tokens, f.d_model), dtype=dt, device=device)
        b.grads = dict(w_gate=torch.empty((f.d_model, f.d_hidden), **g),
                       w_up=torch.empty((f.d_model, f.d_hidden), **g),
                       w_down=torch.empty((f.d_hidden, f.d_model), **g))
    return b


def _want_ffn(f, x, weights):
    dt, dev = _TORCH[f.dtype], x.device
    up = (f.d_model, f.d_hidden)
    wg, wu, wd = weights["w_gate"], weights["w_up"], weights["w_down"]
    _want("x", x, (f.tokens, f.d_model), dt, dev)
    _want("w_gate", wg, up, dt, dev)
    _want("w_up", wu, up, dt, dev)
    _want("w_down", wd, up[::-1], dt, dev)
    _, c, nsv = _ffn(*f._fields)
    return dt, dev, c, nsv, wg.data_ptr(), wu.data_ptr(), wd.data_ptr()


def _want_saved(buf, least, device):
    # the library is not told this buffer's size
    if buf.saved is None:
        raise ValueError("the buffers were allocated without training=True")
    _want_bytes("saved", buf.saved, least, device)


def gated_ffn(f: GatedFfn, x, weights: Dict, buf: FfnBuffers, training: bool = False, stream=None):
    """The block's forward pass (weights: w_gate, w_up, w_down); returns buf.out."""
    dt, dev, c, nsv, wg, wu, wd = _want_ffn(f, x, weights)
    _want("out", buf.out, (f.tokens, f.d_model), dt, dev)
    _want_bytes("workspace", buf.workspace, 0, dev)
    if training:
        _want_saved(buf, nsv, dev)
    _run("moe_gated_ffn", dev, stream, load().moe_gated_ffn, c, x.data_ptr(), wg, wu, wd,
         buf.saved.data_ptr() if training else None, buf.out.data_ptr(), buf.workspace.data_ptr(),
         buf.workspace.numel())
    return buf.out


def gated_ffn_backward(f: GatedFfn, x, weights: Dict, grad_out, buf: FfnBuffers, stream=None):
    """Gradients of sum(out * grad_out) after ``gated_ffn(..., training=True)``:
    (grad_x, {w_gate, w_up, w_down})."""
    dt, dev, c, nsv, wg, wu, wd = _want_ffn(f, x, weights)
    _want_saved(buf, nsv, dev)
    _want_bytes("workspace", buf.workspace, 0, dev)
    _want("grad_out", grad_out, (f.tokens, f.d_model), dt, dev)
    _want("grad_x", buf.grad_x, (f.tokens, f.d_model), dt, dev)
    g, gdt = buf.grads, _TORCH[f.grad_dtype]
    for name in ("w_gate", "w_up", "w_down"):
        _want("gradient of " + name, g[name], weights[name].shape, gdt, dev)
    _run("moe_gated_ffn_bwd", dev, stream, load().moe_gated_ffn_bwd, c, x.data_ptr(), wg, wu, wd,
         buf.saved.data_ptr(), grad_out.data_ptr(), buf.grad_x.data_ptr(), g["w_gate"].data_ptr(),
         g["w_up"].data_ptr(), g["w_down"].data_ptr(), buf.workspace.data_ptr(), buf.workspace.numel())
    return buf.grad_x, g


# ------------------------------------------------- products in 8-bit integers

@dataclass(frozen=True)
class LinearI8:
    """A product with weights in 8-bit integers, dense (groups 1) or grouped by
    the layer's routing; see moe_linear_i8."""

    tokens: int
    inputs: int
    outputs: int  # weight rows of a group; when gated, gate rows then up rows
    dtype: str = "bf16"  # of the output
    groups: int = 1
    top_k: int = 1
    gated: bool = False
    sorted_input: bool = False  # routed: x rows are in expert order, not tokens
    capacity: int = 0

    @property
    def rows(self) -> int:
        return self.tokens * self.top_k

    @property
    def columns(self) -> int:
        return self.outputs // 2 if self.gated else self.outputs

    @property
    def input_rows(self) -> int:
        return self.rows if self.sorted_input else self.tokens

    def struct(self, x_dtype: int, routed: bool) -> moe_i8_linear:
        """The C problem, the caller's own to change."""
        return moe_i8_linear(self.tokens, self.inputs, self.outputs, x_dtype, DTYPES[self.dtype],
                             self.groups, self.top_k, int(routed and not self.sorted_input),
                             int(self.gated), self.capacity)


@lru_cache(maxsize=256)
def _i8(l, x_dtype, routed):
    c = l.struct(x_dtype, routed)
    return c, ctypes.byref(c), moe_i8_pitch(l.inputs)


@dataclass
class I8Buffers:
    """Device buffers of one product, allocated once."""

    y: object
    workspace: object


def allocate_linear_i8(l: LinearI8, device="cuda") -> I8Buffers:
    device = _device(device)
    nws = moe_linear_i8_workspace_bytes(l.struct(MOE_FP32, l.groups > 1))
    if nws == 0:
        raise ValueError(f"unsupported problem {l}")
    return I8Buffers(y=torch.empty((l.rows, l.columns), dtype=_TORCH[l.dtype], device=device),
                     workspace=torch.empty(nws, dtype=torch.uint8, device=device))


def quantize_rows(x, q=None, scale=None, stream=None):
    """Rows of x [rows, width] as (q int8 [rows, pitch], scale fp32 [rows])."""
    rows, width = x.shape
    dev = x.device
    ld = _want_rows("x", x, x.shape, x.dtype, dev)
    pitch = moe_i8_pitch(width)
    q = torch.empty((rows, pitch), dtype=torch.int8, device=dev) if q is None else q
    scale = torch.empty(rows, dtype=torch.float32, device=dev) if scale is None else scale
    _want("q", q, (rows, pitch), torch.int8, dev)
    _want("scale", scale, (rows,), torch.float32, dev)
    _run("moe_quantize_rows", dev, stream, load().moe_quantize_rows, rows, width, _code(x),
         x.data_ptr(), ld, q.data_ptr(), scale.data_ptr())
    return q, scale


def quantize_weights(*parts, stream=None):
    """Weights [groups, width, outputs] (or one matrix [width, outputs]) as
    (q int8 [groups, rows, pitch], scale fp32 [groups, rows]); several parts of
    one shape (gate and up) follow each other in a group's rows."""
    parts = [w[None] if w.dim() == 2 else w for w in parts]
    groups, width, outputs = parts[0].shape
    dev, rows = parts[0].device, outputs * len(parts)
    pitch = moe_i8_pitch(width)
    q = torch.empty((groups, rows, pitch), dtype=torch.int8, device=dev)
    scale = torch.empty((groups, rows), dtype=torch.float32, device=dev)
    for i, w in enumerate(parts):
        _want("weights", w, (groups, width, outputs), parts[0].dtype, dev)
        _run("moe_quantize_weight", dev, stream, load().moe_quantize_weight, groups, width, outputs,
             _code(w), w.data_ptr(), rows, q[:, i * outputs:].data_ptr(), scale[:, i * outputs:].data_ptr())
    return q, scale


def linear_i8(l: LinearI8, x, wq, w_scale, buf: I8Buffers, bias=None, routing: Optional[Dict] = None,
              x_scale=None, stream=None):
    """The product; x is fp32 or bf16 [rows, inputs] (quantised within the
    call) or int8 [rows, pitch] with x_scale. Returns buf.y."""
    dev, xdt, xs = x.device, x.dtype, None
    whole = xdt is torch.int8
    _, c, pitch = _i8(l, MOE_I8 if whole else _code(x), routing is not None)
    _want("x", x, (l.input_rows, pitch if whole else l.inputs), xdt, dev)
    if whole:
        if x_scale is None:
            raise ValueError("an int8 input needs x_scale")
        _want("x_scale", x_scale, (l.input_rows,), torch.float32, dev)
        xs = x_scale.data_ptr()
    _want("weights", wq, (l.groups, l.outputs, pitch), torch.int8, dev)
    _want("weight scales", w_scale, (l.groups, l.outputs), torch.float32, dev)
    if bias is not None:
        _want("bias", bias, (l.outputs,), torch.float32, dev)
    r = None
    if routing is not None:
        _want("expert_offsets", routing["expert_offsets"], (l.groups + 1,), torch.int32, dev)
        if not l.sorted_input:
            _want("perm", routing["perm"], (l.rows,), torch.int32, dev)
        r = ctypes.byref(routing_struct(routing))
    y = buf.y
    _want("y", y, (l.rows, l.columns), _TORCH[l.dtype], dev)
    _want_bytes("workspace", buf.workspace, 0, dev)
    _run("moe_linear_i8", dev, stream, load().moe_linear_i8, c, x.data_ptr(), xs, wq.data_ptr(),
         w_scale.data_ptr(), _ptr(bias), r, y.data_ptr(), buf.workspace.data_ptr(),
         buf.workspace.numel())
    return y


class _Planned:
    """A problem that keeps its C struct and what its calls compare with once it
    has been used (``_plan``): a copy or a pickle is of the problem alone."""

    def __getstate__(self):
        return {k: v for k, v in vars(self).items() if k != "_plan"}


# ----------------------------------- products with bias, activation and residual

@dataclass(frozen=True)
class Linear(_Planned):
    """A dense product with its epilogue: y = act(x W + bias) + residual."""

    tokens: int
    inputs: int
    outputs: int
    dtype: str = "bf16"
    act: str = "none"
    grad_dtype: str = "fp32"  # of the weights' gradient: fp32, or dtype

    @property
    def _fields(self):
        return (self.tokens, self.inputs, self.outputs, DTYPES[self.dtype], LINEAR_ACTS[self.act],
                DTYPES[self.grad_dtype])

    def struct(self) -> moe_linear:
        """The C problem, the caller's own to change."""
        return moe_linear(*self._fields)

    @cached_property
    def _plan(self):
        c = self.struct()
        return (ctypes.byref(c), moe_linear_saved_bytes(c), torch.Size((self.tokens, self.inputs)),
                torch.Size((self.inputs, self.outputs)), torch.Size((self.tokens, self.outputs)),
                torch.Size((self.outputs,)), _TORCH[self.dtype])


@dataclass
class LinearBuffers:
    """Device buffers of one product, allocated once."""

    y: object
    workspace: object
    saved: Optional[object] = None  # training, with an activation
    grad_x: Optional[object] = None
    grad_w: Optional[object] = None
    grad_bias: Optional[object] = None


def allocate_linear(l: Linear, device="cuda", training: bool = False) -> LinearBuffers:
    dt, device, c = _TORCH[l.dtype], _device(device), l.struct()
    nws = moe_linear_workspace_bytes(c, training)
    if nws == 0:
        raise ValueError(f"unsupported problem {l}")
    b = LinearBuffers(y=torch.empty((l.tokens, l.outputs), dtype=dt, device=device),
                      workspace=torch.empty(nws, dtype=torch.uint8, device=device))
    if training:
        b.saved = torch.empty(moe_linear_saved_bytes(c), dtype=torch.uint8, device=device)
        b.grad_x = torch.empty((l.tokens, l.inputs), dtype=dt, device=device)
        b.grad_w = torch.empty((l.inputs, l.outputs), dtype=_TORCH[l.grad_dtype], device=device)
        b.grad_bias = torch.empty(l.outputs, dtype=torch.float32, device=device)
    return b


def linear(l: Linear, x, w, buf: LinearBuffers, bias=None, residual=None, training: bool = False,
           stream=None):
    """The product of x [tokens, inputs] and w [inputs, outputs] with its
    epilogue; bias is fp32. Returns buf.y, which may not be the residual's memory."""
    c, nsv, xs, ws, ys, bs, dt = l._plan
    dev, y = x.device, buf.y
    _want("x", x, xs, dt, dev)
    _want("w", w, ws, dt, dev)
    if bias is not None:
        _want("bias", bias, bs, torch.float32, dev)
    if residual is not None:
        _want("residual", residual, ys, dt, dev)
    _want("y", y, ys, dt, dev)
    out, add = y.data_ptr(), None if residual is None else residual.data_ptr()
    if add == out and l.tokens:  # the library refuses whatever else is shared
        raise ValueError("residual: is the buffer of y; rows are stored while others are still read")
    _want_bytes("workspace", buf.workspace, 0, dev)
    if training:
        _want_saved(buf, nsv, dev)
    _run("moe_linear_fwd", dev, stream, load().moe_linear_fwd, c, x.data_ptr(), w.data_ptr(),
         None if bias is None else bias.data_ptr(), add, buf.saved.data_ptr() if training else None, out,
         buf.workspace.data_ptr(), buf.workspace.numel())
    return y


def linear_backward(l: Linear, x, w, grad_out, buf: LinearBuffers, bias: bool = True, stream=None):
    """Gradients of sum(y * grad_out) after ``linear(..., training=True)`` with
    the same buffers: (grad_x, grad_w, grad_bias), the last None where bias is
    False; the residual's gradient is grad_out."""
    if not isinstance(bias, bool):
        raise ValueError("bias: True or False, whether its gradient is wanted")
    c, nsv, xs, ws, ys, bs, dt = l._plan
    dev = x.device
    _want("x", x, xs, dt, dev)
    _want("w", w, ws, dt, dev)
    _want_saved(buf, nsv, dev)
    _want("grad_out", grad_out, ys, dt, dev)
    _want("grad_x", buf.grad_x, xs, dt, dev)
    _want("gradient of w", buf.grad_w, ws, _TORCH[l.grad_dtype], dev)
    if bias:
        _want("gradient of bias", buf.grad_bias, bs, torch.float32, dev)
    _want_bytes("workspace", buf.workspace, 0, dev)
    _run("moe_linear_bwd", dev, stream, load().moe_linear_bwd, c, x.data_ptr(), w.data_ptr(),
         buf.saved.data_ptr(), grad_out.data_ptr(), buf.grad_x.data_ptr(), buf.grad_w.data_ptr(),
         buf.grad_bias.data_ptr() if bias else None, buf.workspace.data_ptr(), buf.workspace.numel())
    return buf.grad_x, buf.grad_w, buf.grad_bias if bias else None


# ---------------------------------------------------------- between two blocks

@dataclass(frozen=True)
class ResidualNorm(_Planned):
    """What lies between two blocks: out = scale res + gate (norm(z) post_weight
    + post_bias), y = norm(out) pre_weight + pre_bias; without post the block's
    output z is added as it is, without pre there is no y."""

    rows: int
    width: int
    dtype: str = "bf16"
    kind: str = "layer"  # of both norms: layer or rms
    eps: float = 1e-5
    scale: float = 1.0
    post: bool = True
    pre: bool = True

    def struct(self, *lds) -> moe_residual_norm:
        """The C problem, the caller's own to change."""
        return moe_residual_norm(self.rows, self.width, DTYPES[self.dtype], NORM_KINDS[self.kind],
                                 int(self.post), int(self.pre), self.eps, self.scale, *lds)

    @cached_property
    def _plan(self):
        # what every call compares with, and the C problem of contiguous matrices
        return (torch.Size((self.rows, self.width)), torch.Size((4, self.rows)), torch.Size((self.width,)),
                _TORCH[self.dtype], ctypes.byref(self.struct()))


@lru_cache(maxsize=256)
def _step(n, *lds):
    return ctypes.byref(n.struct(*lds))


@dataclass
class ResidualNormBuffers:
    """Device buffers of one step, allocated once."""

    out: object
    y: Optional[object]
    stats: object
    grad_z: Optional[object] = None
    grad_res: Optional[object] = None
    grads: Optional[Dict] = None
    workspace: Optional[object] = None
    # what allocate_residual_norm made, with its problem and device: as NormBuffers.made
    made: Optional[tuple] = None


def allocate_residual_norm(n: ResidualNorm, device="cuda", training: bool = False) -> ResidualNormBuffers:
    dt, device = _TORCH[n.dtype], _device(device)
    nws = moe_residual_norm_workspace_bytes(n.struct())
    if nws == 0:
        raise ValueError(f"unsupported problem {n}")
    f32 = dict(dtype=torch.float32, device=device)

    def matrix():
        return torch.empty((n.rows, n.width), dtype=dt, device=device)

    b = ResidualNormBuffers(out=matrix(), y=matrix() if n.pre else None, stats=torch.empty((4, n.rows), **f32))
    if training:
        b.grad_z, b.grad_res = matrix(), matrix()
        b.grads = {name: torch.empty(n.width, **f32) for name in NORM_PARAMS}
        b.workspace = torch.empty(nws, dtype=torch.uint8, device=device)
    b.made = (n, device, b.out, b.y, b.stats, b.grad_z, b.grad_res, b.workspace)
    return b


def _step_params(params, shape, dev, struct=moe_norm_params):
    f32, ptrs = torch.float32, []
    for name in NORM_PARAMS:
        t = params.get(name)
        if t is not None:
            if t.shape != shape or t.dtype is not f32 or t.device != dev or not t.is_contiguous():
                _refuse(name, t, shape, f32, dev)
            t = t.data_ptr()
        ptrs.append(t)
    return struct(*ptrs)


def _fits(t, shape, dt, dev):
    return t.shape == shape and t.dtype is dt and t.device == dev and t.is_contiguous()


def residual_norm(n: ResidualNorm, z, res, params: Dict, buf: ResidualNormBuffers, stream=None):
    """The step from a block's output z and the residual res [rows, width]
    (rows may be strided); params may hold post_weight, post_bias, gate,
    pre_weight and pre_bias (fp32). Returns (buf.out, buf.y), with buf.stats
    kept for the backward pass."""
    _run("moe_residual_norm_fwd", z.device, stream, load().moe_residual_norm_fwd,
         *_step_forward(n, z, res, params, buf))
    return buf.out, buf.y if n.pre else None


def _step_forward(n, z, res, params, buf):
    """The checked arguments of residual_norm's call."""
    shape, stats, width, dt, c = n._plan
    dev, out, y, st, m = z.device, buf.out, buf.y, buf.stats, buf.made
    known = m and m[0] is n and m[1] == dev and out is m[2] and y is m[3] and st is m[4]
    if not (known and _fits(z, shape, dt, dev) and _fits(res, shape, dt, dev)):
        lds = [_want_rows(name, t, shape, dt, dev) for name, t in (("z", z), ("res", res), ("out", out))]
        if n.pre:
            if y is None:
                raise ValueError("y: the buffers were allocated for a step without the norm before the next block")
            lds.append(_want_rows("y", y, shape, dt, dev))
        _want("stats", st, stats, torch.float32, dev)
        c = _step(n, *lds)
    if not n.pre:
        y = None
    p = _step_params(params, width, dev)
    return (c, z.data_ptr(), res.data_ptr(), ctypes.byref(p), out.data_ptr(), None if y is None else y.data_ptr(),
            st.data_ptr())


def residual_norm_backward(n: ResidualNorm, z, res, params: Dict, grad_out, grad_y,
                           buf: ResidualNormBuffers, stream=None):
    """Gradients of sum(out * grad_out) + sum(y * grad_y) after
    ``residual_norm`` with the same buffers: (grad_z, grad_res, {the gradients,
    fp32, of the parameters that params holds}). grad_out may be None; grad_y is
    None without the norm before the next block."""
    args, grads = _step_backward(n, z, res, params, grad_out, grad_y, buf)
    _run("moe_residual_norm_bwd", z.device, stream, load().moe_residual_norm_bwd, *args)
    return buf.grad_z, buf.grad_res, grads


def _step_backward(n, z, res, params, grad_out, grad_y, buf):
    """The checked arguments of residual_norm_backward's call, and the gradients
    that it returns."""
    shape, stats, width, dt, c = n._plan
    dev, st, gz, gr, ws, m, f32 = z.device, buf.stats, buf.grad_z, buf.grad_res, buf.workspace, buf.made, torch.float32
    if gz is None:
        raise ValueError("the buffers were allocated without training=True")
    if (grad_y is not None) != n.pre:
        raise ValueError("grad_y: expected exactly where there is a norm before the next block")
    known = (m and m[0] is n and m[1] == dev and st is m[4] and gz is m[5] and gr is m[6] and ws is m[7]
             and _fits(z, shape, dt, dev) and _fits(res, shape, dt, dev))
    if not (known and (grad_out is None or _fits(grad_out, shape, dt, dev))
            and (grad_y is None or _fits(grad_y, shape, dt, dev))):
        ld_z, ld_res = _want_rows("z", z, shape, dt, dev), _want_rows("res", res, shape, dt, dev)
        ld_go = 0 if grad_out is None else _want_rows("grad_out", grad_out, shape, dt, dev)
        ld_gy = 0 if grad_y is None else _want_rows("grad_y", grad_y, shape, dt, dev)
        ld_gz, ld_gr = _want_rows("grad_z", gz, shape, dt, dev), _want_rows("grad_res", gr, shape, dt, dev)
        _want("stats", st, stats, f32, dev)
        _want_bytes("workspace", ws, 0, dev)
        c = _step(n, ld_z, ld_res, 0, 0, ld_go, ld_gy, ld_gz, ld_gr)
    p = _step_params(params, width, dev)
    grads = {name: buf.grads[name] for name in NORM_PARAMS if params.get(name) is not None}
    g = _step_params(grads, width, dev, moe_norm_grads)
    return (c, z.data_ptr(), res.data_ptr(), ctypes.byref(p), st.data_ptr(),
            None if grad_out is None else grad_out.data_ptr(), None if grad_y is None else grad_y.data_ptr(),
            gz.data_ptr(), gr.data_ptr(), ctypes.byref(g), ws.data_ptr(), ws.numel()), grads


# ------------------------------------------------------ balance of the router

@dataclass(frozen=True)
class BalanceLoss(_Planned):
    """The router's balance loss and z loss over a batch; see moe_balance_loss."""

    tokens: int
    experts: int
    top_k: int
    d_model: int
    dtype: str = "bf16"
    balance: float = 0.01
    z: float = 0.001

    def struct(self) -> moe_balance:
        """The C problem, the caller's own to change."""
        return moe_balance(self.tokens, self.experts, self.top_k, self.d_model, DTYPES[self.dtype],
                           self.balance, self.z)

    @cached_property
    def _plan(self):
        c = self.struct()
        return (ctypes.byref(c), moe_balance_saved_bytes(c), torch.Size((self.tokens, self.d_model)),
                torch.Size((self.d_model, self.experts)), torch.Size((self.tokens, self.top_k)),
                torch.Size((self.experts,)), _TORCH[self.dtype])


@dataclass
class BalanceBuffers:
    """Device buffers of one balance loss, allocated once."""

    loss: object       # [3] fp32: the weighted sum, the balance loss, the z loss
    mean_prob: object  # [experts] fp32
    counts: object     # [experts] int32
    workspace: object
    saved: Optional[object] = None
    grad_x: Optional[object] = None
    grad_router: Optional[object] = None
    # what allocate_balance_loss made, with its problem and device: as NormBuffers.made
    made: Optional[tuple] = None


def allocate_balance_loss(b: BalanceLoss, device="cuda", training: bool = False) -> BalanceBuffers:
    device, c = _device(device), b.struct()
    nws = moe_balance_workspace_bytes(c)
    if nws == 0:
        raise ValueError(f"unsupported problem {b}")
    f32 = dict(dtype=torch.float32, device=device)
    buf = BalanceBuffers(loss=torch.empty(3, **f32), mean_prob=torch.empty(b.experts, **f32),
                         counts=torch.empty(b.experts, dtype=torch.int32, device=device),
                         workspace=torch.empty(nws, dtype=torch.uint8, device=device))
    if training:
        buf.saved = torch.empty(moe_balance_saved_bytes(c), dtype=torch.uint8, device=device)
        buf.grad_x = torch.empty((b.tokens, b.d_model), dtype=_TORCH[b.dtype], device=device)
        buf.grad_router = torch.empty((b.d_model, b.experts), **f32)
    buf.made = (b, device, buf.loss, buf.mean_prob, buf.counts, buf.workspace)
    return buf


def _want_mask(mask, b, device):
    if mask is None:
        return None
    if mask.dtype is not torch.uint8:
        _want("mask", mask, (b.tokens,), torch.bool, device)
    else:
        _want("mask", mask, (b.tokens,), torch.uint8, device)
    return mask.data_ptr()


def balance_loss(b: BalanceLoss, x, w_router, topk_idx, buf: BalanceBuffers, mask=None,
                 training: bool = False, stream=None):
    """The loss over the tokens x [tokens, d_model] that the routing topk_idx
    [tokens, top_k] was made of (the routing's dictionary holds it); mask [tokens]
    (bool or uint8) leaves out tokens where it is false. Returns buf.loss, with
    buf.mean_prob and buf.counts beside it."""
    _run("moe_balance_loss", x.device, stream, load().moe_balance_loss,
         *_balance_forward(b, x, w_router, topk_idx, buf, mask, training))
    return buf.loss


def _balance_forward(b, x, w_router, topk_idx, buf, mask, training):
    """The checked arguments of balance_loss's call."""
    c, nsv, xs, ws, ks, es, dt = b._plan
    dev = x.device
    _want("x", x, xs, dt, dev)
    _want("w_router", w_router, ws, torch.float32, dev)
    _want("topk_idx", topk_idx, ks, torch.int32, dev)
    m = _want_mask(mask, b, dev)
    made = buf.made
    if not (made and made[0] is b and made[1] == dev and made[2] is buf.loss and made[3] is buf.mean_prob
            and made[4] is buf.counts and made[5] is buf.workspace):
        _want("counts", buf.counts, es, torch.int32, dev)
        _want("mean_prob", buf.mean_prob, es, torch.float32, dev)
        _want("loss", buf.loss, (3,), torch.float32, dev)
        _want_bytes("workspace", buf.workspace, 0, dev)
    if training:
        _want_saved(buf, nsv, dev)
    return (c, x.data_ptr(), w_router.data_ptr(), topk_idx.data_ptr(), m, buf.counts.data_ptr(),
            buf.mean_prob.data_ptr(), buf.loss.data_ptr(), buf.saved.data_ptr() if training else None,
            buf.workspace.data_ptr(), buf.workspace.numel())


def balance_loss_backward(b: BalanceLoss, x, w_router, buf: BalanceBuffers, grad_loss=None, mask=None,
                          add_to=None, stream=None):
    """Gradients of grad_loss * loss[0] (grad_loss: an fp32 tensor of one
    number, or None: 1) after ``balance_loss(..., training=True)`` with the same
    buffers and mask: (grad_x, grad_router). w_router is the forward's, whose
    values the buffers hold (only its shape is looked at). add_to: a pair of gradients, the
    layer's own for instance, that they are added to in place of the buffers'."""
    _run("moe_balance_loss_bwd", x.device, stream, load().moe_balance_loss_bwd,
         *_balance_backward(b, x, w_router, buf, grad_loss, mask, add_to))
    return (buf.grad_x, buf.grad_router) if add_to is None else tuple(add_to)


def _balance_backward(b, x, w_router, buf, grad_loss, mask, add_to):
    """The checked arguments of balance_loss_backward's call."""
    c, nsv, xs, ws, _, _, dt = b._plan
    dev = x.device
    gx, gw = (buf.grad_x, buf.grad_router) if add_to is None else add_to
    _want("x", x, xs, dt, dev)
    _want("w_router", w_router, ws, torch.float32, dev)
    m = _want_mask(mask, b, dev)
    _want_saved(buf, nsv, dev)
    if grad_loss is not None:
        _want("grad_loss", grad_loss.reshape(-1), (1,), torch.float32, dev)
    _want("grad_x", gx, xs, dt, dev)
    _want("gradient of w_router", gw, ws, torch.float32, dev)
    _want_bytes("workspace", buf.workspace, 0, dev)
    return (c, x.data_ptr(), m, buf.saved.data_ptr(), _ptr(grad_loss), int(add_to is not None), gx.data_ptr(),
            gw.data_ptr(), buf.workspace.data_ptr(), buf.workspace.numel())


# ------------------------------------------------------- with the layer itself

@dataclass(frozen=True)
class _Layer:
    """What the layer's stages take for a problem, as (name, shape, type)."""

    x: tuple
    routing: tuple
    weights: tuple
    grads: tuple
    sorted: tuple
    shared: bool
    tiles: int
    saved: int


@lru_cache(maxsize=256)
def _layer(T, E, k, d, h, hs, dtype, block_m, capacity):
    c = ctypes.byref(binding.moe_problem(T, E, k, d, h, hs, dtype, block_m, capacity))
    lib, dt, f32, i32 = _load_library(), _TORCH[dtype], torch.float32, torch.int32
    w = [("w_gate", (E, d, h)), ("w_up", (E, d, h)), ("w_down", (E, h, d))]
    if hs > 0:
        w += [("ws_gate", (d, hs)), ("ws_up", (d, hs)), ("ws_down", (hs, d))]
    size, tiles = torch.Size, int(lib.moe_max_tiles(c))  # no tiles: a problem that the library refuses
    return _Layer((size((T, d)), dt),
                  tuple((n, size(s), t) for n, s, t in (
                      ("topk_idx", (T, k), i32), ("topk_w", (T, k), f32), ("expert_offsets", (E + 1,), i32),
                      ("perm", (T * k,), i32), ("inv_perm", (T * k,), i32), ("num_tiles", (1,), i32))),
                  tuple([("w_router", size((d, E)), f32)] + [(n, size(s), dt) for n, s in w]),
                  tuple([("w_router", size((d, E)), f32)] + [(n, size(s), f32) for n, s in w]),
                  (size((T * k, d)), dt), hs > 0, tiles, int(lib.moe_saved_bytes(c)))


def _want_all(what, tensors, specs, device):
    for name, shape, dtype in specs:
        _want(what + name, tensors[name], shape, dtype, device)


def _want_layer(p, name, x, buf, weights: Optional[Dict] = None, training: bool = False, grad_out=None):
    """The layer's input, buffers and, where they are given, weights and
    output gradient fit its problem: ``binding`` passes their pointers on as
    they are."""
    l = _layer(p.tokens, p.experts, p.top_k, p.d_model, p.d_hidden, p.d_shared, _dtype(p.dtype), p.block_m,
               getattr(p, "capacity", 0))
    dev, r = x.device, buf.routing
    _want(name, x, *l.x, dev)
    _want_all("", r, l.routing, dev)
    _want("tiles", r["tiles"], (max(1, l.tiles, r["tiles"].shape[0]), 3), torch.int32, dev)
    _want("out", buf.out, *l.x, dev)
    _want_bytes("workspace", buf.workspace, 0, dev)
    if weights is not None:
        _want_all("", weights, l.weights, dev)
        _want("y_sorted", buf.y_sorted, *l.sorted, dev)
        if l.shared:
            _want("shared_out", buf.shared_out, *l.x, dev)
        if training:
            _want_saved(buf, l.saved, dev)
    if grad_out is not None:
        _want("grad_out", grad_out, *l.x, dev)
        _want("grad_x of the layer", buf.grad_x, *l.x, dev)
        _want_all("gradient of ", buf.grads, l.grads, dev)
    _want_gpu(dev)


def prenorm_forward(p, x, weights: Dict, buf, norm: NormBuffers, eps: float = 1e-5,
                    training: bool = False, stream=None):
    """The MoE layer behind its norm, MoE(norm(x)): ``binding.forward`` on
    the normalised tokens; weights holds norm_weight and norm_bias (either may
    be missing) beside the layer's own. Returns buf.out."""
    _want_layer(p, "y of the norm", norm.y, buf, weights, training)
    h = layer_norm(x, weights.get("norm_weight"), weights.get("norm_bias"), eps, norm, stream)
    with torch.cuda.device(x.device):
        return binding.forward(p, h, weights, buf, training=training, stream=stream)


def prenorm_backward(p, x, weights: Dict, grad_out, buf, norm: NormBuffers, stream=None,
                     side_stream=None):
    """Gradients of sum(out * grad_out) after prenorm_forward(..., training=True)
    with the same buffers: (grad_x, the layer's weight gradients with
    norm_weight and norm_bias beside them)."""
    if buf.grads is None:
        raise ValueError("the buffers were allocated without training=True")
    _want_layer(p, "y of the norm", norm.y, buf, weights, True, grad_out)
    with torch.cuda.device(x.device):
        gh, grads = binding.backward(p, norm.y, weights, grad_out, buf, stream=stream,
                                     side_stream=side_stream)
    gx, gw, gb = layer_norm_backward(x, weights.get("norm_weight"), gh, norm, stream)
    return gx, dict(grads, norm_weight=gw, norm_bias=gb)


def _want_loss(p, loss):
    b = loss[0]
    if ((b.tokens, b.experts, b.top_k, b.d_model, DTYPES[b.dtype])
            != (p.tokens, p.experts, p.top_k, p.d_model, _dtype(p.dtype))):
        raise ValueError(f"loss: of {b}, not of {p}")


def residual_layer_forward(p, h, res, weights: Dict, buf, n: ResidualNorm, step: ResidualNormBuffers,
                           loss=None, mask=None, training: bool = False, stream=None):
    """The MoE layer as a block of a residual stream: ``binding.forward`` on h
    (the last step's y), then the step from its output and res; weights holds the
    step's parameters (``NORM_PARAMS``, each may be missing) beside the layer's.
    loss: a pair (BalanceLoss, BalanceBuffers) to have the router's balance loss
    of the tokens that mask keeps in its buffers. Returns (step.out, step.y)."""
    # every part is checked before the first is launched
    _want_layer(p, "h", h, buf, weights, training)
    if loss is not None:
        _want_loss(p, loss)
        balance = _balance_forward(loss[0], h, weights["w_router"], buf.routing["topk_idx"], loss[1], mask, training)
    after = _step_forward(n, buf.out, res, weights, step)
    with torch.cuda.device(h.device):
        binding.forward(p, h, weights, buf, training=training, stream=stream)
    if loss is not None:
        _run("moe_balance_loss", h.device, stream, load().moe_balance_loss, *balance)
    _run("moe_residual_norm_fwd", h.device, stream, load().moe_residual_norm_fwd, *after)
    return step.out, step.y if n.pre else None


def residual_layer_backward(p, h, res, weights: Dict, grad_out, grad_y, buf, n: ResidualNorm,
                            step: ResidualNormBuffers, loss=None, grad_loss=None, mask=None, stream=None,
                            side_stream=None):
    """Gradients of sum(out * grad_out) + sum(y * grad_y) + grad_loss * the
    balance loss after residual_layer_forward(..., training=True) with the same
    buffers: (grad_h, grad_res, the layer's weight gradients with the step's
    parameters' beside them), the loss's part added to the layer's."""
    if buf.grads is None:
        raise ValueError("the buffers were allocated without training=True")
    # every part is checked before the first is launched
    if loss is not None:
        _want_loss(p, loss)
        balance = _balance_backward(loss[0], h, weights["w_router"], loss[1], grad_loss, mask,
                                    (buf.grad_x, buf.grads["w_router"]))
    after, steps = _step_backward(n, buf.out, res, weights, grad_out, grad_y, step)
    _want_layer(p, "h", h, buf, weights, True, step.grad_z)
    _run("moe_residual_norm_bwd", h.device, stream, load().moe_residual_norm_bwd, *after)
    with torch.cuda.device(h.device):
        gh, grads = binding.backward(p, h, weights, step.grad_z, buf, stream=stream, side_stream=side_stream)
    if loss is not None:
        _run("moe_balance_loss_bwd", h.device, stream, load().moe_balance_loss_bwd, *balance)
    return gh, step.grad_res, dict(grads, **steps)


@dataclass
class ExpertsI8Buffers:
    """Buffers of the routed experts in 8 bits: both products' outputs."""

    gate_up: LinearI8
    down: LinearI8
    hidden: I8Buffers
    sorted: I8Buffers


@lru_cache(maxsize=256)
def _experts(tokens, experts, top_k, d_model, d_hidden, dtype, cap):
    name = "bf16" if dtype == MOE_BF16 else "fp32"
    up = LinearI8(tokens, d_model, 2 * d_hidden, name, experts, top_k, gated=True, capacity=cap)
    down = LinearI8(tokens, d_hidden, d_model, name, experts, top_k, sorted_input=True, capacity=cap)
    return up, down


def _experts_of(p):
    return _experts(p.tokens, p.experts, p.top_k, p.d_model, p.d_hidden, _dtype(p.dtype),
                    int(getattr(p, "capacity", 0)))


def allocate_experts_i8(p, device="cuda") -> ExpertsI8Buffers:
    up, down = _experts_of(p)
    return ExpertsI8Buffers(up, down, allocate_linear_i8(up, device), allocate_linear_i8(down, device))


def forward_i8(p, x, w_router, gate_up, down, buf, experts: ExpertsI8Buffers, shared_out=None,
               stream=None):
    """The layer's forward with routed experts in 8-bit integers: route ->
    permute -> gated product -> product -> combine. gate_up and down are
    (q, scale) pairs of ``quantize_weights(w_gate, w_up)`` and
    ``quantize_weights(w_down)``; buf is ``binding.allocate(p)``, and a shared
    expert's output may be given to be added. Returns buf.out."""
    _want("w_router", w_router, (p.d_model, p.experts), torch.float32, x.device)
    if shared_out is not None:
        _want("shared_out", shared_out, x.shape, x.dtype, x.device)
    if (experts.gate_up, experts.down) != _experts_of(p):
        raise ValueError(f"experts: buffers of {experts.gate_up} and {experts.down}, not of {p}")
    _want_layer(p, "x", x, buf)
    with torch.cuda.device(x.device):
        binding.moe_route(p, x, w_router, buf.routing, stream)
        binding.moe_permute(p, buf.routing, buf.workspace, stream=stream)
        h = linear_i8(experts.gate_up, x, *gate_up, experts.hidden, routing=buf.routing, stream=stream)
        y = linear_i8(experts.down, h, *down, experts.sorted, routing=buf.routing, stream=stream)
        binding.moe_combine(p, y, buf.routing, shared_out, buf.out, stream)
    return buf.out
