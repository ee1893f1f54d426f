"""Dense operators of a coefficient network: layer norm, residual norm, linear layer and the gated feed-forward block.

The values of a matrix often come from a network over the grid cells (one token a cell) that is
trained through the solve; layer norm and feed-forward block are the two halves of its residual block
z + gated_ffn(layer_norm(z)), linear layers stand around the scan of a mixing block (``scan.py``), and the residual norm
joins a block's result with the residual stream z and norms the sum for the next block.
As everywhere in this package the compute is libsla's (``csrc/sla_norm.cu``, ``sla_resnorm.cu``, ``sla_linear.cu``, ``sla_ffn.cu``,
C ABI in ``include/sla.h``): this module marshals torch tensors, and a CPU tensor raises.

Data is float32, float16 or bfloat16.  The sla_* functions are the C calls under their names (no
autograd graph, leading dimensions allowed); layer_norm, residual_norm, linear and gated_ffn are differentiable.
"""
from __future__ import annotations

import ctypes
import functools
import inspect
from typing import NamedTuple, Optional, Tuple

import torch
from torch.autograd.forward_ad import unpack_dual
from torch.autograd.function import once_differentiable

from . import _abi
from ._buffers import usable

ACTIVATIONS = {"silu": _abi.SLA_ACT_SILU, "gelu": _abi.SLA_ACT_GELU, "gelu_tanh": _abi.SLA_ACT_GELU_TANH,
               "relu": _abi.SLA_ACT_RELU}
_DT = {torch.float32: _abi.SLA_F32, torch.float16: _abi.SLA_F16, torch.bfloat16: _abi.SLA_BF16}


_library = None


def _lib():
    global _library
    if _library is None:
        import differentiable_sparse_iterative_gb300 as base  # the package imports this module
        _library = base.lib()
    return _library


def _check(status: int, where: str) -> None:
    if status != _abi.SLA_OK:
        from . import SlaError
        raise SlaError(status, where)


# a call is a few microseconds of GPU time for one token: the stream's handle without a Stream object
_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch._C._cuda_getDevice
_empty = torch.empty


def _on_device_of_first(call):
    """call, with the device of its first argument (of the first tensor, where that is None) as the current one: libsla
    launches on the current device and asks it for its size, and the handle of a default stream names no device."""
    first = next(iter(inspect.signature(call).parameters))

    @functools.wraps(call)
    def run(*args, **kw):
        t = args[0] if args else kw.get(first)
        if t is None:
            t = next((a for a in (*args, *kw.values()) if isinstance(a, torch.Tensor)), None)
        if t is not None and t.is_cuda and t.get_device() != _current_device():
            with torch.cuda.device(t.get_device()):
                return call(*args, **kw)
        return call(*args, **kw)

    return run


def _rows(t: torch.Tensor, name: str, like: Optional[torch.Tensor] = None) -> Tuple[int, int, int]:
    """(address, rows, elements between rows) of a tensor read as rows of its last dimension."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (libsla has no CPU path)")
    if like is not None and (t.dtype != like.dtype or t.get_device() != like.get_device()):
        raise ValueError(f"{name} must have dtype {like.dtype} on {like.device}, got {t.dtype} on {t.device}")
    dim = t.dim()
    width = t.size(dim - 1) if dim else 0
    if width < 1:
        raise ValueError(f"{name} must have a last dimension of at least one element")
    rows = t.size(0) if dim == 2 else t.numel() // width
    if t.is_contiguous():
        return t.data_ptr(), rows, width
    if dim == 2 and (width == 1 or t.stride(1) == 1) and (t.stride(0) >= width or rows <= 1):
        return t.data_ptr(), rows, t.stride(0)
    raise ValueError(f"{name} must be contiguous, or a matrix with contiguous rows that do not overlap")


# What a call needs that depends on its sizes alone is asked for once: two or three calls less of a
# microsecond each, where one token's kernels take ten.
@functools.lru_cache(maxsize=512)
def _ln_backward_bytes(rows: int, width: int, dt: int, device: int) -> int:
    return _lib().sla_layernorm_backward_workspace_bytes(rows, width, dt)


class _FFNSizes:
    def __init__(self, tokens, width, hidden, out, dt, act):
        self.descriptor = _abi.sla_ffn(tokens, width, hidden, out, dt, act)
        self.ref = ctypes.byref(self.descriptor)
        self.tokens, self.hidden, self.out = tokens, hidden, out
        self.key = (tokens, width, hidden, out, dt, act)
        lib = _lib()
        self.saved = lib.sla_gated_ffn_saved_bytes(self.ref)
        self.forward = lib.sla_gated_ffn_workspace_bytes(self.ref)
        self.backward = lib.sla_gated_ffn_backward_workspace_bytes(self.ref)


@functools.lru_cache(maxsize=512)
def _ffn_sizes(tokens, width, hidden, out, dt, act, device) -> _FFNSizes:
    return _FFNSizes(tokens, width, hidden, out, dt, act)


def _param(t: Optional[torch.Tensor], name: str, shape, dtype, device: int) -> Optional[int]:
    if t is None:
        return None
    if not t.is_cuda or t.get_device() != device:
        raise ValueError(f"{name} must be a CUDA tensor on cuda:{device}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.dtype != dtype:
        raise ValueError(f"{name} must have dtype {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _type(t: torch.Tensor, name: str) -> int:
    dt = _DT.get(t.dtype)
    if dt is None:
        raise ValueError(f"{name} must be float32, float16 or bfloat16, got {t.dtype}")
    return dt


def _scratch(need: int, device, ws: Optional[torch.Tensor]) -> Tuple[torch.Tensor, int]:
    """(buffer, bytes): the caller's workspace where it is large enough, else a new one."""
    if usable(ws, need, device):
        return ws, ws.numel() * ws.element_size()
    need = max(need, 256)
    return _empty(need, dtype=torch.uint8, device=device), need


# --------------------------------------------------------------------------- layer norm

def _ln_params(x, weight, bias):
    pt = weight.dtype if weight is not None else bias.dtype if bias is not None else x.dtype
    if pt != x.dtype and pt != torch.float32:
        raise ValueError(f"weight and bias must have dtype {x.dtype} or torch.float32, got {pt}")
    return pt


@_on_device_of_first
def sla_layernorm(x: torch.Tensor, weight: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None,
                  eps: float = 1e-5, y: Optional[torch.Tensor] = None, stats: bool = False):
    """Layer norm over the last dimension (asynchronous).  weight and bias ([width], of x's type or
    float32) default to one and zero.  Returns y, or with stats=True (y, mean, rstd): the rows'
    float32 statistics that sla_layernorm_backward takes."""
    ptr, rows, ldx = _rows(x, "x")
    xt, dev, index, shape = x.dtype, x.device, x.get_device(), x.shape
    dt, width = _type(x, "x"), shape[-1]
    pt = _ln_params(x, weight, bias)
    wp = _param(weight, "weight", (width,), pt, index)
    bp = _param(bias, "bias", (width,), pt, index)
    if y is None:
        y = _empty(shape, dtype=xt, device=dev)
        yp = y.data_ptr()
    else:
        yp = _param(y, "y", shape, xt, index)
    mean = rstd = mp = rp = None
    if stats:
        mean, rstd = _empty(rows, dtype=torch.float32, device=dev), _empty(rows, dtype=torch.float32, device=dev)
        mp, rp = mean.data_ptr(), rstd.data_ptr()
    _check(_lib().sla_layernorm(rows, width, dt, _DT[pt], ptr, ldx, wp, bp, eps, yp, mp, rp, _stream(index)),
           "sla_layernorm")
    return (y, mean, rstd) if stats else y


def sla_layernorm_backward_workspace_bytes(rows: int, width: int, dtype: torch.dtype) -> int:
    return _lib().sla_layernorm_backward_workspace_bytes(int(rows), int(width), _DT[dtype])


@_on_device_of_first
def sla_layernorm_backward(dy: torch.Tensor, x: torch.Tensor, weight: Optional[torch.Tensor], mean: torch.Tensor,
                           rstd: torch.Tensor, want_grad_x: bool = True, want_grad_weight: bool = True,
                           want_grad_bias: bool = True, param_dtype: Optional[torch.dtype] = None,
                           workspace: Optional[torch.Tensor] = None):
    """Gradients of sla_layernorm (asynchronous): (dx, dweight, dbias), None where not wanted.
    dweight and dbias have weight's type (param_dtype, default x's, when there is no weight)."""
    ptr, rows, ldx = _rows(x, "x")
    gptr, _, lddy = _rows(dy, "dy", x)
    xt, dev, index, shape = x.dtype, x.device, x.get_device(), x.shape
    if dy.shape != shape:
        raise ValueError(f"dy must have x's shape {tuple(shape)}, got {tuple(dy.shape)}")
    dt, width = _type(x, "x"), shape[-1]
    pt = weight.dtype if weight is not None else param_dtype or xt
    if pt != xt and pt != torch.float32:
        raise ValueError(f"weight must have dtype {xt} or torch.float32, got {pt}")
    wp = _param(weight, "weight", (width,), pt, index)
    mp = _param(mean, "mean", (rows,), torch.float32, index)
    rp = _param(rstd, "rstd", (rows,), torch.float32, index)
    dx = dw = db = dxp = dwp = dbp = wsp = None
    nbytes = 0
    if want_grad_x:
        dx = _empty(shape, dtype=xt, device=dev)
        dxp = dx.data_ptr()
    if want_grad_weight:
        dw = _empty(width, dtype=pt, device=dev)
        dwp = dw.data_ptr()
    if want_grad_bias:
        db = _empty(width, dtype=pt, device=dev)
        dbp = db.data_ptr()
    lib = _lib()
    if want_grad_weight or want_grad_bias:
        ws, nbytes = _scratch(_ln_backward_bytes(rows, width, dt, index), dev, workspace)
        wsp = ws.data_ptr()
    _check(lib.sla_layernorm_backward(rows, width, dt, _DT[pt], gptr, lddy, ptr, ldx, wp, mp, rp, dxp, dwp, dbp, wsp,
                                      nbytes, _stream(index)), "sla_layernorm_backward")
    return dx, dw, db


def _matrix_ready(t: torch.Tensor) -> torch.Tensor:
    """t, or a contiguous copy where its rows cannot be read in place (expanded or transposed tensors)."""
    if t.is_contiguous() or (t.dim() == 2 and t.stride(1) == 1 and t.stride(0) >= t.shape[1]):
        return t
    return t.contiguous()


class LayerNorm(torch.autograd.Function):
    """y = layer norm of x's last dimension.  Saved for backward: x, the weight and two floats a row."""

    @staticmethod
    def forward(ctx, x, weight, bias, eps):
        x = _matrix_ready(x)
        y, mean, rstd = sla_layernorm(x, weight, bias, eps=eps, stats=True)
        ctx.save_for_backward(x, weight, mean, rstd)
        ctx.param_dtype = _ln_params(x, weight, bias)
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, weight, mean, rstd = ctx.saved_tensors
        need_x, need_w, need_b = ctx.needs_input_grad[:3]
        dx, dw, db = sla_layernorm_backward(_matrix_ready(dy), x, weight, mean, rstd, need_x, need_w, need_b,
                                            param_dtype=ctx.param_dtype)
        return dx, dw, db, None


def _wants_grad(*tensors) -> bool:
    """Whether the call belongs in the autograd graph.  A tensor with a forward-mode tangent takes the node as
    well, which refuses it (NotImplementedError): past the node the tangent would be lost without a word."""
    grad = torch.is_grad_enabled()
    return any(t is not None and ((grad and t.requires_grad) or unpack_dual(t).tangent is not None) for t in tensors)


def layer_norm(x: torch.Tensor, weight: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None,
               eps: float = 1e-5) -> torch.Tensor:
    """Differentiable layer norm over the last dimension (gradients flow to x, weight and bias)."""
    if _wants_grad(x, weight, bias):
        return LayerNorm.apply(x, weight, bias, eps)
    return sla_layernorm(_matrix_ready(x), weight, bias, eps=eps)


# --------------------------------------------------------------------------- residual norm

NORMS = {"layer": _abi.SLA_NORM_LAYER, "rms": _abi.SLA_NORM_RMS}
GATE_ACTIVATIONS = {"none": _abi.SLA_GATE_NONE, "sigmoid": _abi.SLA_GATE_SIGMOID, "silu": _abi.SLA_GATE_SILU}


class ResidualNormGrads(NamedTuple):
    """Gradients of a residual norm, None where not wanted."""
    block: Optional[torch.Tensor]
    z: Optional[torch.Tensor]
    gate: Optional[torch.Tensor]
    scale: Optional[torch.Tensor]
    post_weight: Optional[torch.Tensor]
    post_bias: Optional[torch.Tensor]
    weight: Optional[torch.Tensor]
    bias: Optional[torch.Tensor]


def _param_type(x, params):
    """The parameters' common type: x's or float32."""
    pt = next((p.dtype for p in params if p is not None), x.dtype)
    if pt != x.dtype and pt != torch.float32:
        raise ValueError(f"parameters must have dtype {x.dtype} or torch.float32, got {pt}")
    return pt


def _choice(value, choices, name):
    found = choices.get(value)
    if found is None:
        raise ValueError(f"unknown {name} {value!r} (one of {', '.join(choices)})")
    return found


def _same_rows(t, x, name):
    """(address, elements between rows) of a tensor of x's shape, or None."""
    if t is None:
        return None, 0
    if t.shape != x.shape:
        raise ValueError(f"{name} must have the block's shape {tuple(x.shape)}, got {tuple(t.shape)}")
    ptr, _, ld = _rows(t, name, x)
    return ptr, ld


@functools.lru_cache(maxsize=512)
def _resnorm_descriptor(rows, width, dt, pt, norm, post_norm, gate_activation, eps):
    d = _abi.sla_resnorm(rows, width, dt, pt, norm, post_norm, gate_activation, 0, eps)
    return d, ctypes.byref(d)


class _ResNorm:
    """A call's descriptor, the addresses of its inputs and their parameters."""

    def __init__(self, block, z, gate, names, params, norm, post_norm, gate_activation, eps, param_dtype=None):
        ptr, rows, ld = _rows(block, "block")
        self.rows, self.width, self.index = rows, block.shape[-1], block.get_device()
        if param_dtype is not None and all(p is None for p in params):
            if param_dtype != block.dtype and param_dtype != torch.float32:
                raise ValueError(f"param_dtype must be {block.dtype} or torch.float32, got {param_dtype}")
            self.pt = param_dtype
        else:
            self.pt = _param_type(block, params)
        zp, ldz = _same_rows(z, block, "z")
        gp, ldg = _same_rows(gate, block, "gate")
        self.arrays = (ptr, ld, zp, ldz, gp, ldg)
        shape, pt, index = (self.width,), self.pt, self.index
        self.params = [None if t is None else _param(t, name, shape, pt, index) for t, name in zip(params, names)]
        self.types = (_type(block, "block"), _DT[pt])
        self.descriptor, self.ref = _resnorm_descriptor(
            rows, self.width, *self.types, _choice(norm, NORMS, "norm"), 1 if post_norm else 0,
            _choice(gate_activation, GATE_ACTIVATIONS, "gate activation"), eps)


_RESNORM_PARAMS = ("scale", "post_weight", "post_bias", "weight", "bias")


@_on_device_of_first
def sla_residual_norm(block: torch.Tensor, z: torch.Tensor, gate: Optional[torch.Tensor] = None,
                      scale: Optional[torch.Tensor] = None, post_weight: Optional[torch.Tensor] = None,
                      post_bias: Optional[torch.Tensor] = None, weight: Optional[torch.Tensor] = None,
                      bias: Optional[torch.Tensor] = None, norm: str = "layer", post_norm: bool = True,
                      next_norm: bool = True, gate_activation: str = "none", eps: float = 1e-5, stats: bool = False):
    """A block's result joins the residual stream z (asynchronous): z' = z + scale * act(gate) * N(block) and
    y = N(z'), the next block's input.

    N(block) has post_weight and post_bias (post_norm=False: the block itself), N(z') weight and bias
    (next_norm=False: y is None); norm is "layer" or "rms", gate_activation "none", "sigmoid" or "silu".  block, z and
    gate have one shape; the parameters are [width], of its type or float32.  Returns (z', y), or with stats=True
    (z', y, stats): the rows' float32 statistics that sla_residual_norm_backward takes."""
    n = _ResNorm(block, z, gate, _RESNORM_PARAMS, (scale, post_weight, post_bias, weight, bias), norm, post_norm,
                 gate_activation, eps)
    shape, dt, dev = block.shape, block.dtype, block.device
    z_out = _empty(shape, dtype=dt, device=dev)
    y = _empty(shape, dtype=dt, device=dev) if next_norm else None
    kept = _empty((n.rows, 4), dtype=torch.float32, device=dev) if stats else None
    _check(_lib().sla_residual_norm(n.ref, *n.arrays, *n.params, z_out.data_ptr(), y.data_ptr() if next_norm else None,
                                    kept.data_ptr() if stats else None, _stream(n.index)), "sla_residual_norm")
    return (z_out, y, kept) if stats else (z_out, y)


@functools.lru_cache(maxsize=512)
def _resnorm_backward_bytes(rows, width, dt, pt, device) -> int:
    return _lib().sla_residual_norm_backward_workspace_bytes(ctypes.byref(_abi.sla_resnorm(rows, width, dt, pt, 0, 1, 0, 0, 0.0)))


@_on_device_of_first
def sla_residual_norm_backward(dz: Optional[torch.Tensor], dy: Optional[torch.Tensor], block: torch.Tensor,
                               z: torch.Tensor, stats: torch.Tensor, gate: Optional[torch.Tensor] = None,
                               scale: Optional[torch.Tensor] = None, post_weight: Optional[torch.Tensor] = None,
                               post_bias: Optional[torch.Tensor] = None, weight: Optional[torch.Tensor] = None,
                               norm: str = "layer", post_norm: bool = True, gate_activation: str = "none",
                               eps: float = 1e-5, want_grad_block: bool = True, want_grad_z: bool = True,
                               want_grad_gate: bool = True, want_grad_params: bool = True,
                               param_dtype: Optional[torch.dtype] = None,
                               workspace: Optional[torch.Tensor] = None) -> ResidualNormGrads:
    """Gradients of sla_residual_norm (asynchronous).  dz and dy belong to its two results; one of them may be None (zero).
    The other arguments are the forward call's.  The parameters' gradients have the parameters' type (param_dtype, default the
    block's, when there is none), also where the parameter itself was left out."""
    n = _ResNorm(block, z, gate, _RESNORM_PARAMS, (scale, post_weight, post_bias, weight), norm, post_norm, gate_activation,
                 eps, param_dtype)
    up = [*_same_rows(dz, block, "dz"), *_same_rows(dy, block, "dy")]
    sp = _param(stats, "stats", (n.rows, 4), torch.float32, n.index)
    dev = block.device

    def rows_like(wanted):
        return _empty(block.shape, dtype=block.dtype, device=dev) if wanted else None

    def params_like(wanted):
        return _empty(n.width, dtype=n.pt, device=dev) if wanted else None

    post = want_grad_params and post_norm
    after = want_grad_params and dy is not None
    grads = ResidualNormGrads(rows_like(want_grad_block), rows_like(want_grad_z),
                              rows_like(want_grad_gate and gate is not None), params_like(want_grad_params),
                              params_like(post), params_like(post), params_like(after), params_like(after))
    wsp, nbytes = None, 0
    if want_grad_params:
        ws, nbytes = _scratch(_resnorm_backward_bytes(n.rows, n.width, *n.types, n.index), dev, workspace)
        wsp = ws.data_ptr()
    _check(_lib().sla_residual_norm_backward(n.ref, *up, *n.arrays, *n.params, sp,
                                             *[None if t is None else t.data_ptr() for t in grads], wsp, nbytes,
                                             _stream(n.index)), "sla_residual_norm_backward")
    return grads


class ResidualNorm(torch.autograd.Function):
    """(z', y).  Saved for backward: block, z, the gate, the parameters and four floats a row (z' is formed again)."""

    @staticmethod
    def forward(ctx, block, z, gate, scale, post_weight, post_bias, weight, bias, how):
        block, z = _matrix_ready(block), _matrix_ready(z)
        gate = None if gate is None else _matrix_ready(gate)
        z_out, y, stats = sla_residual_norm(block, z, gate, scale, post_weight, post_bias, weight, bias, stats=True, **how)
        ctx.save_for_backward(block, z, gate, scale, post_weight, post_bias, weight, stats)
        ctx.how = {k: v for k, v in how.items() if k != "next_norm"}
        ctx.param_dtype = _param_type(block, (scale, post_weight, post_bias, weight, bias))
        ctx.set_materialize_grads(False)
        return z_out, y

    @staticmethod
    @once_differentiable
    def backward(ctx, dz, dy):
        block, z, gate, scale, post_weight, post_bias, weight, stats = ctx.saved_tensors
        if dz is None and dy is None:
            return (None,) * 9
        need = ctx.needs_input_grad
        dz, dy = (None if t is None else _matrix_ready(t) for t in (dz, dy))
        with torch.cuda.device(block.device):
            g = sla_residual_norm_backward(dz, dy, block, z, stats, gate, scale, post_weight, post_bias, weight,
                                           want_grad_block=need[0], want_grad_z=need[1], want_grad_gate=need[2],
                                           want_grad_params=any(need[3:8]), param_dtype=ctx.param_dtype, **ctx.how)
        return (*[t if n else None for t, n in zip(g, need)], None)


def residual_norm(block: torch.Tensor, z: torch.Tensor, gate: Optional[torch.Tensor] = None,
                  scale: Optional[torch.Tensor] = None, post_weight: Optional[torch.Tensor] = None,
                  post_bias: Optional[torch.Tensor] = None, weight: Optional[torch.Tensor] = None,
                  bias: Optional[torch.Tensor] = None, norm: str = "layer", post_norm: bool = True,
                  next_norm: bool = True, gate_activation: str = "none", eps: float = 1e-5):
    """Differentiable residual norm (gradients flow to block, z, the gate and the parameters): (z', y)."""
    how = {"norm": norm, "post_norm": post_norm, "next_norm": next_norm, "gate_activation": gate_activation, "eps": eps}
    if _wants_grad(block, z, gate, scale, post_weight, post_bias, weight, bias):
        return ResidualNorm.apply(block, z, gate, scale, post_weight, post_bias, weight, bias, how)
    return sla_residual_norm(_matrix_ready(block), _matrix_ready(z), None if gate is None else _matrix_ready(gate), scale,
                             post_weight, post_bias, weight, bias, **how)


# --------------------------------------------------------------------------- linear layer

LINEAR_ACTIVATIONS = {"none": _abi.SLA_ACT_NONE, **ACTIVATIONS}


class _LinearSizes:
    def __init__(self, tokens, width, out, dt, act):
        self.descriptor = _abi.sla_layer(tokens, width, out, dt, act)
        self.ref = ctypes.byref(self.descriptor)
        self.out = out
        self.key = (tokens, width, out, dt, act)
        lib = _lib()
        self.saved = lib.sla_linear_saved_bytes(self.ref)
        self.forward = lib.sla_linear_workspace_bytes(self.ref)
        self.backward = lib.sla_linear_backward_workspace_bytes(self.ref)


@functools.lru_cache(maxsize=512)
def _linear_sizes(tokens, width, out, dt, act, device) -> _LinearSizes:
    return _LinearSizes(tokens, width, out, dt, act)


def _linear(x, weight, activation):
    """(sizes, address of x, its leading dimension, address of the weight)"""
    ptr, rows, ldx = _rows(x, "x")
    act = _choice(activation, LINEAR_ACTIVATIONS, "activation")
    if weight.dim() != 2:
        raise ValueError(f"weight must be [out, width], got {tuple(weight.shape)}")
    out, width, index = weight.size(0), x.size(-1), x.get_device()
    f = _linear_sizes(rows, width, out, _type(x, "x"), act, index)
    return f, ptr, ldx, _param(weight, "weight", (out, width), x.dtype, index)


@_on_device_of_first
def sla_linear(x: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor] = None,
               residual: Optional[torch.Tensor] = None, activation: str = "none", y: Optional[torch.Tensor] = None,
               save: bool = False, workspace: Optional[torch.Tensor] = None):
    """y = act(x weight^T + bias) + residual (asynchronous).

    weight is [out, width], bias [out], residual of y's shape; activation: "none", "silu", "gelu", "gelu_tanh" or
    "relu".  Returns y, or with save=True (y, saved): the byte buffer of intermediates that sla_linear_backward takes."""
    f, ptr, ldx, wp = _linear(x, weight, activation)
    dt, dev, index = x.dtype, x.device, x.get_device()
    bp = _param(bias, "bias", (f.out,), dt, index)
    shape = x.shape[:-1] + (f.out,)
    rp, ldr = None, 0
    if residual is not None:
        if residual.shape != shape:
            raise ValueError(f"residual must have shape {tuple(shape)}, got {tuple(residual.shape)}")
        rp, _, ldr = _rows(residual, "residual", x)
    if y is None:
        y = _empty(shape, dtype=dt, device=dev)
        yp = y.data_ptr()
    else:
        yp = _param(y, "y", shape, dt, index)
    saved, sp, sn = None, None, 0
    if save:
        saved, sn = _scratch(f.saved, dev, None)
        saved.made_for = f.key
        sp = saved.data_ptr()
    wsp, nbytes = None, 0
    if f.forward:
        ws, nbytes = _scratch(f.forward, dev, workspace)
        wsp = ws.data_ptr()
    _check(_lib().sla_linear(f.ref, ptr, ldx, wp, bp, rp, ldr, yp, sp, sn, wsp, nbytes, _stream(index)), "sla_linear")
    return (y, saved) if save else y


@_on_device_of_first
def sla_linear_backward(dy: torch.Tensor, x: torch.Tensor, weight: torch.Tensor, saved: torch.Tensor,
                        activation: str = "none", want_grad_x: bool = True, want_grad_weight: bool = True,
                        want_grad_bias: bool = False, workspace: Optional[torch.Tensor] = None):
    """Gradients of sla_linear (asynchronous): (dx, dweight, dbias), None where not wanted; the residual's is dy.  x, the
    weight, the activation and `saved` are the forward call's."""
    f, ptr, ldx, wp = _linear(x, weight, activation)
    gptr, _, lddy = _rows(dy, "dy", x)
    if dy.shape != x.shape[:-1] + (f.out,):
        raise ValueError(f"dy must have shape {tuple(x.shape[:-1]) + (f.out,)}, got {tuple(dy.shape)}")
    if saved.dtype != torch.uint8 or saved.get_device() != x.get_device() or not saved.is_contiguous():
        raise ValueError("saved must be the buffer that sla_linear(..., save=True) returned")
    # a copy of the buffer has lost the note of what it was made for, but not its size
    if getattr(saved, "made_for", f.key) != f.key or saved.numel() > max(f.saved, 256):
        raise ValueError("saved is from a forward call of other sizes, another type or another activation")
    dt, dev = x.dtype, x.device
    dx = _empty(x.shape, dtype=dt, device=dev) if want_grad_x else None
    dw = _empty(weight.shape, dtype=dt, device=dev) if want_grad_weight else None
    db = _empty(f.out, dtype=dt, device=dev) if want_grad_bias else None
    ws, nbytes = _scratch(f.backward, dev, workspace)
    _check(_lib().sla_linear_backward(f.ref, gptr, lddy, ptr, ldx, wp, saved.data_ptr(), saved.numel(),
                                      *[None if t is None else t.data_ptr() for t in (dx, dw, db)], ws.data_ptr(), nbytes,
                                      _stream(x.get_device())), "sla_linear_backward")
    return dx, dw, db


class Linear(torch.autograd.Function):
    """y = act(x weight^T + bias) + residual.  Saved for backward: x, the weight, act'(x weight^T + bias) where there is an
    activation, and the copies that were laid out anew for the tensor core (float32, or a width that 8 does not divide; none up to
    16 tokens and for layers of few outputs, which are not the tensor core's)."""

    @staticmethod
    def forward(ctx, x, weight, bias, residual, activation):
        x, weight = _matrix_ready(x), weight.contiguous()
        residual = None if residual is None else _matrix_ready(residual)
        y, saved = sla_linear(x, weight, bias, residual, activation=activation, save=True)
        ctx.save_for_backward(x, weight, saved)
        ctx.activation = activation
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, weight, saved = ctx.saved_tensors
        need = ctx.needs_input_grad
        dx = dw = db = None
        if any(need[:3]):
            dx, dw, db = sla_linear_backward(_matrix_ready(dy), x, weight, saved, activation=ctx.activation,
                                             want_grad_x=need[0], want_grad_weight=need[1], want_grad_bias=need[2])
        return dx, dw, db, dy if need[3] else None, None


def linear(x: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor] = None,
           residual: Optional[torch.Tensor] = None, activation: str = "none") -> torch.Tensor:
    """Differentiable linear layer (gradients flow to x, the weight, the bias and the residual)."""
    if _wants_grad(x, weight, bias, residual):
        return Linear.apply(x, weight, bias, residual, activation)
    return sla_linear(_matrix_ready(x), weight.contiguous(), bias, None if residual is None else _matrix_ready(residual),
                      activation=activation)


# --------------------------------------------------------------------------- gated feed-forward block

def _ffn(x, w_in, w_out, activation):
    """(sizes, address of x, its leading dimension, addresses of w_in and w_out)"""
    ptr, rows, ldx = _rows(x, "x")
    act = ACTIVATIONS.get(activation)
    if act is None:
        raise ValueError(f"unknown activation {activation!r} (one of {', '.join(ACTIVATIONS)})")
    if w_in.dim() != 2 or w_out.dim() != 2 or w_in.size(0) != 2 * w_out.size(1):
        raise ValueError("w_in must be [2 * hidden, width] and w_out [out, hidden], got "
                         f"{tuple(w_in.shape)} and {tuple(w_out.shape)}")
    out, hidden = w_out.shape
    width, index = x.size(-1), x.get_device()
    f = _ffn_sizes(rows, width, hidden, out, _type(x, "x"), act, index)
    return (f, ptr, ldx, _param(w_in, "w_in", (2 * hidden, width), x.dtype, index),
            _param(w_out, "w_out", (out, hidden), x.dtype, index))


@_on_device_of_first
def sla_gated_ffn(x: torch.Tensor, w_in: torch.Tensor, w_out: torch.Tensor, b_in: Optional[torch.Tensor] = None,
                  b_out: Optional[torch.Tensor] = None, activation: str = "silu", y: Optional[torch.Tensor] = None,
                  save: bool = False, workspace: Optional[torch.Tensor] = None):
    """y = (act(x Wg^T + bg) * (x Wu^T + bu)) w_out^T + b_out (asynchronous).

    w_in stacks Wg over Wu ([2 hidden, width]), b_in likewise; w_out is [out, hidden].  activation:
    "silu", "gelu", "gelu_tanh" or "relu".  Returns y, or with save=True (y, saved): the byte buffer
    of intermediates that sla_gated_ffn_backward takes."""
    f, ptr, ldx, wip, wop = _ffn(x, w_in, w_out, activation)
    lib, dt, dev, index = _lib(), x.dtype, x.device, x.get_device()
    bip = _param(b_in, "b_in", (2 * f.hidden,), dt, index)
    bop = _param(b_out, "b_out", (f.out,), dt, index)
    shape = (f.tokens, f.out) if x.dim() == 2 else x.shape[:-1] + (f.out,)
    if y is None:
        y = _empty(shape, dtype=dt, device=dev)
        yp = y.data_ptr()
    else:
        yp = _param(y, "y", shape, dt, index)
    saved, sp, sn = None, None, 0
    if save:
        saved, sn = _scratch(f.saved, dev, None)
        saved.made_for = f.key
        sp = saved.data_ptr()
    ws, nbytes = _scratch(f.forward, dev, workspace)
    _check(lib.sla_gated_ffn(f.ref, ptr, ldx, wip, bip, wop, bop, yp, sp, sn, ws.data_ptr(), nbytes, _stream(index)),
           "sla_gated_ffn")
    return (y, saved) if save else y


@_on_device_of_first
def sla_gated_ffn_backward(dy: torch.Tensor, x: torch.Tensor, w_in: torch.Tensor, w_out: torch.Tensor,
                           saved: torch.Tensor, activation: str = "silu", want_grad_x: bool = True,
                           want_grad_weights: bool = True, want_grad_bias: bool = False,
                           workspace: Optional[torch.Tensor] = None):
    """Gradients of sla_gated_ffn (asynchronous): (dx, dw_in, dw_out, db_in, db_out), None where not
    wanted.  x, the weights, the activation and `saved` are the forward call's."""
    f, ptr, ldx, wip, wop = _ffn(x, w_in, w_out, activation)
    gptr, _, lddy = _rows(dy, "dy", x)
    if dy.shape != x.shape[:-1] + (f.out,):
        raise ValueError(f"dy must have shape {tuple(x.shape[:-1]) + (f.out,)}, got {tuple(dy.shape)}")
    if saved.dtype != torch.uint8 or saved.get_device() != x.get_device() or not saved.is_contiguous():
        raise ValueError("saved must be the buffer that sla_gated_ffn(..., save=True) returned")
    # a copy of the buffer has lost the note of what it was made for, but not its size
    if getattr(saved, "made_for", f.key) != f.key or saved.numel() > max(f.saved, 256):
        raise ValueError("saved is from a forward call of other sizes, another type or another activation")
    lib, dt, dev = _lib(), x.dtype, x.device
    dx = dw_in = dw_out = db_in = db_out = None
    if want_grad_x:
        dx = _empty(x.shape, dtype=dt, device=dev)
    if want_grad_weights:
        dw_in, dw_out = _empty(w_in.shape, dtype=dt, device=dev), _empty(w_out.shape, dtype=dt, device=dev)
    if want_grad_bias:
        db_in, db_out = _empty(2 * f.hidden, dtype=dt, device=dev), _empty(f.out, dtype=dt, device=dev)
    grads = (dx, dw_in, dw_out, db_in, db_out)
    ws, nbytes = _scratch(f.backward, dev, workspace)
    _check(lib.sla_gated_ffn_backward(f.ref, gptr, lddy, ptr, ldx, wip, wop, saved.data_ptr(), saved.numel(),
                                      *[None if t is None else t.data_ptr() for t in grads], ws.data_ptr(), nbytes,
                                      _stream(x.get_device())), "sla_gated_ffn_backward")
    return grads


def sla_gated_ffn_check(device: Optional[int] = None) -> None:
    """Synchronises the device's current stream and raises SlaError(SLA_TIMEOUT) if a bounded wait inside a
    gated_ffn kernel on it has expired (never expected) that this thread has not been told of.  The other calls
    raise it as well, for an earlier call's wait, without synchronising."""
    device = torch.cuda.current_device() if device is None else device
    with torch.cuda.device(device):
        _check(_lib().sla_gated_ffn_check(_stream(device)), "sla_gated_ffn_check")


def sla_test_expire_wait() -> None:
    """Test hook: a bounded wait on the current stream that expires (see sla.h)."""
    _check(_lib().sla_test_expire_wait(_stream(torch.cuda.current_device())), "sla_test_expire_wait")


class GatedFFN(torch.autograd.Function):
    """y = (act(x Wg^T + bg) * (x Wu^T + bu)) w_out^T + b_out.  Saved for backward: x, the weights and
    u act'(g), act(g) and h (3 hidden values a token), and the copies that were laid out anew for the
    tensor core (float32, or a width or hidden size that 8 does not divide)."""

    @staticmethod
    def forward(ctx, x, w_in, w_out, b_in, b_out, activation):
        x, w_in, w_out = _matrix_ready(x), w_in.contiguous(), w_out.contiguous()
        y, saved = sla_gated_ffn(x, w_in, w_out, b_in, b_out, activation=activation, save=True)
        ctx.save_for_backward(x, w_in, w_out, saved)
        ctx.activation = activation
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, w_in, w_out, saved = ctx.saved_tensors
        need = ctx.needs_input_grad
        dx, dw_in, dw_out, db_in, db_out = sla_gated_ffn_backward(
            _matrix_ready(dy), x, w_in, w_out, saved, activation=ctx.activation, want_grad_x=need[0],
            want_grad_weights=need[1] or need[2], want_grad_bias=need[3] or need[4])
        return (dx, dw_in if need[1] else None, dw_out if need[2] else None, db_in if need[3] else None,
                db_out if need[4] else None, None)


def gated_ffn(x: torch.Tensor, w_in: torch.Tensor, w_out: torch.Tensor, b_in: Optional[torch.Tensor] = None,
              b_out: Optional[torch.Tensor] = None, activation: str = "silu") -> torch.Tensor:
    """Differentiable gated feed-forward block (gradients flow to x, the weights and the biases)."""
    if _wants_grad(x, w_in, w_out, b_in, b_out):
        return GatedFFN.apply(x, w_in, w_out, b_in, b_out, activation)
    return sla_gated_ffn(_matrix_ready(x), w_in.contiguous(), w_out.contiguous(), b_in, b_out, activation=activation)
