"""The gated scan: a linear recurrence along the rows of sequences, channel by channel.

    h_t = a_t h_{t-1} + (1 - a_t) x_t,   a_t = 1 / (1 + exp(-gate_t)),   from the sequence's state

In each channel that is the solve of a unit lower bidiagonal system, and its backward pass the solve with the
transpose, as for the sparse systems of this package.  In a coefficient network it carries information from cell to
cell: along the lines of a grid, along a path through all cells, or step by step with a kept state.  The compute is
libsla's (``csrc/sla_scan.cu``, C ABI in ``include/sla.h``): a CPU tensor raises.

Data is float32, float16 or bfloat16, states are float32.  The sla_* functions are the C calls under their names
(no autograd graph, leading dimensions allowed); gated_scan is differentiable.
"""
from __future__ import annotations

import ctypes
import functools
import math
from typing import Optional

import torch
from torch.autograd.function import once_differentiable

from . import _abi
from .dense import _check, _empty, _lib, _on_device_of_first, _param, _rows, _scratch, _stream, _type, _wants_grad

_OFFSETS = {torch.int32: _abi.SLA_I32, torch.int64: _abi.SLA_I64}


@functools.lru_cache(maxsize=512)
def _sizes(rows, channels, sequences, ragged, dt):
    """(bytes kept for the backward call, bytes of scratch)"""
    s = _abi.sla_scan(rows, channels, sequences, 256 if ragged else None, _abi.SLA_I32, dt, 0, 0)
    return _lib().sla_gated_scan_saved_bytes(ctypes.byref(s)), _lib().sla_gated_scan_workspace_bytes(ctypes.byref(s))


def _matrix(t: torch.Tensor) -> torch.Tensor:
    """t as the rows of one matrix where its strides allow that (the halves of a linear layer's rows, say)."""
    if t.dim() == 2 or t.is_contiguous():
        return t
    try:
        return t.view(-1, t.shape[-1])
    except RuntimeError:
        return t  # refused by name


def _matrix_ready(t: torch.Tensor) -> torch.Tensor:
    """t, or a contiguous copy where its rows cannot be read in place."""
    m = _matrix(t)
    if m.is_contiguous() or (m.dim() == 2 and m.stride(1) == 1 and m.stride(0) >= m.shape[1]):
        return t
    return t.contiguous()


class _Scan:
    """A call's descriptor and what follows from it."""

    def __init__(self, x, gate, offsets, reverse, outside):
        if x.dim() < 2:
            raise ValueError(f"x must be [..., length, channels], got shape {tuple(x.shape)}")
        if gate.shape != x.shape:
            raise ValueError(f"gate must have x's shape {tuple(x.shape)}, got {tuple(gate.shape)}")
        self.x, rows, self.ldx = _rows(_matrix(x), "x")
        self.gate, _, self.ldg = _rows(_matrix(gate), "gate", x)
        self.channels, self.dt, self.index = x.shape[-1], _type(x, "x"), x.get_device()
        address = kind = None
        if offsets is None:
            self.sequences = math.prod(x.shape[:-2])
        else:
            if x.dim() != 2:
                raise ValueError(f"with offsets x must be [rows, channels], got shape {tuple(x.shape)}")
            kind = _OFFSETS.get(offsets.dtype)
            if kind is None or offsets.dim() != 1 or offsets.numel() < 1:
                raise ValueError("offsets must be an int32 or int64 vector of at least one element, got "
                                 f"{offsets.dtype} of shape {tuple(offsets.shape)}")
            address = _param(offsets, "offsets", offsets.shape, offsets.dtype, self.index)
            self.sequences = offsets.numel() - 1
        self.descriptor = _abi.sla_scan(rows, self.channels, self.sequences, address, kind or 0, self.dt,
                                        1 if reverse else 0, 1 if outside else 0)
        self.ref = ctypes.byref(self.descriptor)
        self.saved, self.scratch = _sizes(rows, self.channels, self.sequences, offsets is not None, self.dt)
        self.key = (rows, self.channels, self.sequences, offsets is not None, self.dt, bool(reverse))
        self.states = (self.sequences, self.channels)

    def state(self, t, name):
        return _param(t, name, self.states, torch.float32, self.index)


@_on_device_of_first
def sla_gated_scan(x: torch.Tensor, gate: torch.Tensor, state: Optional[torch.Tensor] = None,
                   offsets: Optional[torch.Tensor] = None, reverse: bool = False, h: Optional[torch.Tensor] = None,
                   final: Optional[torch.Tensor] = None, save: bool = False,
                   workspace: Optional[torch.Tensor] = None):
    """h_t = a_t h_{t-1} + (1 - a_t) x_t with a = sigmoid(gate), along each sequence (asynchronous).

    x and gate are [..., length, channels]: sequences of one length; or, with offsets ([sequences + 1], int32 or
    int64), [rows, channels]: sequence i has the rows from offsets[i] to offsets[i + 1].  state and final are
    [sequences, channels] float32, before (None: zero) and behind the sequences; final may be state.  reverse: each
    sequence from its last row to its first.  Rows of h that belong to no sequence become zero, or stay as they are in
    an h that is given.  Returns (h, final), or with save=True (h, final, saved): the buffer that
    sla_gated_scan_backward takes."""
    s = _Scan(x, gate, offsets, reverse, h is None)
    dev = x.device
    sp = s.state(state, "state")
    if h is None:
        h = _empty(x.shape, dtype=x.dtype, device=dev)
        hp = h.data_ptr()
    else:
        hp = _param(h, "h", x.shape, x.dtype, s.index)
    if final is None:
        final = _empty(s.states, dtype=torch.float32, device=dev)
    fp = s.state(final, "final")
    saved, kept, kept_bytes = None, None, 0
    if save:
        saved, kept_bytes = _scratch(s.saved, dev, None)
        saved.made_for = s.key
        kept = saved.data_ptr()
    wsp, nbytes = None, 0
    if s.scratch:
        ws, nbytes = _scratch(s.scratch, dev, workspace)
        wsp = ws.data_ptr()
    _check(_lib().sla_gated_scan(s.ref, s.x, s.ldx, s.gate, s.ldg, sp, hp, fp, kept, kept_bytes, wsp, nbytes,
                                 _stream(s.index)), "sla_gated_scan")
    return (h, final, saved) if save else (h, final)


@_on_device_of_first
def sla_gated_scan_backward(dh: Optional[torch.Tensor], x: torch.Tensor, gate: torch.Tensor, saved: torch.Tensor,
                            dfinal: Optional[torch.Tensor] = None, state: Optional[torch.Tensor] = None,
                            offsets: Optional[torch.Tensor] = None, reverse: bool = False, want_grad_x: bool = True,
                            want_grad_gate: bool = True, want_grad_state: bool = True,
                            workspace: Optional[torch.Tensor] = None):
    """Gradients of sla_gated_scan (asynchronous): (dx, dgate, dstate), None where not wanted.  dh or dfinal may be None
    (zero); x, gate, state, offsets, reverse and saved are the forward call's."""
    s = _Scan(x, gate, offsets, reverse, False)
    dev = x.device
    dhp = lddh = None
    if dh is not None:
        if dh.shape != x.shape:
            raise ValueError(f"dh must have x's shape {tuple(x.shape)}, got {tuple(dh.shape)}")
        dhp, _, lddh = _rows(_matrix(dh), "dh", x)
    dfp, sp = s.state(dfinal, "dfinal"), s.state(state, "state")
    if saved.dtype != torch.uint8 or saved.get_device() != s.index or not saved.is_contiguous():
        raise ValueError("saved must be the buffer that sla_gated_scan(..., save=True) returned")
    # a copy of the buffer has lost the note of what it was made for, but not its size
    if getattr(saved, "made_for", s.key) != s.key or saved.numel() > max(s.saved, 256):
        raise ValueError("saved is from a forward call of other sizes, another type or another direction")
    dx = dgate = dstate = dxp = dgp = dsp = None
    if want_grad_x:
        dx = _empty(x.shape, dtype=x.dtype, device=dev)
        dxp = dx.data_ptr()
    if want_grad_gate:
        dgate = _empty(x.shape, dtype=x.dtype, device=dev)
        dgp = dgate.data_ptr()
    if want_grad_state:
        dstate = _empty(s.states, dtype=torch.float32, device=dev)
        dsp = dstate.data_ptr()
    wsp, nbytes = None, 0
    if s.scratch:
        ws, nbytes = _scratch(s.scratch, dev, workspace)
        wsp = ws.data_ptr()
    _check(_lib().sla_gated_scan_backward(s.ref, dhp, lddh or 0, dfp, s.x, s.ldx, s.gate, s.ldg, sp, saved.data_ptr(),
                                          saved.numel(), dxp, dgp, dsp, wsp, nbytes, _stream(s.index)),
           "sla_gated_scan_backward")
    return dx, dgate, dstate


class GatedScan(torch.autograd.Function):
    """(h, states behind the sequences).  Saved for backward: x, the gate, and a float32 state every 16th row (8th of float32)."""

    @staticmethod
    def forward(ctx, x, gate, state, offsets, reverse):
        x, gate = _matrix_ready(x), _matrix_ready(gate)
        h, final, saved = sla_gated_scan(x, gate, state, offsets, reverse, save=True)
        ctx.save_for_backward(x, gate, state, offsets, saved)
        ctx.reverse = reverse
        ctx.set_materialize_grads(False)
        return h, final

    @staticmethod
    @once_differentiable
    def backward(ctx, dh, dfinal):
        x, gate, state, offsets, saved = ctx.saved_tensors
        need = ctx.needs_input_grad
        if dh is None and dfinal is None:
            return None, None, None, None, None
        if dh is not None:
            dh = _matrix_ready(dh)
        if dfinal is not None:
            dfinal = dfinal.contiguous()
        with torch.cuda.device(x.device):
            dx, dgate, dstate = sla_gated_scan_backward(dh, x, gate, saved, dfinal, state, offsets, ctx.reverse, need[0],
                                                        need[1], need[2])
        return dx, dgate, dstate, None, None


def gated_scan(x: torch.Tensor, gate: torch.Tensor, state: Optional[torch.Tensor] = None,
               offsets: Optional[torch.Tensor] = None, reverse: bool = False):
    """Differentiable gated scan (gradients flow to x, gate and state): (h, states behind the sequences)."""
    if state is not None:
        state = state.contiguous()
    if _wants_grad(x, gate, state):
        return GatedScan.apply(x, gate, state, offsets, reverse)
    return sla_gated_scan(_matrix_ready(x), _matrix_ready(gate), state, offsets, reverse)
