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


# What a call needs that depends on its sizes alone is made once: a single step is a few microseconds of GPU time.
@functools.lru_cache(maxsize=512)
def _sizes(rows, channels, sequences, ragged, dt):
    """(bytes kept for the backward call, bytes of scratch)"""
    s = _abi.sla_scan(rows, channels, sequences, 256 if ragged else None, _abi.SLA_I32, dt, 0, 0)
    return _lib().sla_gated_scan_saved_bytes(ctypes.byref(s)), _lib().sla_gated_scan_workspace_bytes(ctypes.byref(s))


class _Uniform:
    """What calls over sequences of one length share."""

    def __init__(self, rows, channels, sequences, dt, reverse, outside):
        self.descriptor = _abi.sla_scan(rows, channels, sequences, None, 0, dt, reverse, outside)
        self.ref = ctypes.byref(self.descriptor)
        self.saved, self.scratch = _sizes(rows, channels, sequences, False, dt)


_uniform = functools.lru_cache(maxsize=512)(_Uniform)


def _matrix_rows(t: torch.Tensor, name: str, like: Optional[torch.Tensor] = None):
    """(address, rows, elements between rows) of a tensor whose strides let it be read as the rows of one matrix (the halves
    of a linear layer's rows, say)."""
    if t.dim() == 3 and not t.is_contiguous() and t.is_cuda:
        q, n, c = t.shape
        sq, sn, sc = t.stride()
        if (sc == 1 or c == 1) and c and (n == 1 or q == 1 or sq == n * sn):
            ld = sq if n == 1 else sn
            if (ld >= c or q * n <= 1) and (like is None or (t.dtype == like.dtype and t.get_device() == like.get_device())):
                return t.data_ptr(), q * n, max(ld, c)
    elif t.dim() > 3 and not t.is_contiguous():
        try:
            t = t.view(-1, t.shape[-1])
        except RuntimeError:
            pass  # refused by name
    return _rows(t, name, like)


def _matrix_ready(t: torch.Tensor) -> torch.Tensor:
    """t, or a contiguous copy where its rows cannot be read in place."""
    if not t.is_contiguous() and t.is_cuda and t.dim() >= 2:
        try:
            _matrix_rows(t, "")
        except ValueError:
            return t.contiguous()
    return t


class _Scan:
    """A call's descriptor and what follows from it."""

    def __init__(self, x, gate, offsets, reverse, outside):
        shape = x.shape
        if len(shape) < 2:
            raise ValueError(f"x must be [..., length, channels], got shape {tuple(shape)}")
        if gate.shape != shape:
            raise ValueError(f"gate must have x's shape {tuple(shape)}, got {tuple(gate.shape)}")
        self.x, rows, self.ldx = _matrix_rows(x, "x")
        self.gate, _, self.ldg = _matrix_rows(gate, "gate", x)
        channels, dt, self.index = shape[-1], _type(x, "x"), x.get_device()
        self.rows, ragged = rows, offsets is not None
        if not ragged:
            self.sequences = shape[0] if len(shape) == 3 else math.prod(shape[:-2])
            u = _uniform(rows, channels, self.sequences, dt, 1 if reverse else 0, 1 if outside else 0)
            self.ref, self.saved, self.scratch = u.ref, u.saved, u.scratch
        else:
            if len(shape) != 2:
                raise ValueError(f"with offsets x must be [rows, channels], got shape {tuple(shape)}")
            kind = _OFFSETS.get(offsets.dtype) if isinstance(offsets, torch.Tensor) else None
            if kind is None or offsets.dim() != 1 or offsets.numel() < 1:
                got = f"{offsets.dtype} of shape {tuple(offsets.shape)}" if isinstance(offsets, torch.Tensor) else type(offsets)
                raise ValueError(f"offsets must be an int32 or int64 vector of at least one element, got {got}")
            address = _param(offsets, "offsets", offsets.shape, offsets.dtype, self.index)
            self.sequences = offsets.numel() - 1
            self.descriptor = _abi.sla_scan(rows, channels, self.sequences, address, kind, dt, 1 if reverse else 0,
                                            1 if outside else 0)
            self.ref = ctypes.byref(self.descriptor)
            self.saved, self.scratch = _sizes(rows, channels, self.sequences, True, dt)
        self.key = (rows, channels, self.sequences, ragged, dt, bool(reverse))
        self.states = (self.sequences, channels)

    def state(self, t, name):
        return None if t is None else _param(t, name, self.states, torch.float32, self.index)


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
        dhp, _, lddh = _matrix_rows(dh, "dh", x)
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


def sla_test_set_scan_wait(withhold: int, clocks: int) -> None:
    """Test hook: what the next scans' blocks wait for, and for how long (see sla.h); (0, 0) restores normal operation."""
    _check(_lib().sla_test_set_scan_wait(int(withhold), int(clocks)), "sla_test_set_scan_wait")


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
