"""Binding of the operators of a residual block and of a beam search
(include/rlca.h): the gated linear recurrence with its gradients and its single
step, the root-mean-square norm with the residual's addition, and the
selection and reordering of beams.

Argument marshalling only, as in sequence.py: shape / dtype / device checks,
output and workspace allocation through torch, and the current HIP stream of
the inputs' device.  The calls build no autograd graph; what a call writes into
a tensor of the caller's counts as a change in place.
"""
from __future__ import annotations

import ctypes
import struct
from typing import NamedTuple, Optional

import torch

from .rlca import (
    REAL_DTYPES, RESET_ON_START, SIGNATURES, SIZE_QUERIES, _check, _current_stream, _p, _sz, lib,
)
from .sequence import (
    _activations, _dense_in, _flags_in, _new, _new_step, _ptr, _scratch, _view, _written,
    _written_outputs,
)

_i32 = ctypes.c_int32
_i64 = ctypes.c_int64
_f64 = ctypes.c_double


class GatedCall(ctypes.Structure):
    """rlca_gated_call of include/rlca.h."""

    _fields_ = [
        ("num_seqs", _i64), ("channels", _i64), ("T", _i64), ("dtype", _i32),
        ("convention", _i32), ("scale", _f64), ("x", _p), ("input_gate", _p), ("decay_gate", _p),
        ("x_stride_seq", _i64), ("x_stride_channel", _i64), ("input_stride_seq", _i64),
        ("input_stride_channel", _i64), ("decay_stride_seq", _i64),
        ("decay_stride_channel", _i64), ("decay", _p), ("input_bias", _p), ("decay_bias", _p),
        ("state", _p), ("flags", _p), ("lengths", _p), ("out", _p), ("final_state", _p),
        ("checkpoints", _p), ("grad_out", _p), ("grad_stride_seq", _i64),
        ("grad_stride_channel", _i64), ("grad_final_state", _p), ("grad_x", _p),
        ("grad_input_gate", _p), ("grad_decay_gate", _p), ("grad_decay", _p),
        ("grad_input_bias", _p), ("grad_decay_bias", _p), ("grad_state", _p),
    ]


class GatedStepCall(ctypes.Structure):
    """rlca_gated_step_call of include/rlca.h."""

    _fields_ = [
        ("num_seqs", _i64), ("channels", _i64), ("places", _i64), ("dtype", _i32),
        ("scale", _f64), ("x", _p), ("input_gate", _p), ("decay_gate", _p),
        ("x_stride_seq", _i64), ("input_stride_seq", _i64), ("decay_stride_seq", _i64),
        ("decay", _p), ("input_bias", _p), ("decay_bias", _p), ("state", _p), ("slots", _p),
        ("starts", _p), ("out", _p),
    ]


SIGNATURES.update({
    "rlca_gated_recurrence": [_p, _p, _sz, _p],
    "rlca_gated_recurrence_backward": [_p, _p, _sz, _p],
    "rlca_gated_step": [_p, _p],
})
SIZE_QUERIES.update({
    "rlca_gated_recurrence_checkpoints_size": [_p],
    "rlca_gated_recurrence_workspace_size": [_p],
    "rlca_gated_recurrence_backward_workspace_size": [_p],
})


def _packer(cls):
    """As sequence.py's, for records that hold doubles too."""
    codes = {_i64: "q", _i32: "i", _p: "P", _f64: "d"}
    return struct.Struct("@" + "".join(codes[kind] for _, kind in cls._fields_)).pack


_pack_gated, _pack_gated_step = _packer(GatedCall), _packer(GatedStepCall)


def _run(name, dev, *args):
    """One library call on the current stream of the inputs' device.  Its default
    stream has no handle of its own, so another device is made the current one."""
    if torch.cuda.current_device() == dev.index:
        status = getattr(lib(), name)(*args, _current_stream(dev))
    else:
        with torch.cuda.device(dev):
            status = getattr(lib(), name)(*args, _current_stream(dev))
    _check(status, name)


# -------------------------------------------------------- the gated recurrence
class GatedGrads(NamedTuple):
    """Gradients of gated_recurrence's inputs; None where there is no such input."""

    x: torch.Tensor
    input_gate: torch.Tensor
    decay_gate: torch.Tensor
    decay: torch.Tensor
    input_bias: Optional[torch.Tensor]
    decay_bias: Optional[torch.Tensor]
    state: Optional[torch.Tensor]


def _gated_inputs(x, input_gate, decay_gate, decay, input_bias, decay_bias, scale, state, flags,
                  convention, lengths):
    """The record's fields up to lengths, and what the outputs are made of."""
    shape, dev, dtype = _activations("x", x, 3)
    N, D, T = shape
    ig = _view("input_gate", input_gate, shape, dtype, dev)
    dg = _view("decay_gate", decay_gate, shape, dtype, dev)
    if decay is None:
        raise ValueError("decay is required")
    f32 = torch.float32
    fields = (N, D, T, REAL_DTYPES[dtype], int(convention), float(scale), x.data_ptr(),
              ig.data_ptr(), dg.data_ptr(), x.stride(0), x.stride(1), ig.stride(0), ig.stride(1),
              dg.stride(0), dg.stride(1), _dense_in("decay", decay, (D,), f32, dev),
              _dense_in("input_bias", input_bias, (D,), f32, dev),
              _dense_in("decay_bias", decay_bias, (D,), f32, dev),
              _dense_in("state", state, (N, D), f32, dev), _flags_in(flags, (N, T), dev),
              _dense_in("lengths", lengths, (N,), torch.int32, dev))
    return fields, shape, dev, dtype


def gated_recurrence(x, input_gate, decay_gate, decay, input_bias=None, decay_bias=None,
                     scale=8.0, state=None, flags=None, convention=RESET_ON_START, lengths=None,
                     with_state=False, with_checkpoints=False, out=None, final_state=None):
    """Gated linear recurrence of each channel:
    a_t = exp(-scale softplus(decay) sigmoid(decay_gate_t + decay_bias)),
    h_t = a_t h_{t-1} + sqrt(1 - a_t^2) sigmoid(input_gate_t + input_bias) x_t.

    x and the gates [num_seqs, channels, T] (float32, bfloat16 or float16; time
    contiguous, other strides free); decay, input_bias and decay_bias [channels]
    and state [num_seqs, channels] float32; flags [num_seqs, T] episode
    boundaries; lengths [num_seqs] int32.
    Returns (h, final state | None, checkpoints | None); the checkpoints are
    what gated_recurrence_backward needs of this call."""
    fields, shape, dev, dtype = _gated_inputs(x, input_gate, decay_gate, decay, input_bias,
                                              decay_bias, scale, state, flags, convention,
                                              lengths)
    o = _new(out, shape, dtype, dev)
    f = c = None
    if with_state or final_state is not None:
        f = _new(final_state, shape[:2], torch.float32, dev, "final_state")
    query = _pack_gated(*fields, *(0,) * 14)
    if with_checkpoints:
        c = _new(None, (lib().rlca_gated_recurrence_checkpoints_size(query) // 4,),
                 torch.float32, dev)
    n = lib().rlca_gated_recurrence_workspace_size(query)
    ws = _scratch(n, dev) if n > 0 else None
    call = _pack_gated(*fields, o.data_ptr(), _ptr(f), _ptr(c), *(0,) * 11)
    _run("rlca_gated_recurrence", dev, call, _ptr(ws), n)
    if out is not None or final_state is not None:
        _written_outputs(out, final_state)
    return o, f, c


def gated_recurrence_backward(grad_out, x, input_gate, decay_gate, decay, checkpoints,
                              input_bias=None, decay_bias=None, scale=8.0, state=None,
                              flags=None, convention=RESET_ON_START, lengths=None,
                              grad_state=None):
    """Gradients of gated_recurrence with these inputs, from its output's
    gradient (and, with grad_state, its final state's) and the checkpoints it
    returned.  Returns GatedGrads."""
    fields, shape, dev, dtype = _gated_inputs(x, input_gate, decay_gate, decay, input_bias,
                                              decay_bias, scale, state, flags, convention,
                                              lengths)
    N, D, _ = shape
    g = _view("grad_out", grad_out, shape, dtype, dev)
    f32 = torch.float32
    gf = _dense_in("grad_state", grad_state, (N, D), f32, dev)
    if checkpoints is None:
        raise ValueError("checkpoints is required")
    query = _pack_gated(*fields, *(0,) * 14)
    n = lib().rlca_gated_recurrence_checkpoints_size(query) // 4
    c = _dense_in("checkpoints", checkpoints, (n,), f32, dev)
    grads = GatedGrads(
        x=_new(None, shape, dtype, dev), input_gate=_new(None, shape, dtype, dev),
        decay_gate=_new(None, shape, dtype, dev), decay=_new(None, (D,), f32, dev),
        input_bias=None if input_bias is None else _new(None, (D,), f32, dev),
        decay_bias=None if decay_bias is None else _new(None, (D,), f32, dev),
        state=None if state is None else _new(None, (N, D), f32, dev))
    call = _pack_gated(*fields, 0, 0, c, g.data_ptr(), g.stride(0), g.stride(1), gf,
                       *(_ptr(t) for t in grads))
    ws = _scratch(lib().rlca_gated_recurrence_backward_workspace_size(query), dev)
    _run("rlca_gated_recurrence_backward", dev, call, ws.data_ptr(), ws.numel())
    return grads


def gated_step(x, input_gate, decay_gate, decay, state, input_bias=None, decay_bias=None,
               scale=8.0, slots=None, flags=None, out=None):
    """One step of gated_recurrence for each sequence: x and the gates [num_seqs,
    channels], state [places, channels] float32 updated in place.  slots and flags
    as for selective_step.  Returns h [num_seqs, channels]."""
    shape, dev, dtype = _activations("x", x, 2)
    N, D = shape
    ig = _view("input_gate", input_gate, shape, dtype, dev)
    dg = _view("decay_gate", decay_gate, shape, dtype, dev)
    f32 = torch.float32
    if decay is None:
        raise ValueError("decay is required")
    if state is None or state.dim() != 2:
        raise ValueError("state is [places, channels]")
    places = state.shape[0]
    s = _dense_in("state", state, (places, D), f32, dev)
    if slots is None and places < N:
        raise ValueError(f"state has {places} places for {N} sequences")
    i = _dense_in("slots", slots, (N,), torch.int32, dev)
    f = _flags_in(flags, (N,), dev)
    o = _new_step(out, x, shape, dtype, dev, "out")
    call = _pack_gated_step(N, D, places, REAL_DTYPES[dtype], float(scale), x.data_ptr(),
                            ig.data_ptr(), dg.data_ptr(), x.stride(0), ig.stride(0),
                            dg.stride(0), _dense_in("decay", decay, (D,), f32, dev),
                            _dense_in("input_bias", input_bias, (D,), f32, dev),
                            _dense_in("decay_bias", decay_bias, (D,), f32, dev), s, i, f,
                            o.data_ptr())
    _run("rlca_gated_step", dev, call)
    _written((state,) if out is None else (state, out))
    return o
