"""Binding of the sequence-model operators of librlca.so (include/rlca.h): the
causal convolution, the selective scan, their single-step forms and gradients,
and the clipping of gradients by their global norm.

Argument marshalling only, as in rlca.py: shape / dtype / device checks, output
and workspace allocation through torch, and the current HIP stream.  The calls
build no autograd graph: results carry none, whatever the inputs require, and the
gradients are calls of their own (recurrent_policy.py wraps them for autograd).
What a call writes into a tensor of the caller's counts as a change in place.
"""
from __future__ import annotations

import ctypes
import math
import struct
import threading
from array import array
from typing import NamedTuple, Optional

import torch

from .rlca import (
    REAL_DTYPES, RESET_ON_START, SIGNATURES, SIZE_QUERIES, _FLAG_DTYPES, _check,
    _current_stream, _out, _p, _real_dtype, _steps, _sz, _workspaces, _workspaces_lock, lib,
)

MAX_STATES = 128
CLIP_WORKSPACE_BYTES = 20736

_i32 = ctypes.c_int32
_i64 = ctypes.c_int64


class ConvCall(ctypes.Structure):
    """rlca_conv_call of include/rlca.h."""

    _fields_ = [
        ("num_seqs", _i64), ("channels", _i64), ("T", _i64), ("width", _i32), ("silu", _i32),
        ("dtype", _i32), ("convention", _i32), ("x", _p), ("x_stride_seq", _i64),
        ("x_stride_channel", _i64), ("weight", _p), ("bias", _p), ("state", _p), ("flags", _p),
        ("lengths", _p), ("out", _p), ("final_state", _p), ("grad_out", _p),
        ("grad_stride_seq", _i64), ("grad_stride_channel", _i64), ("grad_final_state", _p),
        ("grad_x", _p), ("grad_weight", _p), ("grad_bias", _p), ("grad_state", _p),
    ]


class ScanCall(ctypes.Structure):
    """rlca_scan_call of include/rlca.h."""

    _fields_ = [
        ("num_seqs", _i64), ("channels", _i64), ("T", _i64), ("states", _i32), ("groups", _i32),
        ("softplus", _i32), ("dtype", _i32), ("convention", _i32), ("u", _p), ("delta", _p),
        ("u_stride_seq", _i64), ("u_stride_channel", _i64), ("delta_stride_seq", _i64),
        ("delta_stride_channel", _i64), ("A", _p), ("B", _p), ("C", _p), ("B_stride_seq", _i64),
        ("B_stride_group", _i64), ("B_stride_state", _i64), ("C_stride_seq", _i64),
        ("C_stride_group", _i64), ("C_stride_state", _i64), ("D", _p), ("delta_bias", _p),
        ("z", _p), ("z_stride_seq", _i64), ("z_stride_channel", _i64), ("state", _p),
        ("flags", _p), ("lengths", _p), ("y", _p), ("final_state", _p), ("checkpoints", _p),
        ("grad_y", _p), ("grad_stride_seq", _i64), ("grad_stride_channel", _i64),
        ("grad_final_state", _p), ("grad_u", _p), ("grad_delta", _p), ("grad_A", _p),
        ("grad_B", _p), ("grad_C", _p), ("grad_D", _p), ("grad_delta_bias", _p), ("grad_z", _p),
        ("grad_state", _p),
    ]


class ConvStepCall(ctypes.Structure):
    """rlca_conv_step_call of include/rlca.h."""

    _fields_ = [
        ("num_seqs", _i64), ("channels", _i64), ("places", _i64), ("width", _i32),
        ("silu", _i32), ("dtype", _i32), ("x", _p), ("x_stride_seq", _i64), ("weight", _p),
        ("bias", _p), ("state", _p), ("slots", _p), ("starts", _p), ("out", _p),
    ]


class ScanStepCall(ctypes.Structure):
    """rlca_scan_step_call of include/rlca.h."""

    _fields_ = [
        ("num_seqs", _i64), ("channels", _i64), ("places", _i64), ("states", _i32),
        ("groups", _i32), ("softplus", _i32), ("dtype", _i32), ("u", _p), ("delta", _p),
        ("u_stride_seq", _i64), ("delta_stride_seq", _i64), ("A", _p), ("B", _p), ("C", _p),
        ("B_stride_seq", _i64), ("B_stride_group", _i64), ("C_stride_seq", _i64),
        ("C_stride_group", _i64), ("D", _p), ("delta_bias", _p), ("z", _p),
        ("z_stride_seq", _i64), ("state", _p), ("slots", _p), ("starts", _p), ("y", _p),
    ]


class GradTensor(ctypes.Structure):
    """rlca_grad_tensor of include/rlca.h."""

    _fields_ = [("data", _p), ("out", _p), ("count", _i64), ("dtype", _i32)]


# The entry points read these records before they return.  They are taken as
# plain addresses, so that a call can pass a packed copy of one (below) and
# code that fills in a structure can pass that.
SIGNATURES.update({
    "rlca_causal_conv": [_p, _p],
    "rlca_causal_conv_backward": [_p, _p, _sz, _p],
    "rlca_selective_scan": [_p, _p],
    "rlca_selective_scan_backward": [_p, _p, _sz, _p],
    "rlca_causal_conv_step": [_p, _p],
    "rlca_selective_step": [_p, _p],
    "rlca_clip_grad_norm": [_p, _i64, ctypes.c_double, ctypes.c_double, _p, _p, _sz, _p],
})
SIZE_QUERIES.update({
    "rlca_causal_conv_backward_workspace_size": [_p],
    "rlca_selective_scan_checkpoints_size": [_p],
    "rlca_selective_scan_backward_workspace_size": [_p],
})


def _packer(cls):
    """Packs a record's values, in the order of its fields, into bytes laid out
    as the structure is: a quarter of the time that filling one takes."""
    codes = {_i64: "q", _i32: "i", _p: "P"}
    return struct.Struct("@" + "".join(codes[kind] for _, kind in cls._fields_)).pack


_pack_conv, _pack_scan, _pack_conv_step, _pack_scan_step = (
    _packer(cls) for cls in (ConvCall, ScanCall, ConvStepCall, ScanStepCall))


def _ptr(t):
    return 0 if t is None else t.data_ptr()


class ConvGrads(NamedTuple):
    """Gradients of causal_conv's inputs; None where there is no such input."""

    x: torch.Tensor
    weight: torch.Tensor
    bias: Optional[torch.Tensor]
    state: Optional[torch.Tensor]


class ScanGrads(NamedTuple):
    """Gradients of selective_scan's inputs; None where there is no such input."""

    u: torch.Tensor
    delta: torch.Tensor
    A: torch.Tensor
    B: torch.Tensor
    C: torch.Tensor
    D: Optional[torch.Tensor]
    z: Optional[torch.Tensor]
    delta_bias: Optional[torch.Tensor]
    state: Optional[torch.Tensor]


def _view(name, t, shape, dtype, device):
    """A tensor of this shape whose last dimension is contiguous; the others
    may have any strides that do not run backwards."""
    if t is None:
        raise ValueError(f"{name} is required")
    # every check in one expression first; the detailed ones below name the
    # failure
    if t.dtype is dtype and t.shape == shape and t.get_device() == device.index \
            and (t.stride(-1) == 1 or t.shape[-1] <= 1):
        return t
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    raise ValueError(f"{name} must be contiguous in its last dimension")


def _dense_in(name, t, shape, dtype, device):
    """A dense tensor's address, or 0 for None (an optional input)."""
    if t is None:
        return 0
    if t.dtype is dtype and t.shape == shape and t.get_device() == device.index \
            and t.is_contiguous():
        return t.data_ptr()
    return _steps(name, t, tuple(shape), dtype, device).data_ptr()


def _flags_in(t, shape, device):
    if t is None:
        return 0
    if t.dtype in _FLAG_DTYPES:
        return _dense_in("flags", t, shape, t.dtype, device)
    return _steps("flags", t, tuple(shape), "flag", device).data_ptr()


def _activations(name, t, dims):
    """[num_seqs, channels(, T)] on a GPU; its shape, device and storage type."""
    shape = t.shape
    if len(shape) != dims:
        raise ValueError(f"{name} is [num_seqs, channels{', T' if dims == 3 else ''}]")
    if not t.is_cuda:
        raise ValueError("inputs must be GPU tensors")
    dtype = _real_dtype(name, t)
    if t.stride(-1) != 1 and shape[-1] > 1:
        raise ValueError(f"{name} must be contiguous in its last dimension")
    return shape, t.device, dtype


def _new(out, shape, dtype, device, name="out"):
    """An output tensor, the caller's or a new one."""
    if out is None:
        return torch.empty(tuple(shape), dtype=dtype, device=device)
    return _out(out, tuple(shape), device, dtype, name=name)


def _new_step(out, like, shape, dtype, device, name):
    """As _new for one step's output; the cheapest allocation where it fits."""
    if out is None and like.is_contiguous():
        return torch.empty_like(like)
    return _new(out, shape, dtype, device, name)


def _grouped(name, t, N, S, last, dtype, dev):
    """B or C as [N, G, S(, T)]; one group may be given without its dimension."""
    if t is None:
        raise ValueError(f"{name} is required")
    full = 3 + len(last)
    if t.dim() == full - 1:
        t = t.unsqueeze(1)
    if t.dim() != full:
        raise ValueError(f"{name} is [num_seqs, groups, states{', T' if last else ''}]")
    return _view(name, t, (N, t.shape[1], S, *last), dtype, dev)


# Tells autograd that tensors (a sequence) were written: a backward pass that has
# saved one refuses to use it.  Torch's own, without the public function's wrapper.
_written = getattr(torch._C, "_increment_version", torch.autograd.graph.increment_version)


def _written_outputs(*tensors):
    """As _written, for outputs that the caller may have brought."""
    _written([t for t in tensors if t is not None])


def _scratch(nbytes, dev):
    """A workspace that needs no initialisation; torch's allocator keeps it
    alive on the current stream."""
    return torch.empty(max(nbytes, 16), dtype=torch.uint8, device=dev)


# ------------------------------------------------------------- the convolution
def _taps(weight):
    if weight is None or weight.dim() != 2:
        raise ValueError("weight is [channels, width]")
    W = weight.shape[1]
    if not 2 <= W <= 4:
        raise ValueError(f"weight has {W} taps, expected 2, 3 or 4")
    return W


def _conv_inputs(x, weight, bias, state, flags, convention, lengths, silu):
    """The record's fields up to lengths, and what the outputs are made of."""
    shape, dev, dtype = _activations("x", x, 3)
    N, D, T = shape
    W = _taps(weight)
    fields = (N, D, T, W, 1 if silu else 0, REAL_DTYPES[dtype], int(convention), x.data_ptr(),
              x.stride(0), x.stride(1), _dense_in("weight", weight, (D, W), torch.float32, dev),
              _dense_in("bias", bias, (D,), torch.float32, dev),
              _dense_in("state", state, (N, D, W - 1), dtype, dev),
              _flags_in(flags, (N, T), dev),
              _dense_in("lengths", lengths, (N,), torch.int32, dev))
    return fields, shape, W, dev, dtype


def causal_conv(x, weight, bias=None, state=None, flags=None, convention=RESET_ON_START,
                lengths=None, silu=True, with_state=False, out=None, final_state=None):
    """Short causal convolution of each channel, and silu:
    out_t = silu(bias + sum_k weight[k] x[t - (W-1) + k]).

    x [num_seqs, channels, T] (float32, bfloat16 or float16; time contiguous,
    other strides free), weight [channels, W] and bias [channels] float32, W =
    2, 3 or 4; state [num_seqs, channels, W-1] the inputs before the row;
    flags [num_seqs, T] episode boundaries; lengths [num_seqs] int32.
    Returns (out, final state | None)."""
    fields, shape, W, dev, dtype = _conv_inputs(x, weight, bias, state, flags, convention,
                                                lengths, silu)
    o = _new(out, shape, dtype, dev)
    f = None
    if with_state or final_state is not None:
        f = _new(final_state, (shape[0], shape[1], W - 1), dtype, dev, "final_state")
    call = _pack_conv(*fields, o.data_ptr(), _ptr(f), 0, 0, 0, 0, 0, 0, 0, 0)
    _check(lib().rlca_causal_conv(call, _current_stream(dev)), "rlca_causal_conv")
    if out is not None or final_state is not None:
        _written_outputs(out, final_state)
    return o, f


def causal_conv_backward(grad_out, x, weight, bias=None, state=None, flags=None,
                         convention=RESET_ON_START, lengths=None, silu=True, grad_state=None):
    """Gradients of causal_conv with these inputs, from its output's gradient
    (and, with grad_state, its final state's).  Returns ConvGrads."""
    fields, shape, W, dev, dtype = _conv_inputs(x, weight, bias, state, flags, convention,
                                                lengths, silu)
    N, D, _ = shape
    g = _view("grad_out", grad_out, shape, dtype, dev)
    gf = _dense_in("grad_state", grad_state, (N, D, W - 1), dtype, dev)
    grads = ConvGrads(
        x=_new(None, shape, dtype, dev), weight=_new(None, (D, W), torch.float32, dev),
        bias=None if bias is None else _new(None, (D,), torch.float32, dev),
        state=None if state is None else _new(None, (N, D, W - 1), dtype, dev))
    call = _pack_conv(*fields, 0, 0, g.data_ptr(), g.stride(0), g.stride(1), gf,
                      *(_ptr(t) for t in grads))
    ws = _scratch(lib().rlca_causal_conv_backward_workspace_size(call), dev)
    _check(lib().rlca_causal_conv_backward(call, ws.data_ptr(), ws.numel(),
                                           _current_stream(dev)), "rlca_causal_conv_backward")
    return grads


def _pool(state, slots, N, shape, dtype, dev):
    """A step's pool of states [places, ...]: its number of places and address."""
    if state is None or state.dim() != 3:
        raise ValueError(f"state is [places, {', '.join(str(n) for n in shape)}]")
    places = state.shape[0]
    at = _dense_in("state", state, (places, *shape), dtype, dev)
    if slots is None and places < N:
        raise ValueError(f"state has {places} places for {N} sequences")
    return places, at


def causal_conv_step(x, weight, bias, state, slots=None, flags=None, silu=True, out=None):
    """One step of causal_conv for each sequence: x [num_seqs, channels], bias
    [channels] or None, state [places, channels, W-1] updated in place.
    slots [num_seqs] int32 gives each sequence's place in the pool (one out of
    range is an empty seat: output 0); flags [num_seqs] marks sequences whose
    episode begins with this step.  Returns out [num_seqs, channels]."""
    shape, dev, dtype = _activations("x", x, 2)
    N, D = shape
    W = _taps(weight)
    w = _dense_in("weight", weight, (D, W), torch.float32, dev)
    b = _dense_in("bias", bias, (D,), torch.float32, dev)
    places, s = _pool(state, slots, N, (D, W - 1), dtype, dev)
    i = _dense_in("slots", slots, (N,), torch.int32, dev)
    f = _flags_in(flags, (N,), dev)
    o = _new_step(out, x, shape, dtype, dev, "out")
    call = _pack_conv_step(N, D, places, W, 1 if silu else 0, REAL_DTYPES[dtype], x.data_ptr(),
                           x.stride(0), w, b, s, i, f, o.data_ptr())
    _check(lib().rlca_causal_conv_step(call, _current_stream(dev)), "rlca_causal_conv_step")
    _written((state,) if out is None else (state, out))
    return o


# -------------------------------------------------------------------- the scan
def _scan_params(A, D, delta_bias, channels, dev):
    if A is None or A.dim() != 2:
        raise ValueError("A is [channels, states]")
    S = A.shape[1]
    if not 1 <= S <= MAX_STATES:
        raise ValueError(f"A has {S} states, expected 1 to {MAX_STATES}")
    return (S, _dense_in("A", A, (channels, S), torch.float32, dev),
            _dense_in("D", D, (channels,), torch.float32, dev),
            _dense_in("delta_bias", delta_bias, (channels,), torch.float32, dev))


def _groups(B, C, channels):
    G = B.shape[1]
    if C.shape[1] != G:
        raise ValueError(f"B has {G} groups and C {C.shape[1]}")
    if G == 0 or channels % G != 0:
        raise ValueError(f"{channels} channels do not divide into {G} groups")
    return G


def _scan_inputs(u, delta, A, B, C, D, z, delta_bias, state, flags, convention, lengths,
                 softplus):
    """The record's fields up to lengths, and what the outputs are made of."""
    shape, dev, dtype = _activations("u", u, 3)
    N, channels, T = shape
    delta = _view("delta", delta, shape, dtype, dev)
    S, a, d, bias = _scan_params(A, D, delta_bias, channels, dev)
    B = _grouped("B", B, N, S, (T,), dtype, dev)
    C = _grouped("C", C, N, S, (T,), dtype, dev)
    G = _groups(B, C, channels)
    gate = (0, 0, 0)
    if z is not None:
        z = _view("z", z, shape, dtype, dev)
        gate = (z.data_ptr(), z.stride(0), z.stride(1))
    fields = (N, channels, T, S, G, 1 if softplus else 0, REAL_DTYPES[dtype], int(convention),
              u.data_ptr(), delta.data_ptr(), u.stride(0), u.stride(1), delta.stride(0),
              delta.stride(1), a, B.data_ptr(), C.data_ptr(), *B.stride()[:3], *C.stride()[:3],
              d, bias, *gate, _dense_in("state", state, (N, channels, S), torch.float32, dev),
              _flags_in(flags, (N, T), dev),
              _dense_in("lengths", lengths, (N,), torch.int32, dev))
    return fields, shape, S, G, dev, dtype


def selective_scan(u, delta, A, B, C, D=None, z=None, delta_bias=None, state=None, flags=None,
                   convention=RESET_ON_START, lengths=None, softplus=True, with_state=False,
                   with_checkpoints=False, y=None, final_state=None):
    """Selective state space scan of each channel:
    dt = softplus(delta + delta_bias), h_t = exp(dt_t A) h_{t-1} + dt_t u_t B_t,
    y_t = (C_t . h_t + D u_t) silu(z_t).

    u, delta and z (optional gate) [num_seqs, channels, T] (float32, bfloat16
    or float16; time contiguous, other strides free); B and C [num_seqs,
    groups, states, T] (or without groups) of that type; A [channels, states],
    D and delta_bias [channels] and state [num_seqs, channels, states]
    float32; flags [num_seqs, T] episode boundaries; lengths [num_seqs] int32.
    Returns (y, final state | None, checkpoints | None); the checkpoints are
    what selective_scan_backward needs of this call."""
    fields, shape, S, _, dev, dtype = _scan_inputs(u, delta, A, B, C, D, z, delta_bias, state,
                                                   flags, convention, lengths, softplus)
    o = _new(y, shape, dtype, dev, "y")
    f = c = None
    if with_state or final_state is not None:
        f = _new(final_state, (shape[0], shape[1], S), torch.float32, dev, "final_state")
    if with_checkpoints:
        n = lib().rlca_selective_scan_checkpoints_size(_pack_scan(*fields, *(0,) * 16))
        c = _new(None, (n // 4,), torch.float32, dev)
    call = _pack_scan(*fields, o.data_ptr(), _ptr(f), _ptr(c), *(0,) * 13)
    _check(lib().rlca_selective_scan(call, _current_stream(dev)), "rlca_selective_scan")
    if y is not None or final_state is not None:
        _written_outputs(y, final_state)
    return o, f, c


def selective_scan_backward(grad_y, u, delta, A, B, C, checkpoints, D=None, z=None,
                            delta_bias=None, state=None, flags=None, convention=RESET_ON_START,
                            lengths=None, softplus=True, grad_state=None):
    """Gradients of selective_scan with these inputs, from its output's
    gradient (and, with grad_state, its final state's) and the checkpoints it
    returned.  Returns ScanGrads; B's and C's have four dimensions."""
    fields, shape, S, G, dev, dtype = _scan_inputs(u, delta, A, B, C, D, z, delta_bias, state,
                                                   flags, convention, lengths, softplus)
    N, channels, T = shape
    g = _view("grad_y", grad_y, shape, dtype, dev)
    gf = _dense_in("grad_state", grad_state, (N, channels, S), torch.float32, dev)
    if checkpoints is None:
        raise ValueError("checkpoints is required")
    n = lib().rlca_selective_scan_checkpoints_size(_pack_scan(*fields, *(0,) * 16)) // 4
    c = _dense_in("checkpoints", checkpoints, (n,), torch.float32, dev)
    f32 = torch.float32

    def shared():
        # without channels the library writes nothing: sums of no terms
        if channels == 0:
            return torch.zeros(N, G, S, T, dtype=dtype, device=dev)
        return _new(None, (N, G, S, T), dtype, dev)

    grads = ScanGrads(
        u=_new(None, shape, dtype, dev), delta=_new(None, shape, dtype, dev),
        A=_new(None, (channels, S), f32, dev), B=shared(), C=shared(),
        D=None if D is None else _new(None, (channels,), f32, dev),
        z=None if z is None else _new(None, shape, dtype, dev),
        delta_bias=None if delta_bias is None else _new(None, (channels,), f32, dev),
        state=None if state is None else _new(None, (N, channels, S), f32, dev))
    call = _pack_scan(*fields, 0, 0, c, g.data_ptr(), g.stride(0), g.stride(1), gf,
                      grads.u.data_ptr(), grads.delta.data_ptr(), grads.A.data_ptr(),
                      grads.B.data_ptr(), grads.C.data_ptr(), _ptr(grads.D),
                      _ptr(grads.delta_bias), _ptr(grads.z), _ptr(grads.state))
    ws = _scratch(lib().rlca_selective_scan_backward_workspace_size(call), dev)
    _check(lib().rlca_selective_scan_backward(call, ws.data_ptr(), ws.numel(),
                                              _current_stream(dev)),
           "rlca_selective_scan_backward")
    return grads


def selective_step(u, delta, A, B, C, state, D=None, z=None, delta_bias=None, slots=None,
                   flags=None, softplus=True, y=None):
    """One step of selective_scan for each sequence: u, delta and z [num_seqs,
    channels], B and C [num_seqs, groups, states] (or without groups), state
    [places, channels, states] float32 updated in place.  slots and flags as
    for causal_conv_step.  Returns y [num_seqs, channels]."""
    shape, dev, dtype = _activations("u", u, 2)
    N, channels = shape
    delta = _view("delta", delta, shape, dtype, dev)
    S, a, d, bias = _scan_params(A, D, delta_bias, channels, dev)
    B = _grouped("B", B, N, S, (), dtype, dev)
    C = _grouped("C", C, N, S, (), dtype, dev)
    G = _groups(B, C, channels)
    places, s = _pool(state, slots, N, (channels, S), torch.float32, dev)
    i = _dense_in("slots", slots, (N,), torch.int32, dev)
    f = _flags_in(flags, (N,), dev)
    gate = (0, 0)
    if z is not None:
        gate = (_view("z", z, shape, dtype, dev).data_ptr(), z.stride(0))
    o = _new_step(y, u, shape, dtype, dev, "y")
    call = _pack_scan_step(N, channels, places, S, G, 1 if softplus else 0, REAL_DTYPES[dtype],
                           u.data_ptr(), delta.data_ptr(), u.stride(0), delta.stride(0), a,
                           B.data_ptr(), C.data_ptr(), B.stride(0), B.stride(1), C.stride(0),
                           C.stride(1), d, bias, *gate, s, i, f, o.data_ptr())
    _check(lib().rlca_selective_step(call, _current_stream(dev)), "rlca_selective_step")
    _written((state,) if y is None else (state, y))
    return o


# ---------------------------------------------------------------- the clipping
_clip_locks = {}  # by the key of the workspace


def _clip_workspace(dev, stream):
    """A zero-filled workspace per (device, stream), shared with no other call
    kind, and its lock: the running total and the scale live in it from a call's
    first launch to its last, so a call holds the lock over all of them (threads
    may share a stream).  A call captured into a graph gets its own, which the
    graph fills and keeps: graphs may be replayed on any stream, and nothing is
    filled while one is captured."""
    if torch.cuda.is_current_stream_capturing():
        return (torch.zeros(CLIP_WORKSPACE_BYTES, dtype=torch.uint8, device=dev),
                threading.Lock())
    key = (dev.index, stream, "clip")
    with _workspaces_lock:
        ws = _workspaces.get(key)
        if ws is None:
            ws = torch.zeros(CLIP_WORKSPACE_BYTES, dtype=torch.uint8, device=dev)
            _workspaces[key], _clip_locks[key] = ws, threading.Lock()
        return ws, _clip_locks[key]


def _dense(t):
    """Whether the tensor's elements fill one run of memory in some order."""
    order = sorted(range(t.dim()), key=lambda i: (t.stride(i), t.shape[i]))
    return t.permute(order[::-1]).is_contiguous()


def clip_grad_norm(grads, max_norm, eps=1e-6, out=None, norm=None):
    """Scale gradients to a global 2-norm of at most max_norm: every tensor
    times min(1, max_norm / (norm + eps)), in place or, with `out` (a list of
    tensors like `grads`), into those.  The tensors (float32, bfloat16 or
    float16, mixed freely, dense in memory) count as one vector; None, the
    gradient of a parameter that has none, is left out.  Returns the norm before
    the scaling, a float64 tensor [1] on the device; nothing synchronizes.
    max_norm = inf computes the norm only."""
    given = list(grads)
    outs = None if out is None else list(out)
    if outs is not None and len(outs) != len(given):
        raise ValueError(f"out has {len(outs)} tensors, expected {len(given)}")
    grads = [g for g in given if g is not None]
    if outs is not None and len(grads) != len(given):
        if any((g is None) != (o is None) for g, o in zip(given, outs)):
            raise ValueError("out must be None where grads is, and only there")
        outs = [o for o in outs if o is not None]
    if not grads:
        raise ValueError("grads is empty")
    dev = grads[0].device
    if dev.type != "cuda":
        raise ValueError("inputs must be GPU tensors")
    # Properties of all tensors at once, the checks over those lists; a loop
    # names the tensor that fails one.
    tensor = torch.Tensor
    dtypes = [g.dtype for g in grads]
    codes = list(map(REAL_DTYPES.get, dtypes))
    addresses = list(map(tensor.data_ptr, grads))
    if None in codes or set(map(tensor.get_device, grads)) != {dev.index} \
            or not (all(map(tensor.is_contiguous, grads)) or all(map(_dense, grads))):
        for i, g in enumerate(grads):
            _real_dtype(f"grads[{i}]", g)
            if g.device != dev or not _dense(g):
                raise ValueError(f"grads[{i}] must be dense in memory and on {dev}")
    targets = addresses
    if outs is not None:
        targets = list(map(tensor.data_ptr, outs))
        if set(map(tensor.get_device, outs)) != {dev.index} \
                or [o.dtype for o in outs] != dtypes \
                or [o.shape for o in outs] != [g.shape for g in grads] \
                or list(map(tensor.stride, outs)) != list(map(tensor.stride, grads)):
            raise ValueError("every tensor of out must be like the one of grads: device, type, "
                             "shape and strides")
    # address, output's address, count, type: four 8-byte fields a tensor
    packed = array("Q", [0]) * (4 * len(grads))
    packed[0::4] = array("Q", addresses)
    packed[1::4] = array("Q", targets)
    packed[2::4] = array("Q", list(map(tensor.numel, grads)))
    packed[3::4] = array("Q", codes)
    n = _out(norm, (1,), dev, torch.float64, name="norm")
    h = _current_stream(dev)
    ws, lock = _clip_workspace(dev, h)
    with lock:
        status = lib().rlca_clip_grad_norm(packed.buffer_info()[0], len(grads), max_norm, eps,
                                           n.data_ptr(), ws.data_ptr(), ws.numel(), h)
    _check(status, "rlca_clip_grad_norm")
    if not math.isinf(max_norm):
        _written(grads if outs is None else outs)
    if norm is not None:
        _written((norm,))
    return n
