"""Binding of the sequence-model operators of librlca.so (include/rlca.h): the
causal convolution, the selective scan, their single-step forms and gradients,
and the clipping of gradients by their global norm.

Argument marshalling only, as in rlca.py: shape / dtype / device checks, output
and workspace allocation through torch, and the current HIP stream.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple, Optional

import torch

from .rlca import (
    REAL_DTYPES, RESET_ON_START, SIGNATURES, SIZE_QUERIES, _check, _current_stream, _out, _p,
    _ptr, _real_dtype, _steps, _sz, _workspaces, _workspaces_lock, lib,
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


_conv = ctypes.POINTER(ConvCall)
_scan = ctypes.POINTER(ScanCall)
SIGNATURES.update({
    "rlca_causal_conv": [_conv, _p],
    "rlca_causal_conv_backward": [_conv, _p, _sz, _p],
    "rlca_selective_scan": [_scan, _p],
    "rlca_selective_scan_backward": [_scan, _p, _sz, _p],
    "rlca_causal_conv_step": [ctypes.POINTER(ConvStepCall), _p],
    "rlca_selective_step": [ctypes.POINTER(ScanStepCall), _p],
    "rlca_clip_grad_norm": [ctypes.POINTER(GradTensor), _i64, ctypes.c_double, ctypes.c_double,
                            _p, _p, _sz, _p],
})
SIZE_QUERIES.update({
    "rlca_causal_conv_backward_workspace_size": [_conv],
    "rlca_selective_scan_checkpoints_size": [_scan],
    "rlca_selective_scan_backward_workspace_size": [_scan],
})


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
    if t.dtype is dtype and t.shape == shape and t.device == device \
            and (t.stride(-1) == 1 or t.shape[-1] <= 1):
        return t
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    raise ValueError(f"{name} must be contiguous in its last dimension")


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


def _episodes(flags, lengths, N, T, dev):
    return (_steps("flags", flags, (N, T), "flag", dev, optional=True),
            _steps("lengths", lengths, (N,), torch.int32, dev, optional=True))


def _f32(name, t, shape, dev, optional=False):
    return _steps(name, t, shape, torch.float32, dev, optional=optional)


def _grouped(name, t, N, S, last, dtype, dev):
    """B or C as [N, G, S(, T)]; one group may be given without its dimension."""
    if t is None:
        raise ValueError(f"{name} is required")
    full = 3 + len(last)
    if t.dim() == full - 1:
        t = t.unsqueeze(1)
    if t.dim() != full:
        raise ValueError(f"{name} is [num_seqs, groups, states{', T' if last else ''}]")
    return _view(name, t, (N, t.shape[1], S) + last, dtype, dev)


def _scratch(nbytes, dev):
    """A workspace that needs no initialisation; torch's allocator keeps it
    alive on the current stream."""
    return torch.empty(max(nbytes, 16), dtype=torch.uint8, device=dev)


# ------------------------------------------------------------- the convolution
def _conv_call(x, weight, bias, state, flags, convention, lengths, silu):
    (N, D, T), dev, dtype = _activations("x", x, 3)
    if weight is None or weight.dim() != 2:
        raise ValueError("weight is [channels, width]")
    W = weight.shape[1]
    if not 2 <= W <= 4:
        raise ValueError(f"weight has {W} taps, expected 2, 3 or 4")
    w = _f32("weight", weight, (D, W), dev)
    b = _f32("bias", bias, (D,), dev, optional=True)
    s = _steps("state", state, (N, D, W - 1), dtype, dev, optional=True)
    f, ln = _episodes(flags, lengths, N, T, dev)
    call = ConvCall(N, D, T, W, 1 if silu else 0, REAL_DTYPES[dtype], int(convention),
                    x.data_ptr(), x.stride(0), x.stride(1), w.data_ptr(), _ptr(b), _ptr(s),
                    _ptr(f), _ptr(ln))
    return call, (N, D, T, W), dev, dtype


def causal_conv(x, weight, bias=None, state=None, flags=None, convention=RESET_ON_START,
                lengths=None, silu=True, with_state=False, out=None, final_state=None):
    """Short causal convolution of each channel, and silu:
    out_t = silu(bias + sum_k weight[k] x[t - (W-1) + k]).

    x [num_seqs, channels, T] (float32, bfloat16 or float16; time contiguous,
    other strides free), weight [channels, W] and bias [channels] float32, W =
    2, 3 or 4; state [num_seqs, channels, W-1] the inputs before the row;
    flags [num_seqs, T] episode boundaries; lengths [num_seqs] int32.
    Returns (out, final state | None)."""
    call, (N, D, T, W), dev, dtype = _conv_call(x, weight, bias, state, flags, convention,
                                                lengths, silu)
    o = _out(out, (N, D, T), dev, dtype)
    f = None
    if with_state or final_state is not None:
        f = _out(final_state, (N, D, W - 1), dev, dtype, name="final_state")
    call.out, call.final_state = _ptr(o), _ptr(f)
    _check(lib().rlca_causal_conv(ctypes.byref(call), _current_stream(dev)), "rlca_causal_conv")
    return o, f


def causal_conv_backward(grad_out, x, weight, bias=None, state=None, flags=None,
                         convention=RESET_ON_START, lengths=None, silu=True, grad_state=None):
    """Gradients of causal_conv with these inputs, from its output's gradient
    (and, with grad_state, its final state's).  Returns ConvGrads."""
    call, (N, D, T, W), dev, dtype = _conv_call(x, weight, bias, state, flags, convention,
                                                lengths, silu)
    g = _view("grad_out", grad_out, (N, D, T), dtype, dev)
    gf = _steps("grad_state", grad_state, (N, D, W - 1), dtype, dev, optional=True)
    grads = ConvGrads(
        x=torch.empty((N, D, T), dtype=dtype, device=dev),
        weight=torch.empty((D, W), dtype=torch.float32, device=dev),
        bias=None if bias is None else torch.empty(D, dtype=torch.float32, device=dev),
        state=None if state is None else torch.empty((N, D, W - 1), dtype=dtype, device=dev))
    call.grad_out, call.grad_stride_seq, call.grad_stride_channel = _ptr(g), g.stride(0), \
        g.stride(1)
    call.grad_final_state = _ptr(gf)
    call.grad_x, call.grad_weight = _ptr(grads.x), _ptr(grads.weight)
    call.grad_bias, call.grad_state = _ptr(grads.bias), _ptr(grads.state)
    ws = _scratch(lib().rlca_causal_conv_backward_workspace_size(ctypes.byref(call)), dev)
    _check(lib().rlca_causal_conv_backward(ctypes.byref(call), _ptr(ws), ws.numel(),
                                           _current_stream(dev)), "rlca_causal_conv_backward")
    return grads


def _seats(state, slots, flags, N, shape, dtype, dev):
    """A step's pool of states [places, ...], its slots and its start flags."""
    if state is None or state.dim() != 1 + len(shape):
        raise ValueError(f"state is [places, {', '.join(str(n) for n in shape)}]")
    s = _steps("state", state, (state.shape[0],) + shape, dtype, dev)
    i = _steps("slots", slots, (N,), torch.int32, dev, optional=True)
    f = _steps("flags", flags, (N,), "flag", dev, optional=True)
    if i is None and s.shape[0] < N:
        raise ValueError(f"state has {s.shape[0]} places for {N} sequences")
    return s, i, f


def causal_conv_step(x, weight, bias, state, slots=None, flags=None, silu=True, out=None):
    """One step of causal_conv for each sequence: x [num_seqs, channels], bias
    [channels] or None, state [places, channels, W-1] updated in place.
    slots [num_seqs] int32 gives each sequence's place in the pool (one out of
    range is an empty seat: output 0); flags [num_seqs] marks sequences whose
    episode begins with this step.  Returns out [num_seqs, channels]."""
    (N, D), dev, dtype = _activations("x", x, 2)
    if weight is None or weight.dim() != 2:
        raise ValueError("weight is [channels, width]")
    W = weight.shape[1]
    if not 2 <= W <= 4:
        raise ValueError(f"weight has {W} taps, expected 2, 3 or 4")
    w = _f32("weight", weight, (D, W), dev)
    b = _f32("bias", bias, (D,), dev, optional=True)
    s, i, f = _seats(state, slots, flags, N, (D, W - 1), dtype, dev)
    o = _out(out, (N, D), dev, dtype)
    call = ConvStepCall(N, D, s.shape[0], W, 1 if silu else 0, REAL_DTYPES[dtype], x.data_ptr(),
                        x.stride(0), w.data_ptr(), _ptr(b), s.data_ptr(), _ptr(i), _ptr(f),
                        o.data_ptr())
    _check(lib().rlca_causal_conv_step(ctypes.byref(call), _current_stream(dev)),
           "rlca_causal_conv_step")
    return o


# -------------------------------------------------------------------- the scan
def _scan_params(A, D, delta_bias, channels, dev):
    if A is None or A.dim() != 2:
        raise ValueError("A is [channels, states]")
    S = A.shape[1]
    if not 1 <= S <= MAX_STATES:
        raise ValueError(f"A has {S} states, expected 1 to {MAX_STATES}")
    return (S, _f32("A", A, (channels, S), dev), _f32("D", D, (channels,), dev, optional=True),
            _f32("delta_bias", delta_bias, (channels,), dev, optional=True))


def _groups(B, C, channels):
    G = B.shape[1]
    if C.shape[1] != G:
        raise ValueError(f"B has {G} groups and C {C.shape[1]}")
    if G == 0 or channels % G != 0:
        raise ValueError(f"{channels} channels do not divide into {G} groups")
    return G


def _scan_call(u, delta, A, B, C, D, z, delta_bias, flags, convention, lengths, softplus):
    (N, channels, T), dev, dtype = _activations("u", u, 3)
    shape = (N, channels, T)
    delta = _view("delta", delta, shape, dtype, dev)
    S, A, D, delta_bias = _scan_params(A, D, delta_bias, channels, dev)
    B = _grouped("B", B, N, S, (T,), dtype, dev)
    C = _grouped("C", C, N, S, (T,), dtype, dev)
    G = _groups(B, C, channels)
    if z is not None:
        z = _view("z", z, shape, dtype, dev)
    f, ln = _episodes(flags, lengths, N, T, dev)
    gate = (None, 0, 0) if z is None else (z.data_ptr(), *z.stride()[:2])
    call = ScanCall(N, channels, T, S, G, 1 if softplus else 0, REAL_DTYPES[dtype],
                    int(convention), u.data_ptr(), delta.data_ptr(), *u.stride()[:2],
                    *delta.stride()[:2], A.data_ptr(), B.data_ptr(), C.data_ptr(),
                    *B.stride()[:3], *C.stride()[:3], _ptr(D), _ptr(delta_bias), *gate, None,
                    _ptr(f), _ptr(ln))
    return call, (N, channels, T, S, G), dev, dtype


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
    call, (N, channels, T, S, _), dev, dtype = _scan_call(
        u, delta, A, B, C, D, z, delta_bias, flags, convention, lengths, softplus)
    s = _f32("state", state, (N, channels, S), dev, optional=True)
    o = _out(y, (N, channels, T), dev, dtype, name="y")
    f = c = None
    if with_state or final_state is not None:
        f = _out(final_state, (N, channels, S), dev, name="final_state")
    if with_checkpoints:
        c = torch.empty(lib().rlca_selective_scan_checkpoints_size(ctypes.byref(call)) // 4,
                        dtype=torch.float32, device=dev)
    call.state, call.y, call.final_state, call.checkpoints = _ptr(s), _ptr(o), _ptr(f), _ptr(c)
    _check(lib().rlca_selective_scan(ctypes.byref(call), _current_stream(dev)),
           "rlca_selective_scan")
    return o, f, c


def selective_scan_backward(grad_y, u, delta, A, B, C, checkpoints, D=None, z=None,
                            delta_bias=None, state=None, flags=None, convention=RESET_ON_START,
                            lengths=None, softplus=True, grad_state=None):
    """Gradients of selective_scan with these inputs, from its output's
    gradient (and, with grad_state, its final state's) and the checkpoints it
    returned.  Returns ScanGrads; B's and C's have four dimensions."""
    call, (N, channels, T, S, G), dev, dtype = _scan_call(
        u, delta, A, B, C, D, z, delta_bias, flags, convention, lengths, softplus)
    g = _view("grad_y", grad_y, (N, channels, T), dtype, dev)
    gf = _f32("grad_state", grad_state, (N, channels, S), dev, optional=True)
    _f32("state", state, (N, channels, S), dev, optional=True)
    n = lib().rlca_selective_scan_checkpoints_size(ctypes.byref(call)) // 4
    c = _f32("checkpoints", checkpoints, (n,), dev)

    def like(*shape, dtype=torch.float32):
        return torch.empty(shape, dtype=dtype, device=dev)

    rows = (N, channels, T)
    grads = ScanGrads(
        u=like(*rows, dtype=dtype), delta=like(*rows, dtype=dtype), A=like(channels, S),
        B=like(N, G, S, T, dtype=dtype), C=like(N, G, S, T, dtype=dtype),
        D=None if D is None else like(channels),
        z=None if z is None else like(*rows, dtype=dtype),
        delta_bias=None if delta_bias is None else like(channels),
        state=None if state is None else like(N, channels, S))
    call.checkpoints, call.grad_y = _ptr(c), _ptr(g)
    call.grad_stride_seq, call.grad_stride_channel = g.stride(0), g.stride(1)
    call.grad_final_state = _ptr(gf)
    for name, t in zip(grads._fields, grads):
        setattr(call, "grad_" + name, _ptr(t))
    ws = _scratch(lib().rlca_selective_scan_backward_workspace_size(ctypes.byref(call)), dev)
    _check(lib().rlca_selective_scan_backward(ctypes.byref(call), _ptr(ws), ws.numel(),
                                              _current_stream(dev)),
           "rlca_selective_scan_backward")
    return grads


def selective_step(u, delta, A, B, C, state, D=None, z=None, delta_bias=None, slots=None,
                   flags=None, softplus=True, y=None):
    """One step of selective_scan for each sequence: u, delta and z [num_seqs,
    channels], B and C [num_seqs, groups, states] (or without groups), state
    [places, channels, states] float32 updated in place.  slots and flags as
    for causal_conv_step.  Returns y [num_seqs, channels]."""
    (N, channels), dev, dtype = _activations("u", u, 2)
    delta = _view("delta", delta, (N, channels), dtype, dev)
    S, A, D, delta_bias = _scan_params(A, D, delta_bias, channels, dev)
    B = _grouped("B", B, N, S, (), dtype, dev)
    C = _grouped("C", C, N, S, (), dtype, dev)
    G = _groups(B, C, channels)
    s, i, f = _seats(state, slots, flags, N, (channels, S), torch.float32, dev)
    o = _out(y, (N, channels), dev, dtype, name="y")
    gate = (None, 0)
    if z is not None:
        gate = (_view("z", z, (N, channels), dtype, dev).data_ptr(), z.stride(0))
    call = ScanStepCall(N, channels, s.shape[0], S, G, 1 if softplus else 0, REAL_DTYPES[dtype],
                        u.data_ptr(), delta.data_ptr(), u.stride(0), delta.stride(0),
                        A.data_ptr(), B.data_ptr(), C.data_ptr(), *B.stride()[:2],
                        *C.stride()[:2], _ptr(D), _ptr(delta_bias), *gate, s.data_ptr(), _ptr(i),
                        _ptr(f), o.data_ptr())
    _check(lib().rlca_selective_step(ctypes.byref(call), _current_stream(dev)),
           "rlca_selective_step")
    return o


# ---------------------------------------------------------------- the clipping
def _clip_workspace(dev, stream):
    """A zero-filled workspace per (device, stream), shared with no other call
    kind: the running total and the scale live in it between launches."""
    key = (dev.index, stream, "clip")
    with _workspaces_lock:
        ws = _workspaces.get(key)
        if ws is None:
            ws = torch.zeros(CLIP_WORKSPACE_BYTES, dtype=torch.uint8, device=dev)
            _workspaces[key] = ws
    return ws


def _dense(t):
    """Whether the tensor's elements fill one run of memory in some order."""
    order = sorted(range(t.dim()), key=lambda i: (t.stride(i), t.shape[i]))
    return t.permute(order[::-1]).is_contiguous()


def clip_grad_norm(grads, max_norm, eps=1e-6, out=None, norm=None):
    """Scale gradients to a global 2-norm of at most max_norm: every tensor
    times min(1, max_norm / (norm + eps)), in place or, with `out` (a list of
    tensors like `grads`), into those.  The tensors (float32, bfloat16 or
    float16, mixed freely, dense in memory) count as one vector.  Returns the
    norm before the scaling, a float64 tensor [1] on the device; nothing
    synchronizes.  max_norm = inf computes the norm only."""
    grads = list(grads)
    if not grads:
        raise ValueError("grads is empty")
    dev = grads[0].device
    if dev.type != "cuda":
        raise ValueError("inputs must be GPU tensors")
    outs = grads if out is None else list(out)
    if len(outs) != len(grads):
        raise ValueError(f"out has {len(outs)} tensors, expected {len(grads)}")
    entries = []
    for i, (g, o) in enumerate(zip(grads, outs)):
        dtype = REAL_DTYPES.get(g.dtype)
        if dtype is None or g.device != dev or not (g.is_contiguous() or _dense(g)):
            _real_dtype(f"grads[{i}]", g)
            raise ValueError(f"grads[{i}] must be dense in memory and on {dev}")
        at = to = g.data_ptr()
        if o is not g:
            if o.dtype != g.dtype or o.shape != g.shape or o.stride() != g.stride() \
                    or o.device != dev:
                raise ValueError(f"out[{i}] must be like grads[{i}]")
            to = o.data_ptr()
        entries.append((at, to, g.numel(), dtype))
    arr = (GradTensor * len(entries))(*entries)
    n = _out(norm, (1,), dev, torch.float64, name="norm")
    h = _current_stream(dev)
    ws = _clip_workspace(dev, h)
    _check(lib().rlca_clip_grad_norm(arr, len(grads), float(max_norm), float(eps), _ptr(n),
                                     _ptr(ws), ws.numel(), h), "rlca_clip_grad_norm")
    return n
