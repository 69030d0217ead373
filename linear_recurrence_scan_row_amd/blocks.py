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
from array import array
from typing import NamedTuple, Optional

import torch

from .rlca import (
    REAL_DTYPES, RESET_ON_START, SIGNATURES, SIZE_QUERIES, _check, _current_stream, _p, _sz, lib,
)
from .sequence import (
    _activations, _dense_in, _flags_in, _new, _new_step, _ptr, _scratch, _view, _written,
    _written_outputs,
)

MAX_BEAMS = 64

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


class NormCall(ctypes.Structure):
    """rlca_norm_call of include/rlca.h."""

    _fields_ = [
        ("num_seqs", _i64), ("channels", _i64), ("T", _i64), ("dtype", _i32), ("eps", _f64),
        ("x", _p), ("x_stride_seq", _i64), ("x_stride_channel", _i64), ("residual", _p),
        ("residual_stride_seq", _i64), ("residual_stride_channel", _i64), ("weight", _p),
        ("lengths", _p), ("out", _p), ("out8", _p), ("scale", _p), ("sum", _p), ("grad_out", _p),
        ("grad_stride_seq", _i64), ("grad_stride_channel", _i64), ("grad_sum", _p),
        ("grad_sum_stride_seq", _i64), ("grad_sum_stride_channel", _i64), ("grad_x", _p),
        ("grad_weight", _p),
    ]


class BeamCall(ctypes.Structure):
    """rlca_beam_call of include/rlca.h."""

    _fields_ = [
        ("num_searches", _i64), ("beams", _i64), ("vocab", _i64), ("picks", _i32),
        ("dtype", _i32), ("pad_token", _i32), ("logits", _p), ("logits_stride_search", _i64),
        ("logits_stride_beam", _i64), ("scores", _p), ("finished", _p), ("out_scores", _p),
        ("out_tokens", _p), ("out_parents", _p),
    ]


class StatePool(ctypes.Structure):
    """rlca_state_pool of include/rlca.h."""

    _fields_ = [("data", _p), ("place_bytes", _i64)]


SIGNATURES.update({
    "rlca_gated_recurrence": [_p, _p, _sz, _p],
    "rlca_gated_recurrence_backward": [_p, _p, _sz, _p],
    "rlca_gated_step": [_p, _p],
    "rlca_rms_norm": [_p, _p],
    "rlca_rms_norm_backward": [_p, _p, _sz, _p],
    "rlca_beam_select": [_p, _p, _sz, _p],
    "rlca_beam_reorder": [_p, _i64, _i64, _i64, _i64, _p, _p, _p, _p],
})
SIZE_QUERIES.update({
    "rlca_gated_recurrence_checkpoints_size": [_p],
    "rlca_gated_recurrence_workspace_size": [_p],
    "rlca_gated_recurrence_backward_workspace_size": [_p],
    "rlca_rms_norm_backward_workspace_size": [_p],
    "rlca_beam_select_workspace_size": [_p],
})


def _packer(cls):
    """As sequence.py's, for records that hold doubles too."""
    codes = {_i64: "q", _i32: "i", _p: "P", _f64: "d"}
    return struct.Struct("@" + "".join(codes[kind] for _, kind in cls._fields_)).pack


_pack_gated, _pack_gated_step, _pack_norm, _pack_beam = (
    _packer(cls) for cls in (GatedCall, GatedStepCall, NormCall, BeamCall))


# The current device's index: torch's own getter is several times cheaper than the
# public function's wrapper around it.
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _run(name, dev, *args):
    """One library call on the current stream of the inputs' device.  Its default
    stream has no handle of its own, so another device is made the current one."""
    call = getattr(lib(), name)
    if _current_device() == dev.index:
        status = call(*args, _current_stream(dev))
    else:
        with torch.cuda.device(dev):
            status = call(*args, _current_stream(dev))
    if status:
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


# -------------------------------------------------------------------- the norm
class NormGrads(NamedTuple):
    """Gradients of rms_norm's inputs: of the normed sum (so of x and residual
    alike) and of the weight, None where there is none."""

    x: torch.Tensor
    weight: Optional[torch.Tensor]


def _rows(name, t, shape, dtype, dev):
    """An array of the norm: its address and the strides of sequences and
    channels.  [num_seqs, channels] stands for [num_seqs, channels, 1]."""
    if t is None:
        return 0, 0, 0
    t = _view(name, t, shape, dtype, dev)
    return t.data_ptr(), t.stride(0), t.stride(1)


def _norm_inputs(x, weight, eps, lengths):
    """The record's fields before x and after the residual, and x's shape."""
    if x is None or x.dim() not in (2, 3):
        raise ValueError("x is [num_seqs, channels, T] or [num_seqs, channels]")
    shape, dev, dtype = _activations("x", x, x.dim())
    N, D = shape[:2]
    T = shape[2] if len(shape) == 3 else 1
    head = (N, D, T, REAL_DTYPES[dtype], float(eps))
    tail = (_dense_in("weight", weight, (D,), torch.float32, dev),
            _dense_in("lengths", lengths, (N,), torch.int32, dev))
    return head, tail, shape, dev, dtype


def _norm(x, weight, residual, eps, lengths, total, out, scale, bits8):
    head, tail, shape, dev, dtype = _norm_inputs(x, weight, eps, lengths)
    o = _new(out, shape, torch.float8_e4m3fn, dev) if bits8 \
        else _new_step(out, x, shape, dtype, dev, "out")
    sc = _new(scale, (shape[0], *shape[2:]), torch.float32, dev, "scale") if bits8 else None
    s = None
    if residual is not None:
        s = _new_step(total, x, shape, dtype, dev, "total")
    elif total is not None:
        raise ValueError("total is given without a residual")
    call = _pack_norm(*head, x.data_ptr(), x.stride(0), x.stride(1),
                      *_rows("residual", residual, shape, dtype, dev), *tail,
                      0 if bits8 else o.data_ptr(), o.data_ptr() if bits8 else 0, _ptr(sc),
                      _ptr(s), *(0,) * 8)
    _run("rlca_rms_norm", dev, call)
    if out is not None or total is not None or scale is not None:
        _written_outputs(out, total, scale)
    return o, sc, s


def rms_norm(x, weight=None, residual=None, eps=1e-6, lengths=None, total=None, out=None):
    """Root-mean-square norm over the channels of each step, after the residual's
    addition: s = x + residual (as it is stored), s / sqrt(mean(s^2) + eps) * weight.

    x and residual [num_seqs, channels, T] (float32, bfloat16 or float16; time
    contiguous, other strides free), or [num_seqs, channels] for single steps (any
    [tokens, channels] array); weight [channels] float32; lengths [num_seqs] int32.
    Returns (out, s), s None without a residual; rms_norm_backward takes s."""
    o, _, s = _norm(x, weight, residual, eps, lengths, total, out, None, False)
    return o, s


def rms_norm_8bit(x, weight=None, residual=None, eps=1e-6, lengths=None, total=None, out=None,
                  scale=None):
    """rms_norm with its output in 8 bits: (out, scale, s), out float8_e4m3fn like x,
    scale [num_seqs, T] (or [num_seqs]) float32, the largest magnitude of a step's
    channels / 448 (at least 2^-120), so that out * scale is the norm.  [tokens,
    channels] goes into an 8-bit matrix product as it is; of rows over time, whose
    steps' channels lie T apart, such a product wants a transposed copy."""
    return _norm(x, weight, residual, eps, lengths, total, out, scale, True)


def rms_norm_backward(grad_out, x, weight=None, eps=1e-6, grad_sum=None, lengths=None):
    """Gradients of rms_norm from its output's gradient: x is what was normed (s, or
    x where there was no residual), grad_sum the gradient that reaches s itself
    further on, added to that of the norm.  Returns NormGrads."""
    head, tail, shape, dev, dtype = _norm_inputs(x, weight, eps, lengths)
    if grad_out is None:
        raise ValueError("grad_out is required")
    grads = NormGrads(x=_new(None, shape, dtype, dev),
                      weight=None if weight is None else _new(None, shape[1:2], torch.float32, dev))
    call = _pack_norm(*head, x.data_ptr(), x.stride(0), x.stride(1), 0, 0, 0, *tail, 0, 0, 0, 0,
                      *_rows("grad_out", grad_out, shape, dtype, dev),
                      *_rows("grad_sum", grad_sum, shape, dtype, dev), grads.x.data_ptr(),
                      _ptr(grads.weight))
    ws = _scratch(lib().rlca_rms_norm_backward_workspace_size(call), dev)
    _run("rlca_rms_norm_backward", dev, call, ws.data_ptr(), ws.numel())
    return grads


# ----------------------------------------------------------------- beam search
class BeamChoice(NamedTuple):
    """A selection, best first, [num_searches, picks]: total log probabilities
    (float32), tokens and the beams that they continue (int32)."""

    scores: torch.Tensor
    tokens: torch.Tensor
    parents: torch.Tensor


def beam_select(logits, scores, picks=None, finished=None, pad_token=0):
    """The best continuations of each search, over all its beams and the vocabulary:
    the `picks` (default: one a beam) highest of score + log_softmax(logits), equal
    ones by the lower beam, those of one beam by the higher logit, then the lower token.

    logits [num_searches, beams, vocab] (float32, bfloat16 or float16; contiguous in
    its last dimension), scores [num_searches, beams] float32 the beams' totals so
    far (-infinity for a beam that is not in use).  finished [num_searches, beams]
    marks beams that go on with pad_token alone, at their own score.  Returns
    BeamChoice."""
    shape = logits.shape
    if len(shape) != 3:
        raise ValueError("logits is [num_searches, beams, vocab]")
    if not logits.is_cuda:
        raise ValueError("inputs must be GPU tensors")
    dtype, dev = logits.dtype, logits.device
    if dtype not in REAL_DTYPES:
        raise TypeError(f"logits must be float32, bfloat16 or float16, got {dtype}")
    logits = _view("logits", logits, shape, dtype, dev)
    N, K, V = shape
    if not 1 <= K <= MAX_BEAMS:
        raise ValueError(f"{K} beams, expected 1 to {MAX_BEAMS}")
    P = K if picks is None else int(picks)
    if not 1 <= P <= min(MAX_BEAMS, K * V):
        raise ValueError(f"{P} picks, expected 1 to {min(MAX_BEAMS, K * V)}")
    if scores is None:
        raise ValueError("scores is required")
    head = (N, K, V, P, REAL_DTYPES[dtype], int(pad_token), logits.data_ptr(), logits.stride(0),
            logits.stride(1), _dense_in("scores", scores, (N, K), torch.float32, dev),
            0 if finished is None else _flags_in(finished, (N, K), dev))
    # one allocation: the scores' bits and the whole numbers are of one size
    bits, tokens, parents = torch.empty((3, N, P), dtype=torch.int32, device=dev).unbind()
    choice = BeamChoice(bits.view(torch.float32), tokens, parents)
    call = _pack_beam(*head, bits.data_ptr(), tokens.data_ptr(), parents.data_ptr())
    ws = _scratch(lib().rlca_beam_select_workspace_size(call), dev)
    _run("rlca_beam_select", dev, call, ws.data_ptr(), ws.numel())
    return choice


def beam_reorder(pools, slots, parents, out=None):
    """The beams' states after a selection, in place in every pool: beam k of a search
    goes on from the state of its beam parents[k].

    pools is a list of tensors [places, ...] of any types, dense (as the single-step
    calls keep them); slots [num_searches, beams] int32 each beam's place in them,
    all different (one out of range holds no state); parents [num_searches, beams]
    int32.  A parent's first child keeps its place, the others' states are copied to
    places of beams without children.  Returns the new slots."""
    pools = list(pools)
    if slots is None or slots.dim() != 2:
        raise ValueError("slots is [num_searches, beams]")
    if not slots.is_cuda:
        raise ValueError("inputs must be GPU tensors")
    N, K = slots.shape
    dev = slots.device
    if not 1 <= K <= MAX_BEAMS:
        raise ValueError(f"{K} beams, expected 1 to {MAX_BEAMS}")
    s = _dense_in("slots", slots, (N, K), torch.int32, dev)
    if parents is None:
        raise ValueError("parents is required")
    f = _dense_in("parents", parents, (N, K), torch.int32, dev)
    places = pools[0].shape[0] if pools and pools[0].dim() > 0 else 0
    packed = array("q", [0]) * (2 * len(pools))
    for i, t in enumerate(pools):
        if t.dim() == 0 or t.shape[0] != places:
            raise ValueError(f"pools[{i}] has shape {tuple(t.shape)}, expected {places} places")
        if t.get_device() != dev.index or not t.is_contiguous():
            raise ValueError(f"pools[{i}] must be contiguous and on {dev}")
        packed[2 * i] = t.data_ptr()
        packed[2 * i + 1] = t.numel() * t.element_size() // places if places > 0 else 0
    o = _new(out, (N, K), torch.int32, dev)
    _run("rlca_beam_reorder", dev, packed.buffer_info()[0], len(pools), N, K, places, s, f,
         o.data_ptr())
    _written(pools if out is None else [*pools, out])
    return o
