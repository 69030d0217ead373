"""Host-side checks of the sequence operators' C entry points: every refusal
comes back as a status before anything touches the device, and calls with
nothing to do are no-ops.  Fake addresses, never dereferenced; no GPU."""
import ctypes
import os
import shutil
import subprocess

import pytest

from linear_recurrence_scan_row_amd import rlca as binding
from linear_recurrence_scan_row_amd import sequence as seq

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

OK, NULLP, SIZE, VALUE, ALIAS, MISAL, HIP = range(7)
STEP = 1 << 32  # between fake arrays


@pytest.fixture(scope="module")
def lib():
    return binding.lib()


class Far:
    """A new fake address, far from the others, at each call."""

    def __init__(self):
        self.n = 0

    def __call__(self):
        self.n += 1
        return self.n * STEP


def conv_call(backward=False, **change):
    at = Far()
    c = dict(num_seqs=2, channels=6, T=40, width=4, silu=1, dtype=binding.RLCA_F32, convention=0,
             x=at(), x_stride_seq=240, x_stride_channel=40, weight=at(), bias=at(), state=at(),
             flags=at(), lengths=at())
    if backward:
        c.update(grad_out=at(), grad_stride_seq=240, grad_stride_channel=40,
                 grad_final_state=at(), grad_x=at(), grad_weight=at(), grad_bias=at(),
                 grad_state=at())
    else:
        c.update(out=at(), final_state=at())
    c.update(change)
    return seq.ConvCall(**c)


def scan_call(backward=False, **change):
    at = Far()
    c = dict(num_seqs=2, channels=6, T=40, states=5, groups=2, softplus=1,
             dtype=binding.RLCA_F32, convention=0, u=at(), delta=at(), u_stride_seq=240,
             u_stride_channel=40, delta_stride_seq=240, delta_stride_channel=40, A=at(), B=at(),
             C=at(), B_stride_seq=400, B_stride_group=200, B_stride_state=40, C_stride_seq=400,
             C_stride_group=200, C_stride_state=40, D=at(), delta_bias=at(), z=at(),
             z_stride_seq=240, z_stride_channel=40, state=at(), flags=at(), lengths=at(),
             checkpoints=at())
    if backward:
        c.update(grad_y=at(), grad_stride_seq=240, grad_stride_channel=40, grad_final_state=at(),
                 grad_u=at(), grad_delta=at(), grad_A=at(), grad_B=at(), grad_C=at(), grad_D=at(),
                 grad_delta_bias=at(), grad_z=at(), grad_state=at())
    else:
        c.update(y=at(), final_state=at())
    c.update(change)
    return seq.ScanCall(**c)


def conv_step_call(**change):
    at = Far()
    c = dict(num_seqs=3, channels=6, places=5, width=4, silu=1, dtype=binding.RLCA_F32, x=at(),
             x_stride_seq=6, weight=at(), bias=at(), state=at(), slots=at(), starts=at(),
             out=at())
    c.update(change)
    return seq.ConvStepCall(**c)


def scan_step_call(**change):
    at = Far()
    c = dict(num_seqs=3, channels=6, places=5, states=5, groups=2, softplus=1,
             dtype=binding.RLCA_F32, u=at(), delta=at(), u_stride_seq=6, delta_stride_seq=6,
             A=at(), B=at(), C=at(), B_stride_seq=10, B_stride_group=5, C_stride_seq=10,
             C_stride_group=5, D=at(), delta_bias=at(), z=at(), z_stride_seq=6, state=at(),
             slots=at(), starts=at(), y=at())
    c.update(change)
    return seq.ScanStepCall(**c)


def run(lib, call, workspace=None, nbytes=1 << 30):
    """The status of a call; backward calls (those with gradients) get a workspace."""
    ref = ctypes.byref(call)
    if isinstance(call, seq.ConvCall):
        if call.grad_weight or call.grad_x:
            return lib.rlca_causal_conv_backward(ref, workspace or 99 * STEP, nbytes, None)
        return lib.rlca_causal_conv(ref, None)
    if isinstance(call, seq.ScanCall):
        if call.grad_A or call.grad_u:
            return lib.rlca_selective_scan_backward(ref, workspace or 99 * STEP, nbytes, None)
        return lib.rlca_selective_scan(ref, None)
    if isinstance(call, seq.ConvStepCall):
        return lib.rlca_causal_conv_step(ref, None)
    return lib.rlca_selective_step(ref, None)


ALL = [conv_call, lambda **k: conv_call(True, **k), scan_call, lambda **k: scan_call(True, **k),
       conv_step_call, scan_step_call]
IDS = ["conv", "conv_backward", "scan", "scan_backward", "conv_step", "scan_step"]


@pytest.mark.skipif(shutil.which("gcc") is None, reason="no gcc")
def test_structures_match_the_header(tmp_path):
    """Size and every field's offset, as a C compiler lays the header's out."""
    lines = []
    for cls, name in ((seq.ConvCall, "rlca_conv_call"), (seq.ScanCall, "rlca_scan_call"),
                      (seq.ConvStepCall, "rlca_conv_step_call"),
                      (seq.ScanStepCall, "rlca_scan_step_call"),
                      (seq.GradTensor, "rlca_grad_tensor")):
        lines.append(f"_Static_assert(sizeof({name}) == {ctypes.sizeof(cls)}, \"{name}\");")
        lines += [f"_Static_assert(offsetof({name}, {f}) == {getattr(cls, f).offset}, \"{f}\");"
                  for f, _ in cls._fields_]
    lines.append(f"_Static_assert(RLCA_MAX_STATES == {seq.MAX_STATES}, \"states\");")
    lines.append(f"_Static_assert(RLCA_CLIP_WORKSPACE_BYTES == {seq.CLIP_WORKSPACE_BYTES}, "
                 "\"workspace\");")
    src = tmp_path / "layout.c"
    src.write_text('#include "rlca.h"\n#include <stddef.h>\n' + "\n".join(lines) + "\n")
    r = subprocess.run(["gcc", "-std=c11", "-fsyntax-only", "-D__HIP_PLATFORM_AMD__", "-I",
                        os.path.join(ROOT, "include"), "-I", "/opt/rocm/include", str(src)],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]


def test_null_call(lib):
    assert lib.rlca_causal_conv(None, None) == NULLP
    assert lib.rlca_causal_conv_backward(None, None, 0, None) == NULLP
    assert lib.rlca_selective_scan(None, None) == NULLP
    assert lib.rlca_selective_scan_backward(None, None, 0, None) == NULLP
    assert lib.rlca_causal_conv_step(None, None) == NULLP
    assert lib.rlca_selective_step(None, None) == NULLP
    assert lib.rlca_causal_conv_backward_workspace_size(None) == 0
    assert lib.rlca_selective_scan_checkpoints_size(None) == 0


@pytest.mark.parametrize("make", ALL, ids=IDS)
def test_sizes(lib, make):
    assert run(lib, make(num_seqs=-1)) == SIZE
    assert run(lib, make(channels=-2)) == SIZE
    assert run(lib, make(num_seqs=1 << 31)) == SIZE
    assert run(lib, make(num_seqs=1 << 20, channels=1 << 12)) == SIZE
    if not hasattr(make(), "places"):
        assert run(lib, make(T=-1)) == SIZE
        assert run(lib, make(T=(1 << 30) + 1)) == SIZE
    else:
        assert run(lib, make(places=-1)) == SIZE
        assert run(lib, make(places=2, slots=None)) == SIZE


@pytest.mark.parametrize("make", ALL, ids=IDS)
def test_values(lib, make):
    for dtype in (binding.RLCA_I32, 4, -1):
        assert run(lib, make(dtype=dtype)) == VALUE
    fields = [f for f, _ in type(make())._fields_]
    if "convention" in fields:
        assert run(lib, make(convention=2)) == VALUE
        assert run(lib, make(convention=-1)) == VALUE
    if "width" in fields:
        for width in (-1, 0, 1, 5):
            assert run(lib, make(width=width)) == VALUE
    else:
        for states in (-1, 0, 129):
            assert run(lib, make(states=states)) == VALUE
        for groups in (-1, 0, 4, 12):
            assert run(lib, make(groups=groups)) == VALUE


REQUIRED = {
    "conv": ("x", "weight", "out"),
    "conv_backward": ("x", "weight", "grad_out", "grad_x", "grad_weight"),
    "scan": ("u", "delta", "A", "B", "C", "y"),
    "scan_backward": ("u", "delta", "A", "B", "C", "grad_y", "checkpoints", "grad_u",
                      "grad_delta", "grad_A", "grad_B", "grad_C", "grad_z"),
    "conv_step": ("x", "weight", "state", "out"),
    "scan_step": ("u", "delta", "A", "B", "C", "state", "y"),
}


@pytest.mark.parametrize("make,name", zip(ALL, IDS), ids=IDS)
def test_required_pointers(lib, make, name):
    for field in REQUIRED[name]:
        assert run(lib, make(**{field: None})) == NULLP, field


@pytest.mark.parametrize("make,name", zip(ALL, IDS), ids=IDS)
def test_alignment(lib, make, name):
    for field in REQUIRED[name]:
        assert run(lib, make(**{field: 50 * STEP + 2})) == MISAL, field
    two = make(dtype=binding.RLCA_BF16)
    first = "x" if "conv" in name else "u"
    setattr(two, first, 50 * STEP + 1)
    assert run(lib, two) == MISAL


@pytest.mark.parametrize("make,name", zip(ALL, IDS), ids=IDS)
def test_negative_strides(lib, make, name):
    for field, _ in type(make())._fields_:
        if "stride" in field:
            used = name.endswith("backward") or not field.startswith("grad_")
            if used:
                assert run(lib, make(**{field: -8})) == SIZE, field
                assert run(lib, make(**{field: 1 << 60})) == SIZE, field


@pytest.mark.parametrize("make,name", zip(ALL, IDS), ids=IDS)
def test_aliasing(lib, make, name):
    """Every output against every other array."""
    base = make()
    outs = {"conv": ("out", "final_state"), "scan": ("y", "final_state", "checkpoints"),
            "conv_backward": ("grad_x", "grad_weight", "grad_bias", "grad_state"),
            "scan_backward": ("grad_u", "grad_delta", "grad_A", "grad_B", "grad_C", "grad_D",
                              "grad_delta_bias", "grad_z", "grad_state"),
            "conv_step": ("state", "out"), "scan_step": ("state", "y")}[name]
    pointers = [f for f, t in type(base)._fields_ if t is binding._p and getattr(base, f)]
    if name == "scan_backward":
        pointers.remove("state")  # not an array of the backward call
    for o in outs:
        for f in pointers:
            if f == o:
                continue
            assert run(lib, make(**{o: getattr(base, f)})) == ALIAS, (o, f)
    if name.endswith("backward"):
        for f in pointers:
            assert run(lib, base, workspace=getattr(base, f)) == ALIAS, f


def test_strided_arrays_cover_their_range(lib):
    # the channel range of a wider projection: [2, 12, 40], channels 6..11 read
    # and the outputs right behind the array
    x = 60 * STEP
    call = conv_call(x=x + 6 * 160, x_stride_seq=480, x_stride_channel=40,
                     out=x + 6 * 160 + 4 * (480 + 5 * 40 + 40) - 4)
    assert run(lib, call) == ALIAS
    # a broadcast row (stride 0) is one row
    call = conv_call(x=x, x_stride_seq=0, x_stride_channel=0, out=x + 156)
    assert run(lib, call) == ALIAS


def test_workspace(lib):
    for make in (lambda **k: conv_call(True, **k), lambda **k: scan_call(True, **k)):
        call = make()
        query = lib.rlca_causal_conv_backward_workspace_size if isinstance(call, seq.ConvCall) \
            else lib.rlca_selective_scan_backward_workspace_size
        need = query(ctypes.byref(call))
        assert need > 0
        assert run(lib, call, nbytes=need - 1) == SIZE
        f = lib.rlca_causal_conv_backward if isinstance(call, seq.ConvCall) \
            else lib.rlca_selective_scan_backward
        assert f(ctypes.byref(call), None, need, None) == NULLP
        assert run(lib, call, workspace=99 * STEP + 2) == MISAL
        assert query(ctypes.byref(make(dtype=9))) == 0


def test_nothing_to_do(lib):
    for make in ALL:
        for zero in ("num_seqs", "channels"):
            call = make()
            if getattr(call, "grad_weight", None) or getattr(call, "grad_A", None):
                if zero == "num_seqs":
                    continue  # gradients of an empty sum are written
            setattr(call, zero, 0)
            assert run(lib, call) == OK
            for f, t in type(call)._fields_:  # and no pointer is needed
                if t is binding._p and f not in ("grad_x", "grad_u"):
                    setattr(call, f, None)
            assert run(lib, call) == OK, zero
    assert run(lib, conv_call(T=0, final_state=None)) == OK
    assert run(lib, scan_call(T=0, final_state=None)) == OK


# ---------------------------------------------------------------- the clipping
def clip(lib, tensors, max_norm=1.0, eps=1e-6, norm=90 * STEP, workspace=91 * STEP,
         nbytes=seq.CLIP_WORKSPACE_BYTES, count=None):
    arr = (seq.GradTensor * max(1, len(tensors)))(*[seq.GradTensor(*t) for t in tensors])
    n = len(tensors) if count is None else count
    return lib.rlca_clip_grad_norm(arr, n, max_norm, eps, norm, workspace, nbytes, None)


def test_clip_refusals(lib):
    t = (STEP, STEP, 100, binding.RLCA_F32)
    nan, inf = float("nan"), float("inf")
    assert clip(lib, [t], count=-1) == SIZE
    assert clip(lib, [t], max_norm=-1.0) == VALUE
    assert clip(lib, [t], max_norm=nan) == VALUE
    for eps in (-1.0, nan, inf):
        assert clip(lib, [t], eps=eps) == VALUE
    assert clip(lib, [t], norm=None) == NULLP
    assert clip(lib, [t], workspace=None) == NULLP
    assert clip(lib, [t], norm=90 * STEP + 4) == MISAL
    assert clip(lib, [t], workspace=91 * STEP + 4) == MISAL
    assert clip(lib, [t], nbytes=seq.CLIP_WORKSPACE_BYTES - 1) == SIZE
    assert lib.rlca_clip_grad_norm(None, 1, 1.0, 0.0, 90 * STEP, 91 * STEP, 1 << 20,
                                   None) == NULLP
    assert clip(lib, [(None, STEP, 4, 0)]) == NULLP
    assert clip(lib, [(STEP, None, 4, 0)]) == NULLP
    assert clip(lib, [(STEP, STEP, -4, 0)]) == SIZE
    assert clip(lib, [(STEP, STEP, 1 << 50, 0)]) == SIZE
    assert clip(lib, [(STEP, STEP, 4, 1)]) == VALUE
    assert clip(lib, [(STEP + 2, STEP, 4, 0)]) == MISAL
    assert clip(lib, [(STEP, STEP + 1, 4, 2)]) == MISAL


def test_clip_aliasing(lib):
    f32 = binding.RLCA_F32
    a, b = STEP, 2 * STEP
    assert clip(lib, [(a, a, 100, f32), (a, a, 100, f32)]) == ALIAS       # scaled twice
    assert clip(lib, [(a, a, 100, f32), (a + 396, a + 396, 5, f32)]) == ALIAS
    assert clip(lib, [(a, b, 100, f32), (b + 396, b + 396, 5, f32)]) == ALIAS
    assert clip(lib, [(a, a + 4, 100, f32)]) == ALIAS                      # shifted over itself
    assert clip(lib, [(a, b, 100, f32)], norm=b) == ALIAS
    assert clip(lib, [(a, a, 100, f32)], workspace=a + 8) == ALIAS
    assert clip(lib, [(a, a, 100, f32)], norm=91 * STEP + 8) == ALIAS
    # many tensors take the same check
    many = [(a + 400 * i, a + 400 * i, 100, f32) for i in range(700)]
    many[3] = (many[600][0] + 8, many[600][0] + 8, 10, f32)
    assert clip(lib, many) == ALIAS


def test_launches_of_too_many_threads(lib):
    for backward in (False, True):
        assert run(lib, scan_call(backward, num_seqs=1 << 24, channels=4, groups=1)) == SIZE
    # forward, 2^8 lanes share a long row
    assert run(lib, conv_call(num_seqs=1, channels=1 << 24, T=4096, x_stride_channel=0,
                              out=1 << 45)) == SIZE
    assert run(lib, scan_step_call(num_seqs=1, channels=1 << 25, groups=1, states=128)) == SIZE
