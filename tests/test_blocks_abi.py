"""Host-side checks of the block and beam operators' C entry points: every refusal
comes back as a status before anything touches the device, and calls with nothing
to do are no-ops.  Fake addresses, never dereferenced; no GPU."""
import ctypes
import os
import shutil
import subprocess

import pytest
import torch

import linear_recurrence_scan_row_amd as rl
from linear_recurrence_scan_row_amd import blocks
from linear_recurrence_scan_row_amd import rlca as binding
from .test_sequence_abi import ALIAS, MISAL, NULLP, OK, ROOT, SIZE, STEP, VALUE, Far


@pytest.fixture(scope="module")
def lib():
    return binding.lib()


def gated_call(backward=False, **change):
    at = Far()
    c = dict(num_seqs=2, channels=6, T=40, dtype=binding.RLCA_F32, convention=0, scale=8.0, x=at(),
             input_gate=at(), decay_gate=at(), x_stride_seq=240, x_stride_channel=40,
             input_stride_seq=240, input_stride_channel=40, decay_stride_seq=240,
             decay_stride_channel=40, decay=at(), input_bias=at(), decay_bias=at(), state=at(),
             flags=at(), lengths=at(), checkpoints=at())
    if backward:
        c.update(grad_out=at(), grad_stride_seq=240, grad_stride_channel=40,
                 grad_final_state=at(), grad_x=at(), grad_input_gate=at(), grad_decay_gate=at(),
                 grad_decay=at(), grad_input_bias=at(), grad_decay_bias=at(), grad_state=at())
    else:
        c.update(out=at(), final_state=at())
    c.update(change)
    return blocks.GatedCall(**c)


def step_call(**change):
    at = Far()
    c = dict(num_seqs=3, channels=6, places=5, dtype=binding.RLCA_F32, scale=8.0, x=at(),
             input_gate=at(), decay_gate=at(), x_stride_seq=6, input_stride_seq=6,
             decay_stride_seq=6, decay=at(), input_bias=at(), decay_bias=at(), state=at(),
             slots=at(), starts=at(), out=at())
    c.update(change)
    return blocks.GatedStepCall(**c)


def norm_call(backward=False, **change):
    at = Far()
    c = dict(num_seqs=2, channels=6, T=40, dtype=binding.RLCA_F32, eps=1e-6, x=at(),
             x_stride_seq=240, x_stride_channel=40, weight=at(), lengths=at())
    if backward:
        c.update(grad_out=at(), grad_stride_seq=240, grad_stride_channel=40, grad_sum=at(),
                 grad_sum_stride_seq=240, grad_sum_stride_channel=40, grad_x=at(),
                 grad_weight=at())
    else:
        c.update(residual=at(), residual_stride_seq=240, residual_stride_channel=40, out=at(),
                 sum=at())
    c.update(change)
    return blocks.NormCall(**c)


def beam_call(**change):
    at = Far()
    c = dict(num_searches=2, beams=3, vocab=50, picks=4, dtype=binding.RLCA_F32, pad_token=7,
             logits=at(), logits_stride_search=150, logits_stride_beam=50, scores=at(),
             finished=at(), out_scores=at(), out_tokens=at(), out_parents=at())
    c.update(change)
    return blocks.BeamCall(**c)


def run(lib, call, workspace=None, nbytes=1 << 30):
    ref, ws = ctypes.byref(call), workspace or 99 * STEP
    if isinstance(call, blocks.GatedCall):
        f = lib.rlca_gated_recurrence_backward if call.grad_decay or call.grad_x \
            else lib.rlca_gated_recurrence
        return f(ref, ws, nbytes, None)
    if isinstance(call, blocks.NormCall):
        if call.grad_out or call.grad_x:
            return lib.rlca_rms_norm_backward(ref, ws, nbytes, None)
        return lib.rlca_rms_norm(ref, None)
    if isinstance(call, blocks.BeamCall):
        return lib.rlca_beam_select(ref, ws, nbytes, None)
    return lib.rlca_gated_step(ref, None)


def back(make):
    return lambda **k: make(True, **k)


ROWS = [gated_call, back(gated_call), norm_call, back(norm_call)]
ROWS_IDS = ["gated", "gated_backward", "norm", "norm_backward"]


@pytest.mark.skipif(shutil.which("gcc") is None, reason="no gcc")
def test_structures_match_the_header(tmp_path):
    """Size and every field's offset, as a C compiler lays the header's out."""
    lines = []
    for cls, name in ((blocks.GatedCall, "rlca_gated_call"),
                      (blocks.GatedStepCall, "rlca_gated_step_call"),
                      (blocks.NormCall, "rlca_norm_call"), (blocks.BeamCall, "rlca_beam_call"),
                      (blocks.StatePool, "rlca_state_pool")):
        lines.append(f"_Static_assert(sizeof({name}) == {ctypes.sizeof(cls)}, \"{name}\");")
        lines += [f"_Static_assert(offsetof({name}, {f}) == {getattr(cls, f).offset}, \"{f}\");"
                  for f, _ in cls._fields_]
    lines.append(f"_Static_assert(RLCA_MAX_BEAMS == {blocks.MAX_BEAMS}, \"beams\");")
    src = tmp_path / "layout.c"
    src.write_text("#include <stddef.h>\n#include \"rlca.h\"\n" + "\n".join(lines) + "\n")
    subprocess.run(["gcc", "-std=c11", "-fsyntax-only", "-D__HIP_PLATFORM_AMD__",
                    "-I/opt/rocm/include", f"-I{os.path.join(ROOT, 'include')}", str(src)],
                   check=True)


def test_packed_records_are_the_structures():
    for pack, cls in ((blocks._pack_gated, blocks.GatedCall),
                      (blocks._pack_gated_step, blocks.GatedStepCall),
                      (blocks._pack_norm, blocks.NormCall), (blocks._pack_beam, blocks.BeamCall)):
        values = list(range(1, len(cls._fields_) + 1))
        record = cls.from_buffer_copy(pack(*values).ljust(ctypes.sizeof(cls), b"\0"))
        assert [getattr(record, f) for f, _ in cls._fields_] == values


@pytest.mark.parametrize("make", ROWS, ids=ROWS_IDS)
def test_sizes_of_rows(lib, make):
    for bad in (dict(num_seqs=-1), dict(channels=-1), dict(T=-1), dict(T=(1 << 30) + 1),
                dict(num_seqs=1 << 20, channels=1 << 11), dict(x_stride_seq=-240),
                dict(x_stride_channel=1 << 61)):
        assert run(lib, make(**bad)) == SIZE, bad
    # nothing to do
    assert run(lib, make(num_seqs=0, channels=0)) == OK


@pytest.mark.parametrize("make", ROWS + [step_call], ids=ROWS_IDS + ["step"])
def test_values(lib, make):
    assert run(lib, make(dtype=7)) == VALUE
    name = "eps" if make(num_seqs=1).__class__ is blocks.NormCall else "scale"
    for bad in (0.0, -1.0, 1e-31, 1e31, float("nan"), float("inf")):
        assert run(lib, make(**{name: bad})) == VALUE, bad
    if hasattr(make(num_seqs=1), "convention"):
        assert run(lib, make(convention=2)) == VALUE


@pytest.mark.parametrize("make", ROWS + [step_call, beam_call], ids=ROWS_IDS + ["step", "beam"])
def test_null_misaligned_and_overlapping_arrays(lib, make):
    call = make(num_seqs=2) if make is not beam_call else make()
    optional = {"input_bias", "decay_bias", "state", "flags", "lengths", "final_state",
                "grad_final_state", "grad_input_bias", "grad_decay_bias", "grad_state", "weight",
                "grad_sum", "grad_weight", "slots", "starts", "residual", "finished"}
    if isinstance(call, blocks.GatedStepCall):
        optional -= {"state"}
    forward_gated = isinstance(call, blocks.GatedCall) and not call.grad_x
    if forward_gated:
        optional |= {"checkpoints"}
    arrays = [f for f, kind in call._fields_ if kind is ctypes.c_void_p and getattr(call, f)]
    written = [f for f in arrays if f.startswith("grad_") and f not in
               ("grad_out", "grad_sum", "grad_final_state") or f.startswith("out")
               or f in ("final_state", "sum") or (f == "state" and step_call is make)
               or (f == "checkpoints" and forward_gated)]
    for f in arrays:
        change = {f: None}
        if f == "residual":
            continue  # with a sum and no residual nothing is wrong: the sum is not used
        if f not in optional:
            assert run(lib, make(**change)) == NULLP, f
        if f not in ("flags", "starts", "finished"):
            assert run(lib, make(**{f: getattr(call, f) + 1})) == MISAL, f
    for w in written:
        for f in arrays:
            if f != w:
                assert run(lib, make(**{w: getattr(call, f)})) == ALIAS, (w, f)
    if make not in (step_call, norm_call):
        if make is not gated_call:
            for w in written:
                assert run(lib, make(), workspace=getattr(call, w)) == ALIAS, w
            assert run(lib, make(), nbytes=0) == SIZE


def test_workspace_of_a_long_row(lib):
    c = gated_call(num_seqs=1, channels=2, T=1 << 20, x_stride_seq=0, x_stride_channel=0)
    assert lib.rlca_gated_recurrence_workspace_size(ctypes.byref(c)) > 0
    assert run(lib, c, nbytes=8) == SIZE
    short = gated_call()
    assert lib.rlca_gated_recurrence_workspace_size(ctypes.byref(short)) == 0
    assert lib.rlca_gated_recurrence_checkpoints_size(ctypes.byref(short)) == 2 * 6 * 4
    for query in ("rlca_gated_recurrence_workspace_size", "rlca_gated_recurrence_checkpoints_size",
                  "rlca_gated_recurrence_backward_workspace_size"):
        assert getattr(lib, query)(None) == 0
        assert getattr(lib, query)(ctypes.byref(gated_call(T=-1))) == 0


def test_norm_outputs(lib):
    """One of the two outputs, and a scale with the 8-bit one."""
    assert run(lib, norm_call(out=None)) == NULLP
    assert run(lib, norm_call(out8=50 * STEP, scale=51 * STEP)) == VALUE
    assert run(lib, norm_call(out=None, out8=50 * STEP)) == NULLP
    assert run(lib, norm_call(sum=None)) == NULLP
    assert lib.rlca_rms_norm_backward_workspace_size(None) == 0


def test_step_sizes(lib):
    for bad in (dict(places=-1), dict(places=1 << 31), dict(places=2, slots=None),
                dict(num_seqs=-1), dict(channels=1 << 31), dict(x_stride_seq=-1)):
        assert run(lib, step_call(**bad)) == SIZE, bad
    assert run(lib, step_call(num_seqs=0)) == OK
    assert run(lib, step_call(channels=0)) == OK


def test_beam_sizes(lib):
    for bad in (dict(num_searches=-1), dict(num_searches=1 << 24), dict(beams=0), dict(beams=65),
                dict(vocab=0), dict(vocab=1 << 30), dict(picks=0), dict(picks=65),
                dict(beams=1, vocab=3), dict(logits_stride_beam=-1)):
        assert run(lib, beam_call(**bad)) == SIZE, bad
        assert bad.get("logits_stride_beam") or \
            lib.rlca_beam_select_workspace_size(ctypes.byref(beam_call(**bad))) == 0
    for bad in (dict(dtype=9), dict(pad_token=-1), dict(pad_token=50)):
        assert run(lib, beam_call(**bad)) == VALUE, bad
    assert run(lib, beam_call(num_searches=0)) == OK
    assert run(lib, beam_call(num_searches=0, pad_token=99, finished=None)) == OK


def test_reorder_checks(lib):
    def call(pools, n=2, beams=3, places=9, slots=STEP, parents=2 * STEP, new=3 * STEP, count=None):
        packed = (blocks.StatePool * max(1, len(pools)))(*pools)
        return lib.rlca_beam_reorder(ctypes.addressof(packed), len(pools) if count is None else count,
                                     n, beams, places, slots, parents, new, None)

    pool = (10 * STEP, 64)
    for bad in (dict(n=-1), dict(beams=0), dict(beams=65), dict(places=-1), dict(places=1 << 31),
                dict(count=-1)):
        assert call([pool], **bad) == SIZE, bad
    assert call([(10 * STEP, -1)]) == SIZE
    for bad in (dict(slots=None), dict(parents=None), dict(new=None)):
        assert call([pool], **bad) == NULLP, bad
    assert call([(None, 64)]) == NULLP
    assert lib.rlca_beam_reorder(None, 1, 2, 3, 9, STEP, 2 * STEP, 3 * STEP, None) == NULLP
    assert call([pool], slots=STEP + 2) == MISAL
    assert call([pool], new=STEP) == ALIAS
    for other in ("slots", "parents", "new"):
        assert call([pool], **{other: 10 * STEP + 9 * 64 - 4}) == ALIAS
    assert call([pool, (10 * STEP + 9 * 64 - 1, 8)]) == ALIAS
    assert call([pool], n=0) == OK
    assert call([], n=0, count=0) == OK


def test_the_binding_refuses(lib):
    """What the Python functions refuse by themselves, on the CPU."""
    x = torch.zeros(2, 3, 8)
    with pytest.raises(ValueError, match="GPU"):
        rl.gated_recurrence(x, x, x, torch.zeros(3))
    with pytest.raises(ValueError, match="num_seqs"):
        rl.gated_step(x, x, x, torch.zeros(3), torch.zeros(2, 3))
    for f in (rl.rms_norm, rl.rms_norm_8bit):
        with pytest.raises(ValueError, match="GPU"):
            f(x)
        with pytest.raises(ValueError, match="num_seqs"):
            f(torch.zeros(3))
    with pytest.raises(ValueError, match="GPU"):
        rl.rms_norm_backward(x, x)
    with pytest.raises(ValueError, match="GPU"):
        rl.beam_select(x, torch.zeros(2, 3))
    with pytest.raises(ValueError, match="num_searches"):
        rl.beam_select(x[0], torch.zeros(2, 3))
    with pytest.raises(ValueError, match="num_searches"):
        rl.beam_reorder([x], None, None)
    with pytest.raises(ValueError, match="GPU"):
        rl.beam_reorder([x], torch.zeros(1, 2, dtype=torch.int32), None)
