"""Lane-crossing reads keep their distance: the hardware requires two wait states
between a vector instruction's write of a register and a DPP instruction that reads
it from another lane.  The compiler sees to that for its own instructions, not for
what stands in an asm block, nor between a block's last writes and the instruction
after it.  The blocks' text, and the disassembly of the build's own kernels (CPU)."""
import glob
import os
import re
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "linear_recurrence_scan_row_amd", "csrc")
OBJS = sorted(glob.glob(os.path.join(ROOT, "_build", "librlca", "seq_scan*.hip.o")))
LLVM = "/opt/rocm/llvm/bin"
TOOLS = [os.path.join(LLVM, t) for t in ("llvm-objcopy", "clang-offload-bundler", "llvm-objdump")]
WAIT = 2
DPP = re.compile(r"_dpp\b|\b(row_sh[lr]|row_ror|row_newbcast|row_bcast|quad_perm|wave_sh)")


def registers(operand):
    """The vector registers of an operand, as numbers ('%0' counts as one)."""
    m = re.fullmatch(r"-?\|?v\[(\d+):(\d+)\]\|?", operand)
    if m:
        return range(int(m[1]), int(m[2]) + 1)
    m = re.fullmatch(r"-?\|?(?:v|%)(\d+)\|?", operand)
    return [int(m[1])] if m else []


def check(instructions, last=None):
    """(instruction, register) for every DPP read within WAIT states of the write;
    and the wait states since each register's last write, at the end."""
    bad, since = [], {} if last is None else last
    for text in instructions:
        op, _, rest = text.partition(" ")
        if op == "s_nop":
            step = int(rest, 0) + 1
        else:
            operands = [x.strip() for x in rest.split(",")]
            # the last operand is followed by the modifiers
            operands = [x.split(" ")[0] for x in operands]
            if DPP.search(text) and len(operands) > 1:
                bad += [(text, r) for r in registers(operands[1]) if since.get(r, WAIT) < WAIT]
            step = 1
        since = {r: n + step for r, n in since.items() if n + step < WAIT}
        if op.startswith("v_") and not op.startswith("v_cmp"):
            for r in registers(operands[0]):
                since[r] = 0
    return bad, since


def test_reads_that_come_too_soon():
    """What `check` finds, and what it lets pass."""
    assert check(["v_add_f32 v1, v2, v3", "v_mov_b32_dpp v4, v1 row_shr:1"])[0]
    assert check(["v_add_f32 v1, v2, v3", "s_nop 0", "v_mov_b32_dpp v4, v1 row_shr:1"])[0]
    assert not check(["v_add_f32 v1, v2, v3", "s_nop 1", "v_mov_b32_dpp v4, v1 row_shr:1"])[0]
    assert not check(["v_add_f32 v1, v2, v3", "v_add_f32 v5, v2, v3", "v_add_f32 v6, v2, v3",
                      "v_mov_b32_dpp v4, v1 quad_perm:[1,0,3,2]"])[0]
    assert check(["v_add_f32 %1, %1, %0"])[1] == {1: 0}


def asm_block(name, source):
    """The instructions of the asm block in a function, its step macro expanded."""
    with open(os.path.join(CSRC, source)) as f:
        body = f.read()
    body = body[body.index(f" {name}("):]
    body = body[:body.index("#undef RLCA_STEP")]
    macro = re.search(r"#define RLCA_STEP\(SHIFT\)(.*?)\n(?!.*\\\n)(?=\s+(?:if|asm))", body, re.S)[1]
    text = body[body.rindex("asm("):]
    text = text[:text.index(":\n") if ":\n" in text else re.search(r"\n\s+:", text).start()]
    text = re.sub(r'RLCA_STEP\("([^"]*)"\)', lambda m: macro.replace("SHIFT", f'"{m[1]}"'), text)
    return [i.strip() for i in "".join(re.findall(r'"([^"]*)"', text)).replace("\\t", "").split("\\n")
            if i.strip()]


def test_row_sum_leaves_its_results_readable():
    """The caller reads both sums with a lane-crossing move, maybe at once."""
    instructions = asm_block("row_sum", "seq_scan_backward.hip")
    assert sum(i.startswith("v_add_f32_dpp") for i in instructions) == 8
    bad, since = check(instructions)
    assert not bad
    assert not since, f"wait states since the last write: {since}"


def test_row_scan_within():
    instructions = asm_block("row_scan", "seq_scan.hpp")
    assert sum("_dpp" in i for i in instructions) == 16
    assert not check(instructions)[0]


@pytest.mark.skipif(not OBJS, reason="the library's objects are not built")
@pytest.mark.skipif(not all(os.path.exists(t) for t in TOOLS), reason="ROCm LLVM tools missing")
def test_no_kernel_reads_too_early(tmp_path):
    reads = 0
    for obj in OBJS:
        bundle, code = str(tmp_path / "bundle"), str(tmp_path / "code")
        subprocess.run([TOOLS[0], "--dump-section", f".hip_fatbin={bundle}", obj,
                        str(tmp_path / "host.o")], check=True, capture_output=True)
        subprocess.run([TOOLS[1], "--unbundle", "--type=o",
                        "--targets=hipv4-amdgcn-amd-amdhsa--gfx950", f"--input={bundle}",
                        f"--output={code}"], check=True, capture_output=True)
        out = subprocess.run([TOOLS[2], "-d", "--no-show-raw-insn", "--no-leading-addr", code],
                             check=True, capture_output=True, text=True).stdout
        lines = [line.split("//")[0].strip() for line in out.splitlines()]
        lines = [line for line in lines if line.startswith(("v_", "s_", "ds_", "global_"))]
        reads += sum(bool(DPP.search(line)) for line in lines)
        bad, _ = check(lines)
        assert not bad, (os.path.basename(obj), bad[:5])
    assert reads > 1000
