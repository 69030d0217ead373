"""The gated recurrence's lane-crossing asm blocks keep their distance between a write
and the read of it from another lane, by their text and in the build's own kernels, as
test_lane_hazards.py checks it for the selective scan (CPU)."""
import os
import re
import subprocess

import pytest

from .test_lane_hazards import CSRC, DPP, ROOT, TOOLS, check

OBJ = os.path.join(ROOT, "_build", "librlca", "seq_gated.hip.o")


def test_blocks():
    """Every block: a wait, steps, each ending with its results readable."""
    with open(os.path.join(CSRC, "seq_gated.hip")) as f:
        text = f.read()
    macro = re.search(r"#define RLCA_GATE_STEP\(MOVE, ROWS\)(.*?)\n\n", text, re.S)[1]
    blocks = re.findall(r"asm\(((?:\"|RLCA_GATE_STEP).*?)\n\s*:", text, re.S)
    assert len(blocks) == 3
    for block in blocks:
        block = re.sub(r'RLCA_GATE_STEP\("([^"]*)", "([^"]*)"\)',
                       lambda m: macro.replace("MOVE", f'"{m[1]}"').replace("ROWS", f'"{m[2]}"'),
                       block)
        lines = "".join(re.findall(r'"([^"]*)"', block)).replace("\\t", "").split("\\n")
        lines = [line.strip() for line in lines if line.strip()]
        assert lines[0] == "s_nop 1" and sum("_dpp" in line for line in lines) in (4, 8)
        bad, since = check(lines)
        assert not bad and not since


@pytest.mark.skipif(not os.path.exists(OBJ), reason="the library's objects are not built")
@pytest.mark.skipif(not all(os.path.exists(t) for t in TOOLS), reason="ROCm LLVM tools missing")
def test_kernels(tmp_path):
    bundle, code = str(tmp_path / "bundle"), str(tmp_path / "code")
    subprocess.run([TOOLS[0], "--dump-section", f".hip_fatbin={bundle}", OBJ,
                    str(tmp_path / "host.o")], check=True, capture_output=True)
    subprocess.run([TOOLS[1], "--unbundle", "--type=o",
                    "--targets=hipv4-amdgcn-amd-amdhsa--gfx950", f"--input={bundle}",
                    f"--output={code}"], check=True, capture_output=True)
    out = subprocess.run([TOOLS[2], "-d", "--no-show-raw-insn", "--no-leading-addr", code],
                         check=True, capture_output=True, text=True).stdout
    lines = [line.split("//")[0].strip() for line in out.splitlines()]
    lines = [line for line in lines if line.startswith(("v_", "s_", "ds_", "global_"))]
    assert sum(bool(DPP.search(line)) for line in lines) > 500
    assert not check(lines)[0]
