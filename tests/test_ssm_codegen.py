"""Checks of the gfx950 code the state space layer's kernels compile to (CPU
only: hipcc cross-compiles): no instruction reads a register that the register
allocator left undefined, no kernel uses scratch memory but the one that is
faster so, and none has packed FP32 instructions."""
import os
import re
import subprocess

import pytest

from varlen_depthwise_causal_amd import _build

FILES = ("vdc_conv_state.hip", "vdc_scan.hip", "vdc_norm.hip")


def _compile(name, out, extra):
    try:
        hipcc = _build.hipcc()
    except RuntimeError:
        pytest.skip("hipcc not available")
    cmd = [hipcc, *_build.COMMON, *_build.DEVICE_FLAGS, "--cuda-device-only", "-S", "-o", str(out),
           os.path.join(_build.CSRC, name), *extra]
    res = subprocess.run(cmd, capture_output=True, text=True)
    assert res.returncode == 0, res.stderr[-4000:]
    return res.stderr


@pytest.mark.parametrize("name", FILES)
def test_scratch_and_instructions(name, tmp_path):
    asm = tmp_path / "out.s"
    out = _compile(name, asm, ["-Rpass-analysis=kernel-resource-usage"])
    names = re.findall(r"Function Name: (\S+)", out)
    scratch = [int(v) for v in re.findall(r"ScratchSize \[bytes/lane\]: (\d+)", out)]
    assert names and len(names) == len(scratch)
    # The norm's backward of groups of more than 8192 channels keeps a group in
    # registers at the price of some of them.
    limit = {n: 320 if re.search(r"norm_bwd_kernelILi512E", n) else 0 for n in names}
    spilled = [(n, s) for n, s in zip(names, scratch) if s > limit[n]]
    assert not spilled, spilled
    assert not re.search(r"\bv_pk_(add|mul|fma)_f32\b", asm.read_text())


@pytest.mark.parametrize("name", FILES)
def test_no_read_of_undefined_registers(name):
    bad, where = [], None
    for line in _compile(name, os.devnull, ["-mllvm", "-print-after=postmisched"]).splitlines():
        m = re.match(r"# Machine code for function (\S+):", line)
        if m:
            where = m.group(1)
        if "IMPLICIT_DEF" in line or " KILL" in line:
            continue
        # A uniform value that one of two joining paths does not have (and whose
        # users all lie behind the other): the arm without it.
        if "V_READFIRSTLANE_B32 undef" in line:
            continue
        # the tied operand of a move across lanes that writes every lane
        line = re.sub(r"(_dpp) undef \$vgpr\d+\(tied-def 0\)", r"\1", line)
        if re.search(r"undef \$[va]gpr", line.split("=", 1)[1] if "=" in line else line):
            bad.append("%s: %s" % (where, line.strip()[:160]))
    assert where and not bad, "\n".join(bad[:20])
