"""Properties of the layer operators' gfx950 code, checked on the generated assembly (no GPU): every kernel
keeps its values in registers (no spills), and none uses packed fp32 arithmetic."""
import re
import subprocess

import pytest

from chunked_gated_delta_09_amd import build as kbuild
from tests.test_device_code import kernel_meta

SOURCES = [s for s in kbuild.LAYER_SOURCES if s.endswith(".hip")]


@pytest.mark.parametrize("src", SOURCES)
def test_no_spills_and_no_packed_fp32(tmp_path, src):
    out = tmp_path / "k.s"
    cmd = [kbuild._hipcc()] + kbuild.HIP_FLAGS + ["-S", "--cuda-device-only", f"{kbuild.CSRC}/{src}", "-o", str(out)]
    res = subprocess.run(cmd, capture_output=True, text=True)
    assert res.returncode == 0, res.stderr
    asm = out.read_text()
    meta = kernel_meta(asm)
    assert meta
    assert {k: s for k, (_, s) in meta.items() if s} == {}
    assert not re.search(r"\bv_pk_(add|mul|fma)_f32\b", asm)
