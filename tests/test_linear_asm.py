"""The kernels of linear attention as the library builds them (CPU only: hipcc
cross-compiles): the lint of matrix-core results read across lanes under their own
flags, no packed FP32 arithmetic, and the registers that the choice of these flags
and of the chunk's tiles rests on."""
import os
import re
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)
import __graft_entry__ as ge  # noqa: E402
from test_asm_hazards import hazards  # noqa: E402

SOURCES = sorted(ge.DEFAULT_SCHEDULER)


@pytest.mark.skipif(shutil.which(os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")) is None, reason="no hipcc")
@pytest.mark.parametrize("src", SOURCES)
def test_instructions_and_registers(src, tmp_path):
    hipcc = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
    flags = [f for f in ge.flags_of(src) if f not in ("-shared", "-fPIC")]
    assert "-packed-fp32-ops" in flags
    out = tmp_path / (src + ".s")
    cmd = [hipcc, *flags, "--cuda-device-only", "-S", "-I" + os.path.join(ROOT, "include"), "-I" + ge.CSRC,
           os.path.join(ge.CSRC, src), "-o", str(out)]
    res = subprocess.run(cmd, capture_output=True, text=True)
    assert res.returncode == 0, res.stderr[-2000:]
    asm = out.read_text()
    assert "v_mfma" in asm and not re.search(r"v_pk_(add|mul|fma)_f32", asm)
    found = hazards(asm)
    assert not found, found[:10]
    kernels = re.findall(r"\.amdhsa_kernel (\S+)\n(.*?)\.end_amdhsa_kernel", asm, re.S)
    assert len(kernels) >= 4
    for name, body in kernels:
        value = lambda key: int(re.search(key + r" (\d+)", body).group(1))  # noqa: E731
        # two workgroups a CU, but for FP32 outputs of the widest heads, one
        if not re.search(r"(output|grad)_kernelILi128ELi128ELi3E", name):
            assert value("amdhsa_group_segment_fixed_size") <= 80 * 1024, name
            assert value("amdhsa_next_free_vgpr") <= 256, name
        # the widest gradients keep four registers in scratch
        wide = "grad_kernelILi128ELi128ELi2E" in name
        assert value("private_segment_fixed_size") <= (16 if wide else 0), name
