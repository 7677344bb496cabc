"""The compiled kernels of the operators around the recurrence (CPU only: hipcc
cross-compiles).  They use no matrix instructions, so the lint of matrix-core
results read across lanes has nothing to check in them, and no packed FP32
arithmetic, which the build turns off; the one-pass kernels keep their tiles in
registers (no spills in the geometries that the launchers choose by size)."""
import os
import re
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)
import __graft_entry__ as ge  # noqa: E402

HIP_SOURCES = [s for s in ge.LAYER_SOURCES if s.endswith(".hip")]


@pytest.mark.skipif(shutil.which(os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")) is None, reason="no hipcc")
@pytest.mark.parametrize("src", HIP_SOURCES)
def test_instructions_and_registers(src, tmp_path):
    hipcc = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
    flags = [f for f in ge.HIPCC_FLAGS if f not in ("-shared", "-fPIC")]
    out = tmp_path / (src + ".s")
    cmd = [hipcc, *flags, "--cuda-device-only", "-S", "-I" + os.path.join(ROOT, "include"), "-I" + ge.CSRC,
           os.path.join(ge.CSRC, src), "-o", str(out)]
    res = subprocess.run(cmd, capture_output=True, text=True)
    assert res.returncode == 0, res.stderr[-2000:]
    asm = out.read_text()
    assert "v_mfma" not in asm
    assert not re.search(r"v_pk_(add|mul|fma)_f32", asm)
    for name, body in re.findall(r"\.amdhsa_kernel (\S+)\n(.*?)\.end_amdhsa_kernel", asm, re.S):
        scratch = int(re.search(r"private_segment_fixed_size (\d+)", body).group(1))
        assert scratch == 0, (name, scratch)


@pytest.mark.skipif(shutil.which(os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")) is None, reason="no hipcc")
@pytest.mark.parametrize("src,kernels", [("kda_prepare.hip", 7), ("kda_step.hip", 5)])
def test_every_kernel_is_seen(src, kernels, tmp_path):
    """The pattern that looks for spills finds the kernels' descriptors, each with
    its scratch size (the two sources that compile fast)."""
    hipcc = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
    flags = [f for f in ge.HIPCC_FLAGS if f not in ("-shared", "-fPIC")]
    out = tmp_path / (src + ".s")
    cmd = [hipcc, *flags, "--cuda-device-only", "-S", "-I" + os.path.join(ROOT, "include"), "-I" + ge.CSRC,
           os.path.join(ge.CSRC, src), "-o", str(out)]
    res = subprocess.run(cmd, capture_output=True, text=True)
    assert res.returncode == 0, res.stderr[-2000:]
    asm = out.read_text()
    found = re.findall(r"\.amdhsa_kernel (\S+)\n(.*?)\.end_amdhsa_kernel", asm, re.S)
    assert len(found) == kernels == len(re.findall(r"^\s*\.amdhsa_kernel\s", asm, re.M))
    assert all(re.search(r"private_segment_fixed_size \d+", body) for _, body in found)
