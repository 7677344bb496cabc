"""The scan's check of its tickets (CPU only: built with a host compiler)."""
import os
import re
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "gated_delta_rule_37_amd", "csrc")


def test_only_tiles_pass(tmp_path):
    """A ticket from a workspace that another call overwrites can be any word:
    only those below the number of tiles may become addresses."""
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no host C++ compiler")
    exe = str(tmp_path / "ticket_driver")
    cmd = [gxx, "-std=c++17", "-O1", "-D__HIP_PLATFORM_AMD__", "-I" + os.path.join(ROOT, "include"), "-I" + CSRC,
           "-I/opt/rocm/include", os.path.join(ROOT, "tests", "sanitize", "ticket_driver.cpp"), "-o", exe]
    res = subprocess.run(cmd, capture_output=True, text=True)
    assert res.returncode == 0, res.stderr[-3000:]
    most = (1 << 30) // 128
    cases = [(t, n) for n in (1, 2, 512, most) for t in (0, 1, n - 1, n, n + 1, 0x7fc00000, 0x7fffffff, 0x80000000,
                                                         0xbf800000, 0xff800000, 0xfffffffe, 0xffffffff)]
    res = subprocess.run([exe], input="".join(f"{t} {n}\n" for t, n in cases), capture_output=True, text=True, timeout=60)
    assert [int(w) for w in res.stdout.split()] == [int(t < n) for t, n in cases]


def test_both_kernels_check_the_ticket():
    """No tile index of the scan comes from anywhere but a checked ticket."""
    with open(os.path.join(CSRC, "kda_scan.hip")) as f:
        source = f.read()
    kernels = re.findall(r"void (scan\w*_kernel)\(ScanParams p\) \{(.*?)\n\}", source, re.S)
    assert {n for n, _ in kernels} == {"scan_kernel", "scan_backward_kernel"}
    for name, body in kernels:
        assert re.search(r"ticket = take_ticket\(.*?\);\n  if \(!is_tile\(ticket, p\.tiles\)\) return;\n"
                         r"  const int32_t tile = static_cast<int32_t>\(ticket\);", body), name
