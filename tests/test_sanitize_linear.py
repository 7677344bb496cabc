"""The host checks of linear attention and of the norms and rotation before it under
AddressSanitizer and UndefinedBehaviorSanitizer (CPU only): kda_layer_validate.cpp,
built with a host compiler and driven by ``tests/sanitize/linear_driver.cpp``.  Every
buffer at exactly its size passes, up to the largest sizes; each one byte short gives
the documented error."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "gated_delta_rule_37_amd", "csrc")
# buffers of each case; the last one a workspace where True
CASES = dict(rotate=(8, False), rotate_one=(8, False), rotate_most=(8, False), rotate_bwd=(13, True), linear=(9, True),
             linear_uncut=(8, False), linear_most=(9, True), linear_bwd=(14, True), linear_bwd_fixed=(14, True),
             step=(8, False), step_fixed=(8, False))


@pytest.fixture(scope="module")
def driver(tmp_path_factory):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no host C++ compiler")
    exe = str(tmp_path_factory.mktemp("sanitize") / "linear_driver")
    sources = [os.path.join(CSRC, n) for n in ("kda_plan.cpp", "kda_validate.cpp", "kda_layer_validate.cpp")]
    cmd = [gxx, "-std=c++17", "-g", "-O1", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
           "-fno-omit-frame-pointer", "-D__HIP_PLATFORM_AMD__", "-I" + os.path.join(ROOT, "include"), "-I" + CSRC,
           "-I/opt/rocm/include", *sources, os.path.join(ROOT, "tests", "sanitize", "linear_driver.cpp"), "-o", exe]
    res = subprocess.run(cmd, capture_output=True, text=True)
    assert res.returncode == 0, res.stderr[-3000:]
    return exe


@pytest.mark.parametrize("case", CASES)
def test_exact_sizes_pass_and_short_ones_do_not(driver, case):
    n, workspace = CASES[case]
    lines = [f"{case} {i}" for i in range(-1, n)]
    res = subprocess.run([driver], input="\n".join(lines) + "\n", capture_output=True, text=True, timeout=60)
    assert res.returncode == 0 and "runtime error" not in res.stderr, res.stderr[-3000:]
    got = [tuple(int(w) for w in line.split()) for line in res.stdout.split("\n") if line]
    assert [g[1] for g in got] == [n] * (n + 1)
    want = [0] + [-9] * n
    if workspace:
        want[-1] = -8
    assert [g[0] for g in got] == want
