"""Which buffers of a call count as overlapping, on the CPU: every pair of small
matrices byte by byte, and calls on the halves of one buffer
(``tests/sanitize/extents.cpp``)."""

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "cross_rank_collective_amd", "csrc")
HERE = os.path.join(ROOT, "tests", "sanitize")
ROCM_INCLUDE = "/opt/rocm/include"
SAN = ["-g", "-O1", "-fno-omit-frame-pointer", "-fsanitize=address,undefined",
       "-fno-sanitize-recover=all"]


@pytest.mark.skipif(shutil.which("g++") is None or not os.path.isdir(os.path.join(ROCM_INCLUDE, "hip")),
                    reason="needs g++ and the HIP headers")
def test_extents(tmp_path):
    exe = str(tmp_path / "run")
    cmd = ["g++", "-std=c++17", "-Wall", "-Wextra", *SAN, "-D__HIP_PLATFORM_AMD__",
           f"-I{ROCM_INCLUDE}", f"-I{os.path.join(ROOT, 'include')}", f"-I{CSRC}", f"-I{HERE}",
           os.path.join(CSRC, "step", "step_host.cpp"), os.path.join(HERE, "step_stub.cpp"),
           os.path.join(HERE, "extents.cpp"), "-o", exe]
    res = subprocess.run(cmd, capture_output=True, text=True)
    assert res.returncode == 0, res.stderr
    env = {**os.environ, "ASAN_OPTIONS": "detect_leaks=0:halt_on_error=1",
           "UBSAN_OPTIONS": "halt_on_error=1:print_stacktrace=1"}
    res = subprocess.run([exe], capture_output=True, text=True, timeout=120, env=env)
    assert res.returncode == 0, res.stdout + res.stderr
