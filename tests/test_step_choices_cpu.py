"""The kernels of the feed-forward block that the host code takes, on the CPU:
every compiled one is reached by some call, and by one that the GPU tests make
(``tests/sanitize/step_choices.cpp``)."""

import os
import re
import shutil
import subprocess

import pytest

from tests.step_sizes import CASES

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PKG = os.path.join(ROOT, "cross_rank_collective_amd")
CSRC = os.path.join(PKG, "csrc")
HERE = os.path.join(ROOT, "tests", "sanitize")
LIB = os.path.join(PKG, "libptored.so")
ROCM_INCLUDE = "/opt/rocm/include"

pytestmark = pytest.mark.skipif(
    shutil.which("g++") is None or not os.path.isdir(os.path.join(ROCM_INCLUDE, "hip")),
    reason="needs g++ and the HIP headers")


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("step_choices") / "run")
    cmd = ["g++", "-std=c++17", "-O2", "-Wall", "-Wextra", "-D__HIP_PLATFORM_AMD__", f"-I{ROCM_INCLUDE}",
           f"-I{os.path.join(ROOT, 'include')}", f"-I{CSRC}", f"-I{HERE}",
           os.path.join(CSRC, "step", "step_host.cpp"), os.path.join(HERE, "step_stub.cpp"),
           os.path.join(HERE, "step_choices.cpp"), "-o", exe]
    res = subprocess.run(cmd, capture_output=True, text=True)
    assert res.returncode == 0, res.stderr
    return exe


@pytest.fixture(scope="module")
def reached(program):
    """{kernel: a case that takes it} over drawn calls."""
    res = subprocess.run([program, "all", "1000000"], capture_output=True, text=True, timeout=120, check=True)
    return dict(line.split(" | ") for line in res.stdout.splitlines())


@pytest.mark.skipif(shutil.which("nm") is None or not os.path.exists(LIB), reason="needs nm and the library")
def test_every_kernel_that_is_built_is_reached(reached):
    symbols = subprocess.run(["nm", "-C", "--defined-only", LIB], capture_output=True, text=True, check=True).stdout
    built = set(re.findall(r"\b((?:few|product(?:_both)?(?:_join)?)_kernel<[^>]*>)\(", symbols))
    assert len(built) > 50
    assert built == set(reached)


def test_gpu_tests_take_every_kernel(program, reached):
    lines = [f"{dtype} {t} {d} {f} {pad} {call}\n" for bits, t, d, f, pad, call in CASES
             for dtype in ((0,) if bits == 32 else (1, 2))]
    res = subprocess.run([program, "cases"], input="".join(lines), capture_output=True, text=True, check=True)
    taken = [set(line.split("; ")) for line in res.stdout.splitlines()]
    assert len(taken) == len(lines) and all(all(k) for k in taken)
    missing = {k: c for k, c in reached.items() if not any(k in t for t in taken)}
    assert not missing, missing
