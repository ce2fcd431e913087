"""What the host code of the block-boundary operators hands to a launch, under
AddressSanitizer and UndefinedBehaviorSanitizer, on the CPU (no GPU, no HIP
runtime): ``tests/sanitize/block_launches.cpp`` makes the calls with made-up
addresses and looks at what ``tests/sanitize/block_stub.cpp`` recorded.
"""

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

pytestmark = pytest.mark.skipif(
    shutil.which("g++") is None or not os.path.isdir(os.path.join(ROCM_INCLUDE, "hip")),
    reason="needs g++ and the HIP headers")


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("block_launches") / "run")
    cmd = ["g++", "-std=c++17", "-Wall", "-Wextra", *SAN, "-D__HIP_PLATFORM_AMD__",
           f"-I{ROCM_INCLUDE}", f"-I{os.path.join(ROOT, 'include')}", f"-I{CSRC}", f"-I{HERE}",
           os.path.join(CSRC, "block", "block_host.cpp"), os.path.join(HERE, "block_stub.cpp"),
           os.path.join(HERE, "block_launches.cpp"), "-o", exe]
    res = subprocess.run(cmd, capture_output=True, text=True)
    assert res.returncode == 0, res.stderr
    return exe


def run(program, name):
    env = {**os.environ, "ASAN_OPTIONS": "detect_leaks=0:halt_on_error=1",
           "UBSAN_OPTIONS": "halt_on_error=1:print_stacktrace=1"}
    res = subprocess.run([program, name], capture_output=True, text=True, timeout=120, env=env)
    assert res.returncode == 0, res.stdout + res.stderr


def test_without_a_gate_its_rows_are_not_read(program):
    run(program, "no_gate")


def test_rows_without_columns(program):
    run(program, "no_columns")


def test_backward_does_not_read_eps(program):
    run(program, "eps_not_read")


def test_row_cuts_of_the_backward_pass(program):
    run(program, "row_cuts")


def test_token_splits_of_the_weight_gradient(program):
    run(program, "token_splits")


def test_a_single_row_has_no_pitch(program):
    run(program, "one_row")
