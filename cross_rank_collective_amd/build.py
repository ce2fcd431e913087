"""Build libptored.so (HIP for gfx950) in-tree.

Every translation unit under csrc/ is compiled with hipcc in parallel and
linked into ``cross_rank_collective_amd/libptored.so``: the host code, one
unit per element type (copy and push-with-add kernels) and ``treduce_op.hip``
once per (element type, operator) pair (reduction and ring kernels); and from
csrc/block/ the block-boundary operators' kernels, once per floating type,
with their host code, and from csrc/step/ the step's.  Next to it, ``_torch_calls.so``: the block-boundary
calls on torch tensors as an extension module (host code, g++).  Run as
``python -m cross_rank_collective_amd.build`` or through
``__graft_entry__.build()``.
"""

from __future__ import annotations

import os
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libptored.so")
EXT = os.path.join(PKG, "_torch_calls.so")
BUILD_DIR = os.path.join(ROOT, "_build")

DTYPES = ("F32", "BF16", "F16", "I32")
OPS = ("SUM", "MAX", "MIN", "PROD")

# (source, object name, extra defines); the slowest units first.
UNITS = [("treduce_op.hip", f"treduce_op_{dt.lower()}_{op.lower()}",
          (f"-DPTORED_INST_DT=PTORED_{dt}", f"-DPTORED_INST_OP=PTORED_{op}"))
         for dt in ("BF16", "F16", "F32", "I32") for op in OPS]
UNITS += [(f"treduce_{dt.lower()}.hip", f"treduce_{dt.lower()}", ()) for dt in DTYPES]
UNITS += [("treduce_host.cpp", "treduce_host", ())]
# The block-boundary operators: one unit per floating type, and their host code.
UNITS += [("block/block_ops.hip", f"block_ops_{dt.lower()}",
           (f"-DPTORED_INST_DT=PTORED_{dt}", f"-DPTORED_INST_NAME={dt.lower()}"))
          for dt in ("BF16", "F16", "F32")]
UNITS += [("block/block_host.cpp", "block_host", ())]
# The step's operators likewise, and the kernels over lists of gradients.
UNITS = [("step/step_ops.hip", f"step_ops_{dt.lower()}",
          (f"-DPTORED_INST_DT=PTORED_{dt}", f"-DPTORED_INST_NAME={dt.lower()}"))
         for dt in ("BF16", "F16", "F32")] + UNITS
UNITS += [("step/step_host.cpp", "step_host", ()), ("step/grad_clip.hip", "grad_clip", ())]

ARCH = "gfx950"
CFLAGS = [
    f"--offload-arch={ARCH}",
    "-O3",
    "-std=c++17",
    "-fPIC",
    "-Wall",
    # Keep the compiler from forming packed-FP32 instructions.
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    f"-I{INCLUDE}",
    f"-I{CSRC}",
]


def hipcc() -> str:
    for cand in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", shutil.which("hipcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found: install ROCm or set HIPCC")


def _compile(unit) -> str:
    src, name, defines = unit
    obj = os.path.join(BUILD_DIR, name + ".o")
    cmd = [hipcc(), *CFLAGS, *defines, "-x", "hip", "-c", os.path.join(CSRC, src), "-o", obj]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"hipcc failed on {name} ({src}):\n{res.stdout}\n{res.stderr}")
    return obj


def _compile_ext() -> str:
    import sysconfig

    import torch
    from torch.utils import cpp_extension

    obj = os.path.join(BUILD_DIR, "torch_calls.o")
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-Wall",
           "-D__HIP_PLATFORM_AMD__=1", "-DUSE_ROCM=1",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           f"-I{INCLUDE}", "-I" + sysconfig.get_paths()["include"],
           *("-isystem" + p for p in cpp_extension.include_paths()), "-isystem/opt/rocm/include",
           "-c", os.path.join(CSRC, "block", "torch_calls.cpp"), "-o", obj]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"g++ failed on torch_calls.cpp:\n{res.stdout}\n{res.stderr}")
    return obj


def _link_ext(obj: str) -> None:
    from torch.utils import cpp_extension

    cmd = [os.environ.get("CXX", "g++"), "-shared", "-fPIC", obj, "-o", EXT + ".tmp", f"-L{PKG}",
           "-l:libptored.so", "-Wl,-rpath,$ORIGIN",
           *("-L" + p for p in cpp_extension.library_paths()), "-ltorch_python", "-ltorch_cpu",
           "-lc10", "-lc10_hip", "-lamdhip64"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"link of _torch_calls.so failed:\n{res.stdout}\n{res.stderr}")
    os.replace(EXT + ".tmp", EXT)


def build(jobs: int = 0) -> str:
    """Compile every HIP unit for gfx950 and link libptored.so and the tensor
    calls; returns the library's path.  Where the tensor calls cannot be built
    (no g++, no torch headers) the library still is, before the error is raised.
    ``jobs`` = parallel compilers (0: one per CPU, at most 16)."""
    os.makedirs(BUILD_DIR, exist_ok=True)
    if jobs <= 0:
        jobs = min(16, len(os.sched_getaffinity(0)))
    with ThreadPoolExecutor(max(1, min(jobs, len(UNITS) + 1))) as ex:
        ext = ex.submit(_compile_ext)
        objs = list(ex.map(_compile, UNITS))
        tmp = LIB + ".tmp"
        cmd = [hipcc(), f"--offload-arch={ARCH}", "-shared", "-fPIC", *objs, "-o", tmp]
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError(f"link failed:\n{res.stdout}\n{res.stderr}")
        os.replace(tmp, LIB)
        # only now: the library needs neither torch's headers nor g++
        _link_ext(ext.result())
    return LIB


if __name__ == "__main__":
    print(build(int(sys.argv[1]) if len(sys.argv) > 1 else 0))
