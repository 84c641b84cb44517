"""Build librsq.so (the HIP kernels and the C ABI of include/rsq.h) for gfx950,
and _binding.so (host code: torch tensors as arguments of the layer operators).

Run as `python bit_recurrent_state_rsq_amd/build.py` (a plain script: it does
not import the package, which would load the library it is about to rebuild).
Compiles every source in csrc/ with hipcc into the package directory. The
library is always rebuilt.
"""
import os
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
OUT = os.path.join(PKG, "librsq.so")
OBJ = os.path.join(PKG, "_build")

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
ARCH = os.environ.get("RSQ_OFFLOAD_ARCH", "gfx950")

FLAGS = [
    "--offload-arch=" + ARCH,
    "-O3",
    "-std=c++17",
    "-fPIC",
    # one rounding per written operation: no fused multiply-adds the source does not ask for
    "-ffp-contract=off",
    "-fhip-fp32-correctly-rounded-divide-sqrt",
    "-fno-gpu-flush-denormals-to-zero",
    # packed fp32 instructions stay off
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-I" + os.path.join(ROOT, "include"),
    "-I" + CSRC,
    "-Wno-unused-result",
]

# Matrix products keep their results in vector registers here. With results in
# accumulation registers (which the compiler picks for kernels of low occupancy)
# it was seen to read them too early behind a branch.
VGPR_RESULTS = ["-mllvm", "-amdgpu-mfma-vgpr-form"]
SOURCE_FLAGS = {"scan.hip": VGPR_RESULTS, "w4.hip": VGPR_RESULTS}


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".hip"))


def _compile(src):
    obj = os.path.join(OBJ, os.path.basename(src) + ".o")
    cmd = [HIPCC] + FLAGS + SOURCE_FLAGS.get(os.path.basename(src), []) + ["-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    errs = "\n".join(l for l in (r.stdout + r.stderr).splitlines()
                     if "packed-fp32-ops" not in l)
    if r.returncode != 0:
        raise RuntimeError("hipcc failed for %s:\n%s" % (src, errs))
    return obj


def _binding():
    """_binding.so: a Python extension against torch's C++ headers, without device code."""
    import importlib.util
    import sysconfig
    torch = os.path.dirname(importlib.util.find_spec("torch").origin)
    out = os.path.join(PKG, "_binding.so")
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden", "-w",
           "-D_GLIBCXX_USE_CXX11_ABI=%d" % _torch_abi(),
           "-I" + os.path.join(ROOT, "include"), "-I" + os.path.join(torch, "include"),
           "-I" + os.path.join(torch, "include", "torch", "csrc", "api", "include"),
           "-I" + sysconfig.get_paths()["include"], os.path.join(CSRC, "binding.cpp"), "-o", out + ".tmp",
           "-L" + os.path.join(torch, "lib"), "-ltorch", "-ltorch_cpu", "-ltorch_python", "-lc10"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("binding.cpp failed:\n" + r.stdout + r.stderr)
    os.replace(out + ".tmp", out)


def _torch_abi():
    """Which std::string the installed torch was built with."""
    import torch
    return int(torch._C._GLIBCXX_USE_CXX11_ABI)


def build(verbose=True):
    os.makedirs(OBJ, exist_ok=True)
    srcs = sources()
    with ThreadPoolExecutor(max_workers=min(8, len(srcs) + 1)) as ex:
        binding = ex.submit(_binding)
        objs = list(ex.map(_compile, srcs))
        binding.result()
    tmp = OUT + ".tmp"
    cmd = [HIPCC, "--offload-arch=" + ARCH, "-shared", "-fPIC", "-o", tmp] + objs
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n" + r.stdout + r.stderr)
    os.replace(tmp, OUT)
    if verbose:
        print("built", OUT)
    return OUT


if __name__ == "__main__":
    build()
    sys.exit(0)
