"""Build libecc_mi355.so in-tree with hipcc for gfx950.

Usage: ``python -m euler_characteristic_curves_amd.build`` (also called by
``__graft_entry__.build()``).  Sources are compiled in parallel into
``_build/`` at the repository root and linked into
``euler_characteristic_curves_amd/libecc_mi355.so``.  The benchmark's
sigmoid-rate probe is linked on its own into ``libecc_sigmoid_rate.so``, and
torch's binding of the norm's autograd nodes into ``_torch.so``.
"""

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libecc_mi355.so")

SOURCES = ["ecc_api.cpp", "ecc_hard.hip", "ecc_soft.hip", "ecc_soft_grad.hip", "ecc_height.hip", "ecc_static.hip",
           "ecc_train_api.cpp", "ecc_norm_f32.hip", "ecc_norm_f16.hip", "ecc_norm_bf16.hip", "ecc_orth.hip", "ecc_orth_long.hip",
           "ecc_orth_thin_f32.hip", "ecc_orth_thin_f16.hip", "ecc_orth_thin_bf16.hip", "ecc_block_api.cpp",
           "ecc_residual.hip", "ecc_recurrence.hip", "ecc_glu_f32.hip", "ecc_glu_f16.hip", "ecc_glu_bf16.hip"]
RATE_SOURCE = "ecc_sigmoid_rate.hip"
RATE_LIB = os.path.join(PKG, "libecc_sigmoid_rate.so")
TORCH_SOURCES = ["ecc_torch.cpp", "ecc_torch_block.cpp"]
TORCH_LIB = os.path.join(PKG, "_torch.so")
ARCH = os.environ.get("ECC_OFFLOAD_ARCH", "gfx950")

COMMON = [
    "-O3", "-std=c++17", "-fPIC", f"--offload-arch={ARCH}",
    # no packed-fp32 instructions anywhere in the device code
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall", "-Wno-unused-function", "-Wno-unknown-warning-option",
    f"-I{INCLUDE}", f"-I{CSRC}",
]


def hipcc():
    for cand in (os.environ.get("HIPCC"), shutil.which("hipcc"), "/opt/rocm/bin/hipcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found (ROCm is required to build libecc_mi355)")


def _compile(src):
    obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
    lang = ["-x", "hip"]
    cmd = [hipcc()] + COMMON + lang + ["-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed for {src}:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    return obj, r.stderr


def _compile_torch(src):
    """A source of the binding against torch's headers: host code only."""
    import sysconfig

    import torch
    from torch.utils.cpp_extension import include_paths

    obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
    cmd = [shutil.which("g++") or hipcc(), "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-D__HIP_PLATFORM_AMD__=1",
           "-DUSE_ROCM=1", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           f"-isystem{sysconfig.get_paths()['include']}"]
    cmd += [f"-isystem{d}" for d in include_paths("cuda")] + ["-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"compilation failed for {src}:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    return obj


def _torch_libs():
    import torch

    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    return [f"-L{libs}", "-lc10", "-lc10_hip", "-ltorch_cpu", "-ltorch_hip", "-ltorch_python", f"-L{PKG}",
            "-l:libecc_mi355.so", "-Wl,-rpath,$ORIGIN"]


def build(verbose=False):
    """Compile every source and link the shared libraries; returns the path of libecc_mi355.so."""
    os.makedirs(BUILD, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=8) as ex:
        torch_objs = ex.map(_compile_torch, TORCH_SOURCES)
        results = list(ex.map(_compile, SOURCES + [RATE_SOURCE]))
        torch_objs = list(torch_objs)
    rate_obj = results.pop()[0]
    objs = [o for o, _ in results]
    if verbose:
        for _, err in results:
            if err.strip():
                print(err, file=sys.stderr)
    for lib, lib_objs in ((LIB, objs), (RATE_LIB, [rate_obj]), (TORCH_LIB, torch_objs + _torch_libs())):
        tmp = lib + ".tmp"
        cmd = [hipcc(), f"--offload-arch={ARCH}", "-shared", "-fPIC", "-o", tmp] + lib_objs
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, lib)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
