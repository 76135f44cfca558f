"""Build ``libkmeans_mi355x.so`` (the C-ABI HIP library) in-tree for gfx950.

Usage: ``python -m nearest_centroid_assignment_amd.build [--save-temps]``.
hipcc cross-compiles without a GPU, so this runs on any host with ROCm.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
LIB_NAME = "libkmeans_mi355x.so"
LIB_PATH = os.path.join(HERE, LIB_NAME)
SOURCES = ["api.hip", "assign.hip", "update.hip", "fit.hip", "kmeanspp.hip",
           "experts_api.hip", "tokens.hip", "linear.hip", "linear_bf16.hip", "linear_f16.hip",
           "linear_f32.hip", "adamw.hip"]
# Calibration kernels for the measurements (copy, MFMA loop): a separate library.
CALIB_NAME = "libkm_calib.so"
CALIB_PATH = os.path.join(HERE, CALIB_NAME)
CALIB_SOURCES = ["calib.hip"]
# Marshalling of torch tensors for experts.py: a Python extension module.
TORCH_MODULE_PATH = os.path.join(HERE, "_experts_torch.so")
TORCH_MODULE_SOURCE = "experts_torch.cpp"

# Per-source additional flags. The assignment kernel uses LLVM's iterative
# occupancy-driven scheduler (measured, same-box A/B on the large shapes:
# 0.8-0.9 % faster than the max-ilp strategy, which was itself 1-2 % faster
# than the default; max-memory-clause, iterative-ilp and iterative-minreg
# were 0.3-3 % slower).
EXTRA_FLAGS: dict[str, list[str]] = {
    "assign.hip": ["-mllvm", "-amdgpu-sched-strategy=iterative-maxocc"],
}

HIPCC_FLAGS = [
    "--offload-arch=gfx950",
    "-O3",
    "-std=c++17",
    "-fPIC",
    "-shared",
    "-Wall",
    # No packed-FP32 instructions in generated code.
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
]


def hipcc() -> str:
    for cand in (shutil.which("hipcc"), "/opt/rocm/bin/hipcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found (ROCm is required to build the HIP library)")


def _run(cmd, cwd=None, verbose=False):
    if verbose:
        print(" ".join(cmd), flush=True)
    proc = subprocess.run(cmd, cwd=cwd, capture_output=True, text=True)
    # The host pass warns that it does not know the packed-fp32 feature; that
    # warning is expected. Anything else is shown.
    noise = "'-packed-fp32-ops' is not a recognized feature for this target"
    msgs = [l for l in (proc.stdout + proc.stderr).splitlines() if noise not in l and l.strip()]
    if msgs and (verbose or proc.returncode):
        print("\n".join(msgs), file=sys.stderr)
    if proc.returncode != 0:
        raise RuntimeError(f"the compiler failed with exit code {proc.returncode}: {' '.join(cmd)}")


def _compile(sources, out_path, verbose: bool, save_temps: bool, extra_flags=None) -> str:
    """Compile each source to an object (in parallel), then link the library.

    ``extra_flags`` maps a source name to additional hipcc flags for it.
    """
    from concurrent.futures import ThreadPoolExecutor

    extra_flags = extra_flags or {}
    objdir = os.path.join(HERE, "..", "_build")
    os.makedirs(objdir, exist_ok=True)
    compile_flags = [f for f in HIPCC_FLAGS if f != "-shared"]

    def one(src):
        obj = os.path.join(objdir, os.path.basename(out_path) + "." + src + ".o")
        cmd = [hipcc(), *compile_flags, *extra_flags.get(src, []), "-c", "-o", obj,
               os.path.join(CSRC, src)]
        if save_temps:
            cmd.insert(1, "-save-temps")
        _run(cmd, cwd=objdir, verbose=verbose)
        return obj

    with ThreadPoolExecutor(max_workers=len(sources)) as pool:
        objs = list(pool.map(one, sources))
    out_tmp = out_path + ".tmp"
    _run([hipcc(), "--offload-arch=gfx950", "-shared", "-fPIC", "-o", out_tmp, *objs],
         verbose=verbose)
    os.replace(out_tmp, out_path)
    return out_path


def cxx() -> str | None:
    """The C++ compiler of the torch module: the system's, or else ROCm's."""
    for cand in (shutil.which("g++"), shutil.which("c++"), shutil.which("amdclang++"),
                 "/opt/rocm/bin/amdclang++"):
        if cand and os.path.exists(cand):
            return cand
    return None


def torch_module_needs() -> str | None:
    """What the torch module cannot be built without and is missing here."""
    import importlib.util
    import sysconfig

    if not cxx():
        return "a C++ compiler"
    if not os.path.exists(os.path.join(sysconfig.get_paths()["include"], "Python.h")):
        return "Python's C headers"
    spec = importlib.util.find_spec("torch")
    if spec is None:
        return "torch"
    if not os.path.isdir(os.path.join(os.path.dirname(spec.origin), "include", "torch")):
        return "torch's C++ headers"
    return None


def build_torch_module(verbose: bool = False) -> str | None:
    """Compile the module that marshals torch tensors to the experts' entry
    points (host code against torch's C++ headers; it links torch alone). Where
    something that only it needs is missing, says so and returns None: the libraries
    are built all the same, and experts.py raises when it is used."""
    import sysconfig

    missing = torch_module_needs()
    if missing:
        print(f"{os.path.basename(TORCH_MODULE_PATH)} is not built (it takes torch tensors to the "
              f"expert operators): {missing} not found", file=sys.stderr)
        if os.path.exists(TORCH_MODULE_PATH):
            os.remove(TORCH_MODULE_PATH)  # of other sources, for all that is known
        return None
    from torch.utils.cpp_extension import include_paths, library_paths

    out_tmp = TORCH_MODULE_PATH + ".tmp"
    _run([cxx(), "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall", "-D__HIP_PLATFORM_AMD__=1",
          "-DUSE_ROCM=1", *(f"-isystem{p}" for p in include_paths()), "-isystem/opt/rocm/include",
          f"-isystem{sysconfig.get_paths()['include']}", os.path.join(CSRC, TORCH_MODULE_SOURCE),
          *(f"-L{p}" for p in library_paths()), "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10",
          "-lc10_hip", "-o", out_tmp], verbose=verbose)
    os.replace(out_tmp, TORCH_MODULE_PATH)
    return TORCH_MODULE_PATH


def build(verbose: bool = False, save_temps: bool = False) -> str:
    """Compile the k-means library, the calibration library and the torch
    module; returns the path of the k-means library."""
    from concurrent.futures import ThreadPoolExecutor

    with ThreadPoolExecutor(max_workers=1) as pool:
        module = pool.submit(build_torch_module, verbose)
        _compile(CALIB_SOURCES, CALIB_PATH, verbose, save_temps)
        path = _compile(SOURCES, LIB_PATH, verbose, save_temps, EXTRA_FLAGS)
        module.result()
    return path


if __name__ == "__main__":
    build(verbose=True, save_temps="--save-temps" in sys.argv)
