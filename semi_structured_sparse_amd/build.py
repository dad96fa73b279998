"""Build libnmsparse.so in place with hipcc for gfx950, and _nmtorch.so, the quick way from torch
tensors to its decoding calls, with the host compiler where that and torch are there (the calls do
without it, in more time).

Usage: ``python -m semi_structured_sparse_amd.build`` (or call ``build()``).
"""
from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sys
import sysconfig
import tempfile
import warnings
from concurrent.futures import ThreadPoolExecutor

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG_DIR)
CSRC = os.path.join(PKG_DIR, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB_NAME = "libnmsparse.so"
EXT_NAME = "_nmtorch.so"
ARCH = os.environ.get("NM_OFFLOAD_ARCH", "gfx950")

HIP_FLAGS = [
    f"--offload-arch={ARCH}",
    "-O3",
    "-std=c++17",
    "-fPIC",
    "-Wall",
    # Packed-FP32 instructions are kept out of the generated code on this platform.
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
]


def hipcc() -> str:
    for cand in (os.environ.get("HIPCC"), shutil.which("hipcc"), "/opt/rocm/bin/hipcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found (ROCm is required to build libnmsparse.so)")


def sources() -> list:
    return sorted(glob.glob(os.path.join(CSRC, "*.hip")))


def _host_compiler() -> str:
    return os.environ.get("CXX", "g++")


def _rocm() -> str:
    return os.environ.get("ROCM_PATH", "/opt/rocm")


def extension_obstacle() -> str | None:
    """What the extension would need and is not here; None: it can be built."""
    try:
        import torch
    except ImportError:
        return "torch is not importable"
    if shutil.which(_host_compiler()) is None:
        return f"no host compiler {_host_compiler()}"
    base = os.path.dirname(torch.__file__)
    for path in (os.path.join(base, "include", "torch", "csrc", "autograd", "python_variable.h"),
                 os.path.join(base, "lib", "libc10_hip.so"),
                 os.path.join(_rocm(), "include", "hip", "hip_runtime_api.h"),
                 os.path.join(sysconfig.get_paths()["include"], "Python.h")):
        if not os.path.exists(path):
            return f"no {path}"
    return None


def extension_command(out: str) -> list:
    """The host compiler's command for csrc/nm_torch.cpp, against the installed torch."""
    import torch

    base = os.path.dirname(torch.__file__)
    inc, lib = os.path.join(base, "include"), os.path.join(base, "lib")
    # the HIP headers, under a host compiler, have to be told the platform
    return [_host_compiler(), "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall", "-DUSE_ROCM",
            "-D__HIP_PLATFORM_AMD__", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
            f"-I{INCLUDE}", "-isystem", inc, "-isystem", os.path.join(inc, "torch", "csrc", "api", "include"),
            "-isystem", os.path.join(_rocm(), "include"), "-isystem", sysconfig.get_paths()["include"],
            os.path.join(CSRC, "nm_torch.cpp"), "-o", out, f"-L{lib}", "-lc10", "-lc10_hip", "-ltorch_cpu",
            "-ltorch_python", f"-Wl,-rpath,{lib}"]


def build_extension(verbose: bool = False) -> str:
    """Compile csrc/nm_torch.cpp into PKG_DIR/_nmtorch.so (always recompiles)."""
    out = os.path.join(PKG_DIR, EXT_NAME)
    tmp = out + ".tmp"
    cmd = extension_command(tmp)
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"{cmd[0]} failed ({res.returncode}):\n{res.stdout}\n{res.stderr}")
    os.replace(tmp, out)
    return out


def build(verbose: bool = False) -> str:
    """Compile every HIP source into PKG_DIR/libnmsparse.so, and the torch extension beside it
    (always recompiles). Where the extension cannot be built here, an earlier one is taken away and
    a warning says why; one that does not compile is an error."""
    obstacle = extension_obstacle()
    if obstacle is not None:
        earlier = os.path.join(PKG_DIR, EXT_NAME)
        if os.path.exists(earlier):
            os.remove(earlier)
        warnings.warn(f"_nmtorch.so is not built: {obstacle}; the decoding calls go through decode.py's own checks",
                      RuntimeWarning, stacklevel=2)
        return build_library(verbose)
    with ThreadPoolExecutor(1) as pool:      # the extension while hipcc works
        extension = pool.submit(build_extension, verbose)
        out = build_library(verbose)
        extension.result()
    return out


def _workers() -> int:
    """Compilers at once: MAX_JOBS, else the CPUs of this process, up to 16."""
    return max(1, min(16, int(os.environ.get("MAX_JOBS") or len(os.sched_getaffinity(0)))))


def build_library(verbose: bool = False) -> str:
    """Compile every HIP source into PKG_DIR/libnmsparse.so (always recompiles): a compiler for each
    source, several at once, then the link."""
    out = os.path.join(PKG_DIR, LIB_NAME)
    tmp = out + ".tmp"

    def run(cmd) -> str:
        if verbose:
            print(" ".join(cmd), flush=True)
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError(f"hipcc failed ({res.returncode}):\n{res.stdout}\n{res.stderr}")
        return res.stderr

    with tempfile.TemporaryDirectory() as place, ThreadPoolExecutor(_workers()) as pool:
        objects = {src: os.path.join(place, os.path.basename(src) + ".o") for src in sources()}
        said = list(pool.map(lambda src: run([hipcc(), *HIP_FLAGS, f"-I{INCLUDE}", f"-I{CSRC}", "-c", src, "-o",
                                              objects[src]]), objects))
        said.append(run([hipcc(), f"--offload-arch={ARCH}", "-fPIC", "-shared", *objects.values(), "-o", tmp]))
    # the host pass does not know the packed-fp32 target feature and says so; drop that noise
    noise = ("packed-fp32-ops", "is not a recognized feature", "--hip-link")
    msgs = [l for err in said for l in err.splitlines() if l.strip() and not any(n in l for n in noise)]
    if msgs and verbose:
        print("\n".join(msgs), file=sys.stderr)
    os.replace(tmp, out)
    return out


if __name__ == "__main__":
    print(build(verbose=True))
