"""Build libtopk.so in-tree with nvcc for sm_103a.

Each .cu file compiles in parallel to an object file under ``_lib/``; the
objects link into ``_lib/libtopk.so`` (CUDA runtime linked statically).
Beside it, g++ compiles the Python binding of the key-value cache operators
(csrc/kv_binding.cpp) against the installed torch into ``_lib/kv_binding-<torch's
version><Python's suffix>``, so that a module built for another torch or Python
is never taken for this one's.  Nothing is rebuilt when both are newer than
every source.  The library needs no torch: where there is none, or the binding
does not compile, it is built all the same.
"""
from __future__ import annotations

import glob
import importlib.util
import os
import runpy
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB_DIR = os.path.join(HERE, "_lib")
LIB_PATH = os.path.join(LIB_DIR, "libtopk.so")
BINDING_SRC = os.path.join(CSRC, "kv_binding.cpp")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
              "--expt-relaxed-constexpr"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is needed to build libtopk.so")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _inputs():
    return sources() + [BINDING_SRC] + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + \
        glob.glob(os.path.join(ROOT, "include", "*.h"))


def binding_path() -> str | None:
    """Where the binding for the running Python and its torch belongs; None without torch."""
    torch = importlib.util.find_spec("torch")
    if torch is None:
        return None
    version = runpy.run_path(os.path.join(torch.submodule_search_locations[0], "version.py"))["__version__"]
    return os.path.join(LIB_DIR, f"kv_binding-{version}{sysconfig.get_config_var('EXT_SUFFIX')}")


def up_to_date() -> bool:
    made = [p for p in (LIB_PATH, binding_path()) if p]
    if not all(os.path.exists(p) for p in made):
        return False
    t = min(os.path.getmtime(p) for p in made)
    return all(os.path.getmtime(p) <= t for p in _inputs())


def _binding_command(out: str):
    """g++ on the binding, against the torch and Python that are running."""
    torch_dir = importlib.util.find_spec("torch").submodule_search_locations[0]
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(_nvcc())))
    include = [os.path.join(torch_dir, "include"),
               os.path.join(torch_dir, "include", "torch", "csrc", "api", "include"),
               os.path.join(cuda, "include"), sysconfig.get_paths()["include"]]
    return ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-o", out, BINDING_SRC,
            *(f"-I{p}" for p in include), f"-L{os.path.join(torch_dir, 'lib')}", "-ltorch_python", "-ltorch",
            "-ltorch_cuda", "-ltorch_cpu", "-lc10_cuda", "-lc10"]


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and up_to_date():
        return LIB_PATH
    nvcc = _nvcc()
    os.makedirs(LIB_DIR, exist_ok=True)
    procs = []
    objs = []
    for src in sources():
        obj = os.path.join(LIB_DIR, os.path.basename(src)[:-3] + ".o")
        objs.append(obj)
        cmd = [nvcc, *ARCH, *NVCC_FLAGS, "-I", os.path.join(ROOT, "include"), "-c", src, "-o", obj]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        procs.append((src, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)))
    binding = binding_path()
    if binding:
        procs.append((BINDING_SRC, subprocess.Popen(_binding_command(binding + f".tmp{os.getpid()}"),
                                                    stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)))
    failed = []
    for src, p in procs:
        out, _ = p.communicate()
        if verbose or p.returncode != 0:
            sys.stderr.write(out)
        if p.returncode != 0:
            failed.append(src)
    if set(failed) <= {BINDING_SRC}:
        tmp = LIB_PATH + f".tmp{os.getpid()}"
        subprocess.run([nvcc, *ARCH, "-shared", "-o", tmp, *objs, "-cudart", "static"], check=True)
        os.replace(tmp, LIB_PATH)
    if failed:
        raise RuntimeError("compilation failed for: " + ", ".join(os.path.basename(f) for f in failed))
    if binding:
        os.replace(binding + f".tmp{os.getpid()}", binding)
    return LIB_PATH


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
