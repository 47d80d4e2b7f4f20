"""Build the CUDA library librk.so in-tree for sm_103a with nvcc.

One nvcc process per translation unit, run in parallel, then one shared-object
link.  Objects are rebuilt when any source or header is newer than them.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import importlib.util
import os
import shutil
import subprocess
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(BUILD, "librk.so")
# measurement aid of the benchmark (float32 FMA peak), its own shared object
PROBE_SRC = os.path.join(PKG, "probe", "fma_peak.cu")
PROBE_LIB = os.path.join(BUILD, "libfmapeak.so")

# packs torch tensors for the state space entry points: a Python module that
# includes torch's headers, its own shared object.  Left out where there is no
# torch, which the C library does not need.
BINDING_SRC = os.path.join(PKG, "binding", "state_space_binding.cpp")
BINDING_LIB = os.path.join(BUILD, "state_space_binding.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
CFLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
          "-I", INCLUDE, "-I", CSRC]


def _nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build librk.so")
    return cand


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cpp")))


def _headers():
    return glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh")) + \
        glob.glob(os.path.join(INCLUDE, "*.h"))


def _binding_for():
    """What the Python module is built against: the interpreter's binary
    interface and the installed torch; None without torch (not imported here)."""
    spec = importlib.util.find_spec("torch")
    if spec is None or spec.origin is None:
        return None
    try:
        with open(os.path.join(os.path.dirname(spec.origin), "version.py")) as f:
            version = f.read()
    except OSError:
        version = ""
    return f"{sysconfig.get_config_var('SOABI')}\n{spec.origin}\n{version}"


def _built_for():
    try:
        with open(BINDING_LIB + ".for") as f:
            return f.read()
    except OSError:
        return None


def _build_binding():
    """Compile the Python module against the installed torch, if that is one for CUDA."""
    import torch
    if torch.version.cuda is None:
        return
    root = os.path.dirname(torch.__file__)
    cuda = os.path.join(os.path.dirname(os.path.dirname(_nvcc())), "include")
    tmp = BINDING_LIB + f".{os.getpid()}.tmp"
    include = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
               sysconfig.get_paths()["include"], cuda]
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", *(a for i in include for a in ("-I", i)),
           BINDING_SRC, "-o", tmp, "-L", os.path.join(root, "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu",
           "-ltorch_cuda", "-ltorch_python"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"build of state_space_binding.so failed:\n{r.stderr}")
    os.replace(tmp, BINDING_LIB)


def build(force: bool = False, jobs: int | None = None, verbose: bool = False) -> str:
    """Compile every translation unit under csrc/ and link _build/librk.so;
    beside it, where torch is installed, the module that packs its tensors."""
    nvcc = _nvcc()
    os.makedirs(BUILD, exist_ok=True)
    hdr_time = max([os.path.getmtime(h) for h in _headers()] + [0.0])
    srcs = sources()
    todo = []
    objs = []
    for src in srcs:
        obj = os.path.join(BUILD, os.path.basename(src) + ".o")
        objs.append(obj)
        if force or not os.path.exists(obj) or os.path.getmtime(obj) < max(os.path.getmtime(src), hdr_time):
            todo.append((src, obj))

    def compile_one(item):
        src, obj = item
        tmp = obj + f".{os.getpid()}.tmp"
        cmd = [nvcc, *ARCH, *CFLAGS, "-c", src, "-o", tmp]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {os.path.basename(src)}:\n{r.stderr}")
        os.replace(tmp, obj)
        return r.stderr

    binding_for = _binding_for()
    binding = binding_for is not None and (
        force or not os.path.exists(BINDING_LIB) or _built_for() != binding_for or
        os.path.getmtime(BINDING_LIB) < os.path.getmtime(BINDING_SRC))
    extra = None
    if todo or binding:
        n = jobs or min(len(todo) + 1, max(1, os.cpu_count() or 1))
        with cf.ThreadPoolExecutor(max_workers=n) as ex:
            extra = ex.submit(_build_binding) if binding else None
            for log in ex.map(compile_one, todo):
                if verbose and log:
                    print(log)
    lib_time = os.path.getmtime(LIB) if os.path.exists(LIB) else -1.0
    if todo or lib_time < max(os.path.getmtime(o) for o in objs):
        tmp = LIB + f".{os.getpid()}.tmp"
        cmd = [nvcc, *ARCH, "-shared", "-o", tmp, *objs]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link of librk.so failed:\n{r.stderr}")
        os.replace(tmp, LIB)
    if not os.path.exists(PROBE_LIB) or os.path.getmtime(PROBE_LIB) < os.path.getmtime(PROBE_SRC):
        tmp = PROBE_LIB + f".{os.getpid()}.tmp"
        cmd = [nvcc, *ARCH, *CFLAGS, "-shared", PROBE_SRC, "-o", tmp]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"build of libfmapeak.so failed:\n{r.stderr}")
        os.replace(tmp, PROBE_LIB)
    if extra is not None:
        extra.result()  # raises what went wrong there, with the library in place
        if os.path.exists(BINDING_LIB):
            with open(BINDING_LIB + ".for", "w") as f:
                f.write(binding_for)
    return LIB


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
