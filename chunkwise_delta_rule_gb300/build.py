"""Build libkda.so in-tree with nvcc for sm_103a (GB300).

Each translation unit under csrc/ is compiled in parallel, then linked into
chunkwise_delta_rule_gb300/libkda.so (static CUDA runtime, no torch). Beside them
csrc/binding.cpp becomes the Python extension _binding.so (torch's headers, the
host compiler), which calls libkda.so. libkda.so is built without torch's headers
or a host compiler for them too; the extension is then missing.
``python -m chunkwise_delta_rule_gb300.build`` runs it from the command line.
"""

from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libkda.so")
BINDING = os.path.join(PKG, "_binding.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
         "-Xptxas", "-v", "-I", os.path.join(ROOT, "include")]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _stale(obj: str, src: str) -> bool:
    if not os.path.exists(obj):
        return True
    t = os.path.getmtime(obj)
    deps = [src] + [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cuh")]
    deps.append(os.path.join(ROOT, "include", "kda.h"))
    return any(os.path.getmtime(d) > t for d in deps)


def _compile(src: str) -> str:
    obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
    if _stale(obj, src):
        log = obj + ".log"
        cmd = [nvcc()] + ARCH + FLAGS + ["-c", src, "-o", obj + ".tmp"]
        with open(log, "w") as fh:
            r = subprocess.run(cmd, stdout=fh, stderr=subprocess.STDOUT)
        if r.returncode != 0:
            sys.stderr.write(open(log).read())
            raise RuntimeError("nvcc failed for " + src)
        os.replace(obj + ".tmp", obj)
    return obj


def _compile_binding() -> str:
    """csrc/binding.cpp against the installed torch (rebuilt when that changes)."""
    import torch
    from torch.utils import cpp_extension

    src = os.path.join(CSRC, "binding.cpp")
    obj = os.path.join(BUILD, "binding_torch%s.o" % torch.__version__)
    if _stale(obj, src):
        inc = [x for p in cpp_extension.include_paths() for x in ("-isystem", p)]
        inc += ["-isystem", os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include"),
                "-isystem", sysconfig.get_paths()["include"]]
        cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-DTORCH_EXTENSION_NAME=_binding",
               "-DTORCH_API_INCLUDE_EXTENSION_H", "-D_GLIBCXX_USE_CXX11_ABI=%d" % torch.compiled_with_cxx11_abi()]
        with open(obj + ".log", "w") as fh:
            r = subprocess.run(cmd + inc + ["-c", src, "-o", obj + ".tmp"], stdout=fh, stderr=subprocess.STDOUT)
        if r.returncode != 0:
            sys.stderr.write(open(obj + ".log").read())
            raise RuntimeError("the host compiler failed for " + src)
        os.replace(obj + ".tmp", obj)
    return obj


def _link_binding(obj: str) -> None:
    import torch

    if os.path.exists(BINDING) and os.path.getmtime(BINDING) >= os.path.getmtime(obj):
        return
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = BINDING + ".tmp%d" % os.getpid()
    subprocess.run([os.environ.get("CXX", "g++"), "-shared", "-o", tmp, obj, "-L", lib, "-ltorch_python", "-ltorch", "-ltorch_cpu",
                    "-lc10", "-lc10_cuda", "-L", PKG, "-l:libkda.so", "-Wl,-rpath,$ORIGIN", "-Wl,-rpath," + lib], check=True)
    os.replace(tmp, BINDING)


def build(force: bool = False, jobs: int | None = None) -> str:
    os.makedirs(BUILD, exist_ok=True)
    if force:
        for f in os.listdir(BUILD):
            os.remove(os.path.join(BUILD, f))
    srcs = sources()
    jobs = jobs or min(len(srcs), os.cpu_count() or 1)
    with cf.ThreadPoolExecutor(jobs + 1) as ex:
        binding = ex.submit(_compile_binding)
        objs = list(ex.map(_compile, srcs))
    if force or not os.path.exists(LIB) or any(os.path.getmtime(o) > os.path.getmtime(LIB) for o in objs):
        tmp = LIB + ".tmp%d" % os.getpid()
        cmd = [nvcc()] + ARCH + ["-shared", "-o", tmp] + objs + ["-cudart", "static"]
        subprocess.run(cmd, check=True)
        os.replace(tmp, LIB)
    try:
        _link_binding(binding.result())
    except (RuntimeError, OSError, ImportError, subprocess.CalledProcessError) as e:
        # libkda.so does not need it: only the layer operators' Python entries do, and they fail where they are used
        if os.path.exists(BINDING):
            os.remove(BINDING)   # of other sources
        sys.stderr.write("_binding.so was not built (%s: %s): the layer operators' Python entries are not there\n"
                         % (type(e).__name__, e))
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv))
    sys.exit(not os.path.exists(BINDING))
