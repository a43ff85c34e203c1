"""Build the engine's shared library (libsf.so) in-tree with nvcc for sm_103a.

Usage: python -m greedy_speculative_decoding_gb300.build [--force]

Each .cu file under csrc/ is compiled in parallel, then linked into
libsf.so next to this file; the paged operators' Python binding
(csrc/paged_py.cpp, which reads torch's tensors) becomes the extension module
_paged beside it. Only the binding needs torch and its headers: without torch
this file, run by itself, builds libsf.so for C callers, and a binding that
does not compile is reported when libsf.so is in place. A stamp of the sources,
the flags and torch's version skips the build when nothing changed.
"""

import concurrent.futures as cf
import hashlib
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")
OUT = os.path.join(HERE, "libsf.so")
PY_OUT = os.path.join(HERE, "_paged" + sysconfig.get_config_var("EXT_SUFFIX"))
BUILD_DIR = os.path.join(HERE, "_build")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
         "-I", INCLUDE, "--expt-relaxed-constexpr"]
PY_FLAGS = ["-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-I", sysconfig.get_paths()["include"], "-I", INCLUDE]


def _nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found; the CUDA toolkit is required to build libsf.so")
    return cand


def _sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _torch():
    """torch, which the Python binding is compiled against, or None."""
    try:
        import torch
    except ImportError:
        return None
    return torch


def _stamp(srcs, torch) -> str:
    h = hashlib.sha256()
    h.update(" ".join(ARCH + FLAGS + PY_FLAGS + [torch.__version__ if torch else "no torch"]).encode())
    for f in sorted(os.listdir(CSRC)) + [os.path.join(INCLUDE, "sf.h"), os.path.abspath(__file__)]:
        p = f if os.path.isabs(f) else os.path.join(CSRC, f)
        with open(p, "rb") as fh:
            h.update(p.encode())
            h.update(fh.read())
    return h.hexdigest()


def build(force: bool = False, verbose: bool = False) -> str:
    srcs = _sources()
    torch = _torch()
    stamp = _stamp(srcs, torch)
    stamp_file = os.path.join(BUILD_DIR, "stamp")
    if not force and os.path.exists(OUT) and (os.path.exists(PY_OUT) or not torch) and os.path.exists(stamp_file):
        with open(stamp_file) as fh:
            if fh.read() == stamp:
                return OUT
    os.makedirs(BUILD_DIR, exist_ok=True)
    nvcc = _nvcc()

    def run(what, cmd):
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"{what}:\n{r.stderr}")
        if verbose and r.stderr:
            print(r.stderr, file=sys.stderr)

    def compile_one(src):
        obj = os.path.join(BUILD_DIR, os.path.basename(src)[:-3] + ".o")
        run(f"nvcc failed on {src}", [nvcc, *ARCH, *FLAGS, "-c", src, "-o", obj])
        return obj

    def compile_binding():
        home = os.path.dirname(os.path.abspath(torch.__file__))
        obj = os.path.join(BUILD_DIR, "paged_py.o")
        run("compiling the Python binding failed (libsf.so is built)",
            [gxx, *PY_FLAGS, f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}", "-I",
             os.path.join(home, "include"), "-c", os.path.join(CSRC, "paged_py.cpp"), "-o", obj])
        return obj, os.path.join(home, "lib")

    gxx = shutil.which("g++") or "c++"
    with cf.ThreadPoolExecutor(max_workers=min(8, len(srcs))) as ex:
        binding = ex.submit(compile_binding) if torch else None
        objs = list(ex.map(compile_one, srcs))
    run("link failed", [nvcc, *ARCH, "-shared", "-o", OUT + ".tmp", *objs])
    os.replace(OUT + ".tmp", OUT)
    if binding:
        obj, lib = binding.result()
        run("linking the Python binding failed (libsf.so is built)",
            [gxx, "-shared", obj, "-o", PY_OUT + ".tmp", "-L", HERE, "-l:libsf.so", "-Wl,-rpath,$ORIGIN", "-L", lib,
             "-ltorch_python", "-ltorch_cpu", "-lc10"])
        os.replace(PY_OUT + ".tmp", PY_OUT)
    with open(stamp_file, "w") as fh:
        fh.write(stamp)
    return OUT


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
