"""Build the engine's shared library (libsf.so) in-tree with nvcc for sm_103a.

Usage: python -m greedy_speculative_decoding_gb300.build [--force]

Each .cu file under csrc/ is compiled in parallel, then linked into
libsf.so next to this file; the paged operators' Python binding
(csrc/paged_py.cpp, which reads torch's tensors) becomes the extension module
_paged beside it. A stamp of the sources, the flags and torch's version skips
the build when nothing changed.
"""

import concurrent.futures as cf
import hashlib
import os
import shutil
import subprocess
import sys
import sysconfig

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")
OUT = os.path.join(HERE, "libsf.so")
PY_OUT = os.path.join(HERE, "_paged" + sysconfig.get_config_var("EXT_SUFFIX"))
BUILD_DIR = os.path.join(HERE, "_build")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
         "-I", INCLUDE, "--expt-relaxed-constexpr"]
TORCH = os.path.dirname(os.path.abspath(torch.__file__))
PY_FLAGS = ["-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}", "-I", sysconfig.get_paths()["include"],
            "-I", os.path.join(TORCH, "include"), "-I", INCLUDE]


def _nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found; the CUDA toolkit is required to build libsf.so")
    return cand


def _sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _stamp(srcs) -> str:
    h = hashlib.sha256()
    h.update(" ".join(ARCH + FLAGS + PY_FLAGS + [torch.__version__]).encode())
    for f in sorted(os.listdir(CSRC)) + [os.path.join(INCLUDE, "sf.h"), os.path.abspath(__file__)]:
        p = f if os.path.isabs(f) else os.path.join(CSRC, f)
        with open(p, "rb") as fh:
            h.update(p.encode())
            h.update(fh.read())
    return h.hexdigest()


def build(force: bool = False, verbose: bool = False) -> str:
    srcs = _sources()
    stamp = _stamp(srcs)
    stamp_file = os.path.join(BUILD_DIR, "stamp")
    if not force and os.path.exists(OUT) and os.path.exists(PY_OUT) and os.path.exists(stamp_file):
        with open(stamp_file) as fh:
            if fh.read() == stamp:
                return OUT
    os.makedirs(BUILD_DIR, exist_ok=True)
    nvcc = _nvcc()

    gxx = shutil.which("g++") or "c++"

    def compile_one(src):
        base, ext = os.path.splitext(os.path.basename(src))
        obj = os.path.join(BUILD_DIR, base + ".o")
        cmd = [nvcc, *ARCH, *FLAGS] if ext == ".cu" else [gxx, *PY_FLAGS]
        r = subprocess.run([*cmd, "-c", src, "-o", obj], capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"{cmd[0]} failed on {src}:\n{r.stderr}")
        if verbose and r.stderr:
            print(r.stderr, file=sys.stderr)
        return obj

    with cf.ThreadPoolExecutor(max_workers=min(8, len(srcs))) as ex:
        *objs, py_obj = ex.map(compile_one, srcs + [os.path.join(CSRC, "paged_py.cpp")])
    tmp = OUT + ".tmp"
    cmd = [nvcc, *ARCH, "-shared", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, OUT)
    cmd = [gxx, "-shared", py_obj, "-o", PY_OUT + ".tmp", "-L", HERE, "-l:libsf.so", "-Wl,-rpath,$ORIGIN",
           "-L", os.path.join(TORCH, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"building the Python binding failed:\n{r.stderr}")
    os.replace(PY_OUT + ".tmp", PY_OUT)
    with open(stamp_file, "w") as fh:
        fh.write(stamp)
    return OUT


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
