"""Build libttt.so (the C-ABI CUDA library) in-tree for sm_100a with nvcc, and the CPython binding _native.so.

    python -m vision_test_token_b200.build [--force]

Every .cu file under csrc/ is compiled with
``-gencode arch=compute_100a,code=sm_100a -lineinfo -O3`` and linked, with the static CUDA runtime,
into ``vision_test_token_b200/libttt.so``.  No torch headers or libraries are involved in that.
csrc/native.cpp (the fast marshalling of torch tensors for the per-token entries) is compiled with g++ against
torch's headers into ``vision_test_token_b200/_native.so``, which links to libttt.so.  It is built again when torch or Python is
another one, and left out, with a note, where there is no torch: libttt.so serves C callers without it.
"""
import importlib.metadata
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OUT = os.path.join(PKG, "libttt.so")
NATIVE = os.path.join(PKG, "_native.so")
BUILD_DIR = os.path.join(PKG, "_build")
NATIVE_KEY = os.path.join(BUILD_DIR, "native.key")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]


def _nvcc():
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", shutil.which("nvcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libttt.so")


def _sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _newest(files):
    return max(os.path.getmtime(f) for f in files)


def _lib_deps():
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cu", ".cuh", ".h"))]
    return files + [os.path.join(INCLUDE, "ttt.h")]


def _native_key():
    """What _native.so is built for besides its sources; None without torch (found without the slow import of it)."""
    try:
        return f"torch {importlib.metadata.version('torch')}, {sys.implementation.cache_tag}"
    except importlib.metadata.PackageNotFoundError:
        return None


def _native_is_current(key):
    if not os.path.exists(NATIVE) or not os.path.exists(NATIVE_KEY):
        return False
    with open(NATIVE_KEY) as f:
        if f.read() != key:
            return False
    return os.path.getmtime(NATIVE) >= _newest([os.path.join(CSRC, "native.cpp"), os.path.join(INCLUDE, "ttt.h")])


def build(force: bool = False, verbose: bool = False) -> str:
    if force or not os.path.exists(OUT) or os.path.getmtime(OUT) < _newest(_lib_deps()):
        _build_lib(verbose)
    key = _native_key()
    if key is None:
        sys.stderr.write("no torch here: libttt.so is built, its binding for torch tensors (_native.so) is not\n")
    elif force or not _native_is_current(key):
        _build_native()
        os.makedirs(os.path.dirname(NATIVE_KEY), exist_ok=True)
        with open(NATIVE_KEY, "w") as f:
            f.write(key)
    return OUT


def _build_lib(verbose):
    nvcc = _nvcc()
    os.makedirs(BUILD_DIR, exist_ok=True)
    common = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I", INCLUDE, "-I", CSRC]
    if verbose:
        common += ["-Xptxas", "-v"]
    objs = []
    procs = []
    for src in _sources():
        obj = os.path.join(BUILD_DIR, os.path.basename(src)[:-3] + ".o")
        objs.append(obj)
        procs.append(subprocess.Popen([nvcc, *common, "-c", src, "-o", obj],
                                      stdout=subprocess.PIPE, stderr=subprocess.STDOUT))
    failed = []
    for src, p in zip(_sources(), procs):
        out, _ = p.communicate()
        if out and (verbose or p.returncode != 0):
            sys.stderr.write(out.decode())
        if p.returncode != 0:
            failed.append(src)
    if failed:
        raise RuntimeError("nvcc failed on: " + ", ".join(failed))
    tmp = OUT + ".tmp"
    subprocess.run([nvcc, *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs], check=True)
    os.replace(tmp, OUT)


def _build_native():
    import torch                                # its headers and libraries; the import is slow, hence here
    root = os.path.dirname(torch.__file__)
    include = [INCLUDE, os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
               os.path.join(os.path.dirname(os.path.dirname(_nvcc())), "include"), sysconfig.get_paths()["include"]]
    tmp = NATIVE + ".tmp"
    subprocess.run([shutil.which("g++") or "g++", "-O2", "-std=c++17", "-fPIC", "-shared",
                    f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", *(f"-I{d}" for d in include),
                    os.path.join(CSRC, "native.cpp"), "-o", tmp, "-L", PKG, "-l:libttt.so", "-L", os.path.join(root, "lib"),
                    "-ltorch_python", "-ltorch_cpu", "-lc10", "-Wl,-rpath,$ORIGIN"], check=True)
    os.replace(tmp, NATIVE)


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
