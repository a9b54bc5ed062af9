"""Build libhs.so (the C ABI of include/hs_api.h) from csrc/*.cu with nvcc for
sm_103a.  One nvcc process per translation unit, run in parallel, then one
link.  Output: sparse_top_kv_gb300/_build/libhs.so (git-ignored, in-tree), and
beside it the Python extension of the hot calls (csrc/hs_binding.cpp) where
Python's headers are installed."""
import concurrent.futures as cf
import os
import shutil
import subprocess
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OUT_DIR = os.path.join(PKG, "_build")
LIB = os.path.join(OUT_DIR, "libhs.so")
BINDING = os.path.join(OUT_DIR, "_hs_binding.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
         "-I" + INCLUDE, "-I" + CSRC]


def nvcc():
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: libhs.so cannot be built")


def _sources():
    return sorted(f for f in os.listdir(CSRC) if f.endswith(".cu"))


def _deps_mtime():
    paths = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    paths += [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE)]
    paths.append(os.path.abspath(__file__))
    return max(os.path.getmtime(p) for p in paths)


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    os.makedirs(OUT_DIR, exist_ok=True)
    done = [LIB] + ([BINDING] if _python_include() else [])
    if not force and all(os.path.exists(p) and os.path.getmtime(p) >= _deps_mtime()
                         for p in done):
        return LIB
    cc = nvcc()
    objs = []

    def compile_one(src):
        obj = os.path.join(OUT_DIR, src[:-3] + ".o")
        cmd = [cc, *ARCH, *FLAGS, *extra_flags, "-c", os.path.join(CSRC, src), "-o", obj]
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{res.stderr}")
        if verbose and res.stderr:
            print(res.stderr)
        return obj

    with cf.ThreadPoolExecutor(max_workers=max(1, min(8, os.cpu_count() or 1))) as ex:
        binding = ex.submit(_compile_binding)
        objs = list(ex.map(compile_one, _sources()))
        binding = binding.result()
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [cc, *ARCH, "-shared", "-o", tmp, *objs]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"nvcc link failed:\n{res.stderr}")
    os.replace(tmp, LIB)
    if binding is not None:
        tmp = BINDING + f".tmp{os.getpid()}"
        _gcc("-shared", binding, "-o", tmp, "-L" + OUT_DIR, "-l:libhs.so",
             "-L" + os.path.join(_torch(), "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10",
             "-Wl,-rpath,$ORIGIN")
        os.replace(tmp, BINDING)
    return LIB


def _python_include():
    """Folder of Python.h, or None."""
    inc = sysconfig.get_paths()["include"]
    return inc if os.path.exists(os.path.join(inc, "Python.h")) and shutil.which("g++") else None


def _torch():
    import torch
    return os.path.dirname(torch.__file__)


def _gcc(*args):
    res = subprocess.run(["g++", *args], capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"g++ failed on hs_binding.cpp:\n{res.stderr}")


def _compile_binding():
    inc = _python_include()
    if inc is None:
        return None
    obj = os.path.join(OUT_DIR, "hs_binding.o")
    _gcc("-O2", "-std=c++17", "-fPIC", "-I" + inc, "-I" + INCLUDE,
         "-I" + os.path.join(_torch(), "include"), "-c", os.path.join(CSRC, "hs_binding.cpp"),
         "-o", obj)
    return obj


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv,
                extra_flags=["-Xptxas", "-v"] if "--ptxas" in sys.argv else []))
