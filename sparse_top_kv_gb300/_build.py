"""Build libhs.so (the C ABI of include/hs_api.h) from csrc/*.cu with nvcc for
sm_103a.  One nvcc process per translation unit, run in parallel, then one
link.  Output: sparse_top_kv_gb300/_build/libhs.so (git-ignored, in-tree), and
beside it the Python extension of the hot calls (csrc/hs_binding.cpp) where
Python's headers are installed; without it they go through ctypes."""
import concurrent.futures as cf
import os
import shutil
import subprocess
import sys
import sysconfig
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OUT_DIR = os.path.join(PKG, "_build")
LIB = os.path.join(OUT_DIR, "libhs.so")
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


def _fresh(path):
    return os.path.exists(path) and os.path.getmtime(path) >= _deps_mtime()


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    """Build what is missing or older than its sources; returns libhs.so's path.
    The extension is an accelerator: a failure to build it is a warning."""
    os.makedirs(OUT_DIR, exist_ok=True)
    binding = binding_path()
    _drop_other_bindings(binding)
    want_lib = force or not _fresh(LIB)
    # A failed attempt is not repeated until something changes.
    want_binding = binding is not None and (
        force or not (_fresh(binding) or _fresh(binding + ".failed")))
    if want_lib or want_binding:
        with cf.ThreadPoolExecutor(max_workers=max(1, min(8, os.cpu_count() or 1))) as ex:
            compiled = ex.submit(_compile_binding) if want_binding else None
            if want_lib:
                _build_lib(ex, verbose, extra_flags)
        if want_binding:
            _build_binding(binding, compiled)
    return LIB


def _build_lib(ex, verbose, extra_flags):
    cc = nvcc()

    def compile_one(src):
        obj = os.path.join(OUT_DIR, src[:-3] + ".o")
        cmd = [cc, *ARCH, *FLAGS, *extra_flags, "-c", os.path.join(CSRC, src), "-o", obj]
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{res.stderr}")
        if verbose and res.stderr:
            print(res.stderr)
        return obj

    objs = list(ex.map(compile_one, _sources()))
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [cc, *ARCH, "-shared", "-o", tmp, *objs]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"nvcc link failed:\n{res.stderr}")
    os.replace(tmp, LIB)


def _build_binding(path, compiled):
    """Link the extension from its object file (a future), or record why not."""
    # The one of an earlier build may call functions that have changed.
    for old in (path, path + ".failed"):
        if os.path.exists(old):
            os.remove(old)
    try:
        tmp = path + f".tmp{os.getpid()}"
        _gcc("-shared", compiled.result(), "-o", tmp, "-L" + OUT_DIR, "-l:" + os.path.basename(LIB),
             "-L" + os.path.join(_torch(), "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10",
             "-Wl,-rpath,$ORIGIN")
        os.replace(tmp, path)
    except (RuntimeError, OSError) as e:
        with open(path + ".failed", "w") as f:
            f.write(str(e))
        warnings.warn(f"the extension of the hot calls was not built; they go through ctypes: {e}")


def binding_path():
    """Path of the extension for this Python and this torch, or None where
    Python's headers or a compiler are missing."""
    if _python_include() is None:
        return None
    import torch
    return os.path.join(OUT_DIR, f"_hs_binding-{sys.implementation.cache_tag}-"
                                 f"torch{torch.__version__}.so")


def _drop_other_bindings(path):
    """Extensions of another Python or torch, or ones that cannot be rebuilt here."""
    for f in os.listdir(OUT_DIR):
        full = os.path.join(OUT_DIR, f)
        if f.startswith("_hs_binding") and f.endswith(".so") and full != path:
            os.remove(full)


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
    import torch
    obj = os.path.join(OUT_DIR, "hs_binding.o")
    _gcc("-O2", "-std=c++17", "-fPIC",
         f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
         "-I" + _python_include(), "-I" + INCLUDE, "-I" + os.path.join(_torch(), "include"), "-c",
         os.path.join(CSRC, "hs_binding.cpp"), "-o", obj)
    return obj


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv,
                extra_flags=["-Xptxas", "-v"] if "--ptxas" in sys.argv else []))
