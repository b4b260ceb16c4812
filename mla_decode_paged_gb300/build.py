"""Build the native library ``_build/libmla_decode.so`` in-tree with nvcc.

Every ``csrc/*.cu`` translation unit is compiled in parallel for sm_103a
only, then linked into one shared library (CUDA runtime linked statically,
so the library carries no dependency on a particular libcudart build).
``csrc/binding.cpp``, the Python module over part of it, is compiled beside
them with the host compiler against the installed torch (its version is in
the module's file name) and linked to the library.  The library needs
neither: where the module cannot be built (no Python headers, say) the library
is there all the same, and the calls that go through the module raise.
"""

from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sysconfig
import warnings
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(BUILD, "libmla_decode.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr"]


def _torch_dir() -> str:
    import torch

    return os.path.dirname(torch.__file__)


def ops_path() -> str:
    """The Python module's file, for the installed torch and Python."""
    import torch

    tag = "%s-%s" % (torch.__version__, sysconfig.get_config_var("SOABI"))
    return os.path.join(BUILD, "mla_ops-%s.so" % "".join(c if c.isalnum() or c in ".-" else "_" for c in tag))


def _cuda_include() -> str:
    return os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include")


def _ops_compile(obj: str):
    t = os.path.join(_torch_dir(), "include")
    import torch

    return ["g++", "-O2", "-std=c++17", "-fPIC", "-D_GLIBCXX_USE_CXX11_ABI=%d" % torch._C._GLIBCXX_USE_CXX11_ABI,
            "-I" + t, "-I" + os.path.join(t, "torch", "csrc", "api", "include"), "-I" + _cuda_include(),
            "-I" + sysconfig.get_paths()["include"], "-c", os.path.join(CSRC, "binding.cpp"), "-o", obj]


def _ops_link(obj: str, out: str):
    lib = os.path.join(_torch_dir(), "lib")
    return ["g++", "-shared", "-o", out, obj, "-L" + lib, "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda",
            "-ltorch_python", "-L" + BUILD, "-lmla_decode", "-Wl,-rpath,$ORIGIN"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found (CUDA toolkit required to build the library)")


def _deps():
    return glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(ROOT, "include", "*.h"))


def _stale(target: str, sources) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(s) > t for s in sources)


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile (if stale) and link; returns the library path.  A failure of
    the Python module alone is a RuntimeWarning."""
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    deps = _deps()
    jobs = []
    objs = []
    for s in srcs:
        obj = os.path.join(BUILD, os.path.basename(s)[:-3] + ".o")
        objs.append(obj)
        if force or _stale(obj, [s] + deps):
            jobs.append([cc, *ARCH, *NVCC_FLAGS, "-c", s, "-o", obj])
    ops = ops_path()
    ops_obj = ops[:-3] + ".o"
    ops_stale = force or _stale(ops_obj, [os.path.join(CSRC, "binding.cpp")] + deps)

    def run(cmd):
        if verbose:
            print(" ".join(cmd), flush=True)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("%s failed:\n%s\n%s" % (os.path.basename(cmd[0]), " ".join(cmd), r.stderr))
        return r.stderr

    with ThreadPoolExecutor(max_workers=max(1, min(len(jobs) + 1, os.cpu_count() or 4))) as ex:
        module = ex.submit(lambda: run(_ops_compile(ops_obj))) if ops_stale else None
        for msg in ex.map(run, jobs):
            if verbose and msg:
                print(msg)
    if force or jobs or _stale(LIB, objs):
        tmp = LIB + ".tmp%d" % os.getpid()
        run([cc, *ARCH, "-shared", "-o", tmp, *objs, "-Xcompiler", "-fPIC"])
        os.replace(tmp, LIB)
    try:
        if module:
            module.result()
        if ops_stale or _stale(ops, [ops_obj, LIB]):
            tmp = ops + ".tmp%d" % os.getpid()
            run(_ops_link(ops_obj, tmp))
            os.replace(tmp, ops)
    except (OSError, RuntimeError) as e:
        for stale in (ops, ops_obj):        # not a module of other sources beside this library
            if os.path.exists(stale):
                os.remove(stale)
        warnings.warn("the library is built, its Python module is not (the operators but "
                      "kv_append need it): %s" % e, RuntimeWarning, stacklevel=2)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
