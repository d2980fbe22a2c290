"""Build libcca.so in-tree with nvcc for sm_103a (one -gencode, translation units in parallel), and
the CPython binding of its rotary and paged calls with the host compiler."""
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
LIB = os.path.join(PKG, "libcca.so")
BINDING = os.path.join(PKG, "_binding.so")
BINDING_FOR = os.path.join(BUILD, "binding_for")  # what it was built for
SOURCES = ["cca_api.cu", "pool.cu", "attn_f32.cu", "attn_tc.cu", "decode.cu", "bwd.cu", "bwd_tc.cu", "host_pipeline.cu",
           "rope.cu", "pages.cu", "pool_pages.cu", "tree.cu", "tree_tc.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-I", os.path.join(ROOT, "include")]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def cxx() -> str:
    for cand in (os.environ.get("CXX"), shutil.which("g++"), shutil.which("c++")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("no C++ compiler found")


def _binding_command(out: str) -> list[str]:
    import torch
    base = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    inc = [os.path.join(base, "include"), os.path.join(base, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"], os.path.join(cuda, "include"), os.path.join(ROOT, "include")]
    return [cxx(), "-O2", "-std=c++17", "-fPIC", "-shared", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
            *[x for i in inc for x in ("-I", i)], os.path.join(CSRC, "binding.cpp"), "-o", out,
            "-L", os.path.join(base, "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch", "-ltorch_python"]


def _this_torch() -> str:
    import torch
    return f"torch {torch.__version__}, Python {sys.version.split()[0]}"


def binding_is_for_this_torch() -> bool:
    """Whether the binding is there and was built against the torch and Python that run now."""
    try:
        with open(BINDING_FOR) as f:
            return f.read() == _this_torch() and os.path.exists(BINDING)
    except OSError:
        return False


def _deps_mtime() -> float:
    paths = [os.path.join(CSRC, f) for f in os.listdir(CSRC)] + [os.path.join(ROOT, "include", f)
                                                                  for f in os.listdir(os.path.join(ROOT, "include"))]
    return max(os.path.getmtime(p) for p in paths)


def build(force: bool = False, verbose: bool = False, extra_flags: list[str] | None = None) -> str:
    """Builds what is not up to date.  Where the binding's compiler or torch's headers are missing, the
    library is built all the same (all calls but the rotary and paged ones), and then this raises."""
    def current(path):
        return not force and os.path.exists(path) and os.path.getmtime(path) >= _deps_mtime()

    lib_current, binding_current = current(LIB), current(BINDING) and binding_is_for_this_torch()
    if lib_current and binding_current:
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()
    extra = list(extra_flags or [])

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
        cmd = [cc, *ARCH, *FLAGS, *extra, "-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout, r.stderr)
        return obj

    def compile_binding():
        tmp = BINDING + ".tmp%d" % os.getpid()
        r = subprocess.run(_binding_command(tmp), capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"binding failed:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, BINDING)
        with open(BINDING_FOR, "w") as f:
            f.write(_this_torch())

    with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        binding = None if binding_current else ex.submit(compile_binding)
        if not lib_current:
            objs = list(ex.map(compile_one, SOURCES))
            tmp = LIB + ".tmp%d" % os.getpid()
            r = subprocess.run([cc, *ARCH, "-shared", "-o", tmp, *objs], capture_output=True, text=True)
            if r.returncode != 0:
                raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
            os.replace(tmp, LIB)
        if binding is not None:
            binding.result()
    return LIB


if __name__ == "__main__":
    print(build(force=True, verbose=True, extra_flags=sys.argv[1:]))
