"""Build libbre.so (CUDA, sm_103a) in-tree with nvcc and _kv.so (the Python face of its kv_* calls, a C++ file
against PyTorch's headers) with g++; translation units compile in parallel."""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
OUT_DIR = os.path.join(HERE, "_build")
LIB = os.path.join(OUT_DIR, "libbre.so")
BINDING = os.path.join(OUT_DIR, "_kv.so")
BUILT_FOR = os.path.join(OUT_DIR, "_kv.built_for")   # the PyTorch and Python that BINDING was built against
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
         "-I", os.path.join(ROOT, "include"), "-I", CSRC]


def nvcc() -> str:
    for c in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", shutil.which("nvcc")):
        if c and os.path.exists(c):
            return c
    raise RuntimeError("nvcc not found")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return _sources() + glob.glob(os.path.join(CSRC, "*.cpp")) + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + \
        [os.path.join(ROOT, "include", "bre.h"), __file__]


def _versions() -> str:
    import sysconfig

    import torch
    return f"torch {torch.__version__}, {sysconfig.get_config_var('SOABI')}"


def binding_is_current() -> bool:
    """Whether BINDING is there and was built against the PyTorch and Python that run: against others it may load
    and read tensors wrongly."""
    try:
        with open(BUILT_FOR) as f:
            return os.path.exists(BINDING) and f.read() == _versions()
    except OSError:
        return False


def _compile_binding(obj: str) -> None:
    import sysconfig

    from torch.utils import cpp_extension
    inc = [f"-I{p}" for p in (*cpp_extension.include_paths(), sysconfig.get_paths()["include"],
                              os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include"), os.path.join(ROOT, "include"))]
    import torch
    r = subprocess.run(["g++", "-O2", "-std=c++17", "-fPIC", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
                        *inc, "-c", os.path.join(CSRC, "kv_binding.cpp"), "-o", obj], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on kv_binding.cpp:\n{r.stderr}")


def _link_binding(obj: str) -> None:
    from torch.utils import cpp_extension
    tmp = BINDING + f".{os.getpid()}.tmp"
    libs = [a for p in cpp_extension.library_paths() for a in (f"-L{p}", f"-Wl,-rpath,{p}")]
    r = subprocess.run(["g++", "-shared", "-o", tmp, obj, f"-L{OUT_DIR}", "-l:libbre.so", "-Wl,-rpath,$ORIGIN", *libs,
                        "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda", "-ltorch_python"], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link of _kv.so failed:\n{r.stderr}")
    if os.path.exists(BUILT_FOR):
        os.remove(BUILT_FOR)   # it does not stand beside a binding of another version for a moment
    os.replace(tmp, BINDING)
    with open(BUILT_FOR + f".{os.getpid()}.tmp", "w") as f:
        f.write(_versions())
    os.replace(f.name, BUILT_FOR)


def build(force: bool = False, verbose: bool = False, extra=()) -> str:
    os.makedirs(OUT_DIR, exist_ok=True)
    newest = max(os.path.getmtime(p) for p in _deps())
    if not force and binding_is_current() and all(os.path.exists(f) and os.path.getmtime(f) >= newest for f in (LIB, BINDING)):
        return LIB
    cc = nvcc()
    objs = []

    def compile_one(src):
        obj = os.path.join(OUT_DIR, os.path.basename(src) + ".o")
        cmd = [cc, *ARCH, *FLAGS, *extra, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stderr}")
        if verbose and r.stderr:
            print(r.stderr)
        return obj

    with cf.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 4)) as ex:
        bobj = os.path.join(OUT_DIR, "kv_binding.cpp.o")
        binding = ex.submit(_compile_binding, bobj)
        objs = list(ex.map(compile_one, _sources()))
        binding.result()
    tmp = LIB + f".{os.getpid()}.tmp"
    r = subprocess.run([cc, *ARCH, "-shared", "-o", tmp, *objs, "-lcudart"], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, LIB)
    _link_binding(bobj)
    return LIB


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv,
                extra=["-Xptxas", "-v"] if "--ptxas" in sys.argv else []))
