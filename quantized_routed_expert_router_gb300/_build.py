"""Build the CUDA library (_moe.so) in-tree for sm_103a with nvcc, and the
torch binding of the calls around the experts (_calls.so) with g++.

Translation units compile in parallel; the link step produces one shared
object exporting the C ABI of include/moe.h.  _calls.so is a Python extension
that links against it; it holds for the torch and the Python that it was
compiled against, which it names (built_for), as does a stamp beside the objects
for the next build.  _moe.so needs neither and is in place before the binding is
linked.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import subprocess
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OUT_DIR = os.path.join(PKG, "_build")
SO = os.path.join(PKG, "_moe.so")
CALLS_SO = os.path.join(PKG, "_calls.so")
SOURCES = ["moe_api.cu", "moe_kernels.cu", "moe_ffn.cu", "moe_noalloc.cu", "moe_fused_api.cu",
           "moe_fused_q4k.cu", "moe_fused_q2k.cu", "moe_fused_q80.cu", "moe_fused_mx4.cu", "moe_fused_q6k.cu",
           "moe_fused_q3k.cu", "moe_norm.cu", "moe_router_stats.cu", "moe_topk.cu", "moe_rows.cu", "moe_fp8.cu",
           "moe_fp8_rows.cu", "moe_matmul.cu", "moe_matmul_rows.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def _nvcc() -> str:
    for c in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if c and (os.path.sep not in c or os.path.exists(c)):
            return c
    return "nvcc"


BINDING = "binding.cpp"


def _current(so: str, files: list[str]) -> bool:
    if not os.path.exists(so):
        return False
    t = os.path.getmtime(so)
    return all(os.path.getmtime(f) <= t for f in files)


def lib_up_to_date() -> bool:
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f != BINDING]
    return _current(SO, [*files, os.path.join(INCLUDE, "moe.h")])


def calls_stamp() -> str:
    """What the binding is compiled against: torch and its C++ ABI, and Python's."""
    import torch
    return (f"torch {torch.__version__}, cxx11 abi {int(torch._C._GLIBCXX_USE_CXX11_ABI)}, "
            f"{sysconfig.get_config_var('SOABI')}")


def _stamp_file() -> str:
    return os.path.join(OUT_DIR, "calls.stamp")


def built_calls_stamp() -> str | None:
    """calls_stamp() of the binding that is there."""
    try:
        with open(_stamp_file()) as f:
            return f.read()
    except FileNotFoundError:
        return None


def calls_up_to_date() -> bool:
    files = [os.path.join(CSRC, BINDING), os.path.join(INCLUDE, "moe.h")]
    return _current(CALLS_SO, files) and built_calls_stamp() == calls_stamp()


def up_to_date() -> bool:
    return lib_up_to_date() and calls_up_to_date()


def _compile_binding() -> str:
    """binding.cpp against torch's headers; a host object, no CUDA code"""
    import torch
    root = os.path.dirname(torch.__file__)
    inc = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"], os.path.join(os.path.dirname(os.path.dirname(_nvcc())), "include"), INCLUDE]
    obj = os.path.join(OUT_DIR, "binding.o")
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           f'-DCALLS_STAMP="{calls_stamp()}"',
           *(f"-I{p}" for p in inc), "-c", os.path.join(CSRC, BINDING), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for binding.cpp:\n{r.stderr}")
    return obj


def _link_binding(obj: str) -> None:
    import torch
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = CALLS_SO + f".tmp{os.getpid()}"
    cmd = ["g++", "-shared", "-o", tmp, obj, SO, f"-L{lib}", "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10",
           "-lc10_cuda", "-Wl,-rpath,$ORIGIN"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link of the binding failed:\n{r.stderr}")
    if os.path.exists(_stamp_file()):
        os.remove(_stamp_file())
    os.replace(tmp, CALLS_SO)
    with open(_stamp_file(), "w") as f:
        f.write(calls_stamp())


def build(force: bool = False, verbose: bool = False, extra: list[str] | None = None) -> str:
    if not force and up_to_date():
        return SO
    os.makedirs(OUT_DIR, exist_ok=True)
    nvcc = _nvcc()
    flags = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I", INCLUDE,
                    "--expt-relaxed-constexpr"] + (extra or [])

    def compile_one(src):
        obj = os.path.join(OUT_DIR, src.replace(".cu", ".o"))
        cmd = [nvcc, *flags, "-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stderr}")
        if verbose and r.stderr:
            print(r.stderr)
        return obj

    with cf.ThreadPoolExecutor(len(SOURCES) + 1) as ex:
        binding = ex.submit(_compile_binding) if force or not calls_up_to_date() else None
        if force or not lib_up_to_date():
            objs = list(ex.map(compile_one, SOURCES))
            tmp = SO + f".tmp{os.getpid()}"
            cmd = [nvcc, *ARCH, "-shared", "-Xlinker", "-soname,_moe.so", "-o", tmp, *objs, "-lcudart"]
            r = subprocess.run(cmd, capture_output=True, text=True)
            if r.returncode != 0:
                raise RuntimeError(f"link failed:\n{r.stderr}")
            os.replace(tmp, SO)
        if binding:
            try:
                _link_binding(binding.result())
            except Exception as e:
                raise RuntimeError(f"{SO} is built; the binding of the calls around the experts ({CALLS_SO}) is not: "
                                   f"{e}") from e
    return SO


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose=True,
                extra=["-Xptxas", "-v"] if "--ptxas" in sys.argv else None))
