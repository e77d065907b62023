"""Build the codec's CUDA library in-tree: error_bounded_lossy_gb300/_build/libebc_gb300.so.

nvcc compiles each translation unit for sm_103a in parallel, then links one
shared library with the CUDA runtime statically linked.  No torch types cross
the C ABI, so the library is loaded with ctypes.  A second, small module
(_build/_torch_calls-<torch version>-<python ABI>.so, g++ against torch's headers) makes the
expert-parallel and 4-bit calls on torch tensors; it links the first, and is
left out where torch is not installed.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(BUILD, "libebc_gb300.so")
SOURCES = ["ebc_api.cu", "ebc_compress.cu", "ebc_decompress.cu", "ebc_experts.cu", "ebc_mx4.cu",
           "ebc_mx4_product.cu", "ebc_mx8.cu", "ebc_mx8_product.cu", "ebc_norm.cu", "ebc_route.cu"]
HEADERS = ["ebc_internal.cuh", "ebc_types.cuh", "ebc_mx4.cuh", "ebc_mx8.cuh", "ebc_mx_product.cuh", os.path.join("..", "..", "include", "ebc.h")]

TORCH_SOURCE = "ebc_torch.cpp"

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-ffp-contract=off,-O2",
              "--expt-relaxed-constexpr", "-Wno-deprecated-gpu-targets"]


def nvcc() -> str:
    path = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(path):
        raise RuntimeError("nvcc not found: the codec needs the CUDA toolkit to build")
    return path


def torch_module() -> str:
    """The path of the torch module, one for each torch and Python it may be built against."""
    import torch
    return os.path.join(BUILD, f"_torch_calls-{torch.__version__}-{sysconfig.get_config_var('SOABI')}.so")


def _torch_commands(obj: str, out: str):
    """(compile, link) of the torch module."""
    import torch
    root = os.path.dirname(torch.__file__)
    cuda = os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")
    inc = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"), cuda,
           sysconfig.get_paths()["include"]]
    libs = os.path.join(root, "lib")
    return (["g++", "-O2", "-std=c++17", "-fPIC", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
             *(f"-I{i}" for i in inc), "-c", os.path.join(CSRC, TORCH_SOURCE), "-o", obj],
            ["g++", "-shared", "-o", out, obj, f"-L{libs}", "-ltorch_python", "-ltorch_cuda", "-ltorch_cpu", "-ltorch",
             "-lc10_cuda", "-lc10", f"-L{BUILD}", "-l:" + os.path.basename(LIB), f"-Wl,-rpath,{libs}",
             "-Wl,-rpath,$ORIGIN"])


def _stale(out: str, deps) -> bool:
    if not os.path.exists(out):
        return True
    t = os.path.getmtime(out)
    return any(os.path.getmtime(d) > t for d in deps)


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    deps_common = [os.path.join(CSRC, h) for h in HEADERS] + [os.path.abspath(__file__)]
    jobs = []
    for src in SOURCES:
        s = os.path.join(CSRC, src)
        o = os.path.join(BUILD, src.replace(".cu", ".o"))
        if force or ptxas_info or _stale(o, [s] + deps_common):
            cmd = [nvcc(), *ARCH, *NVCC_FLAGS, "-c", s, "-o", o]
            if ptxas_info:
                cmd += ["-Xptxas", "-v"]
            jobs.append(cmd)

    def run(cmd):
        r = subprocess.run(cmd, capture_output=True, text=True)
        return cmd, r

    module = None
    with ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        running = [ex.submit(run, cmd) for cmd in jobs]
        try:
            module = torch_module()   # (imports torch, while nvcc is at work)
        except ImportError:
            pass
        if module:
            module_obj = module[:-3] + ".o"
            torch_deps = [os.path.join(CSRC, TORCH_SOURCE), os.path.join(CSRC, HEADERS[-1]), os.path.abspath(__file__)]
            compile_torch, link_torch = _torch_commands(module_obj, module + f".{os.getpid()}.tmp")
            if force or _stale(module_obj, torch_deps):
                running.append(ex.submit(run, compile_torch))
        for cmd, r in (f.result() for f in running):
            if verbose or ptxas_info or r.returncode != 0:
                sys.stderr.write(r.stdout + r.stderr)
            if r.returncode != 0:
                raise RuntimeError("compilation failed: " + " ".join(cmd))
    objs = [os.path.join(BUILD, s.replace(".cu", ".o")) for s in SOURCES]
    if force or jobs or _stale(LIB, objs):
        tmp = LIB + f".{os.getpid()}.tmp"
        cmd = [nvcc(), *ARCH, "-shared", "-Xcompiler", "-fPIC", "-o", tmp, *objs]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            sys.stderr.write(r.stdout + r.stderr)
            raise RuntimeError("nvcc link failed")
        os.replace(tmp, LIB)
    if module and (force or _stale(module, [module_obj])):
        r = subprocess.run(link_torch, capture_output=True, text=True)
        if r.returncode != 0:
            sys.stderr.write(r.stdout + r.stderr)
            raise RuntimeError("linking the torch module failed")
        os.replace(link_torch[3], module)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True, ptxas_info="--ptxas" in sys.argv)
    print(LIB)
