"""Builds libcsa2.so (the CUDA library behind include/csa2.h) in-tree with nvcc,
and, apart from it, csa2_torch.so (the Python binding's short calls) with g++.

One nvcc process per translation unit, run in parallel, then one link step;
sm_103a only.  The library needs nothing but CUDA; the module also needs the
headers of PyTorch and Python, and is built for the PyTorch that is installed.
The output goes to sparse_attention_decode_step_gb300/_build/.
"""
from __future__ import annotations

import os
import platform
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OUT_DIR = os.path.join(HERE, "_build")
LIB_PATH = os.path.join(OUT_DIR, "libcsa2.so")
EXT_PATH = os.path.join(OUT_DIR, "csa2_torch.so")
EXT_STAMP = os.path.join(OUT_DIR, "csa2_torch.for")     # what EXT_PATH was built for

SOURCES = ["csa2_api.cu", "csa2_append.cu", "csa2_index.cu", "csa2_topk.cu", "csa2_attn_tc.cu",
           "csa2_rows.cu", "csa2_dense.cu", "csa2_mass.cu", "csa2_evict.cu", "csa2_rope.cu"]
HEADERS = ["csa2_device.cuh", "csa2_attn_device.cuh", "csa2_internal.h"]
EXT_SOURCE = "csa2_torch.cpp"
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-rdc=false", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
              "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC]


def _nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def _fresh(out: str, inputs) -> bool:
    if not os.path.exists(out):
        return False
    t = os.path.getmtime(out)
    return all(os.path.getmtime(f) <= t for f in inputs)


def up_to_date() -> bool:
    files = [os.path.join(CSRC, s) for s in SOURCES + HEADERS]
    return _fresh(LIB_PATH, files + [os.path.join(INCLUDE, "csa2.h"), os.path.abspath(__file__)])


def _ext_stamp() -> str:
    """The PyTorch (its version and C++ ABI), Python and machine that the module is good for."""
    import torch
    return f"torch {torch.__version__} abi {int(torch.compiled_with_cxx11_abi())} {sys.implementation.cache_tag} {platform.machine()}"


def ext_up_to_date() -> bool:
    files = [os.path.join(CSRC, EXT_SOURCE), os.path.join(INCLUDE, "csa2.h"), os.path.abspath(__file__)]
    if not (_fresh(EXT_PATH, files) and os.path.exists(EXT_STAMP)):
        return False
    with open(EXT_STAMP) as f:
        return f.read() == _ext_stamp()


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    if not force and up_to_date():
        return LIB_PATH
    os.makedirs(OUT_DIR, exist_ok=True)
    nvcc = _nvcc()
    extra = ["-Xptxas", "-v"] if ptxas_info else []

    def compile_one(src):
        obj = os.path.join(OUT_DIR, os.path.splitext(src)[0] + ".o")
        cmd = [nvcc, *ARCH, *NVCC_FLAGS, *extra, "-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stderr}")
        return obj, r.stderr

    with ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        results = list(ex.map(compile_one, SOURCES))
    if verbose or ptxas_info:
        for _obj, err in results:
            if err:
                sys.stderr.write(err)
    tmp = LIB_PATH + f".tmp{os.getpid()}"
    cmd = [nvcc, *ARCH, "-shared", "-cudart", "shared", "-o", tmp] + [o for o, _ in results]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc link failed:\n{r.stderr}")
    os.replace(tmp, LIB_PATH)
    return LIB_PATH


def build_ext(force: bool = False) -> str:
    """Builds csa2_torch.so against the installed PyTorch (and the library first, if it is stale)."""
    build()
    if not force and ext_up_to_date():
        return EXT_PATH
    import torch
    torch_dir = os.path.dirname(os.path.abspath(torch.__file__))
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    inc = [INCLUDE, os.path.join(torch_dir, "include"),
           os.path.join(torch_dir, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"], os.path.join(cuda, "include")]
    tmp = EXT_PATH + f".tmp{os.getpid()}"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
           *[f for d in inc for f in ("-I", d)], os.path.join(CSRC, EXT_SOURCE), "-o", tmp,
           "-L", os.path.join(torch_dir, "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python",
           "-L", OUT_DIR, "-l:libcsa2.so", "-Wl,-rpath,$ORIGIN"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on {EXT_SOURCE}:\n{r.stderr}")
    os.replace(tmp, EXT_PATH)
    with open(EXT_STAMP, "w") as f:
        f.write(_ext_stamp())
    return EXT_PATH


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True, ptxas_info="--ptxas" in sys.argv))
