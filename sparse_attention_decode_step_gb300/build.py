"""Builds libcsa2.so (the CUDA library behind include/csa2.h) in-tree with nvcc,
and csa2_torch.so (the Python binding's short calls) with g++.

One compiler process per translation unit, run in parallel, then a link step
each; sm_103a only.  The output goes to sparse_attention_decode_step_gb300/_build/.
"""
from __future__ import annotations

import importlib.util
import os
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

SOURCES = ["csa2_api.cu", "csa2_append.cu", "csa2_index.cu", "csa2_topk.cu", "csa2_attn_tc.cu",
           "csa2_rows.cu", "csa2_dense.cu"]
HEADERS = ["csa2_device.cuh", "csa2_attn_device.cuh", "csa2_internal.h"]
EXT_SOURCE = "csa2_torch.cpp"
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-rdc=false", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
              "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC]


def _nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def _torch_dir() -> str:
    return importlib.util.find_spec("torch").submodule_search_locations[0]


def _inputs():
    files = [os.path.join(CSRC, s) for s in SOURCES + HEADERS + [EXT_SOURCE]]
    files.append(os.path.join(_torch_dir(), "version.py"))     # (the binding is built against this PyTorch)
    files.append(os.path.join(INCLUDE, "csa2.h"))
    files.append(os.path.abspath(__file__))
    return files


def up_to_date() -> bool:
    if not (os.path.exists(LIB_PATH) and os.path.exists(EXT_PATH)):
        return False
    t = min(os.path.getmtime(LIB_PATH), os.path.getmtime(EXT_PATH))
    return all(os.path.getmtime(f) <= t for f in _inputs())


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

    torch_dir = _torch_dir()
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    ext_obj = os.path.join(OUT_DIR, "csa2_torch.o")

    def compile_ext():
        inc = [INCLUDE, os.path.join(torch_dir, "include"),
               os.path.join(torch_dir, "include", "torch", "csrc", "api", "include"),
               sysconfig.get_paths()["include"], os.path.join(cuda, "include")]
        cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-D_GLIBCXX_USE_CXX11_ABI=1",
               *[f for d in inc for f in ("-I", d)], "-c", os.path.join(CSRC, EXT_SOURCE), "-o", ext_obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"g++ failed on {EXT_SOURCE}:\n{r.stderr}")

    with ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        ext = ex.submit(compile_ext)
        results = list(ex.map(compile_one, SOURCES))
        ext.result()
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
    tmp = EXT_PATH + f".tmp{os.getpid()}"
    cmd = ["g++", "-shared", "-o", tmp, ext_obj, "-L", os.path.join(torch_dir, "lib"), "-lc10", "-lc10_cuda",
           "-ltorch_cpu", "-ltorch_python", "-L", OUT_DIR, "-l:libcsa2.so", "-Wl,-rpath,$ORIGIN"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ link failed:\n{r.stderr}")
    os.replace(tmp, EXT_PATH)
    return LIB_PATH


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True, ptxas_info="--ptxas" in sys.argv))
