"""In-tree build of libspecprefill.so for sm_103a (nvcc, no cmake) and of the
torch side of its paged operators (g++ against torch's headers).

Translation units compile in parallel; both shared objects land next to
this file. Rebuilds only when a source or header is newer than they are.
"""

import os
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libspecprefill.so")
TORCH_LIB = os.path.join(HERE, "_paged_torch.so")
TORCH_SOURCE = "sp_paged_torch.cpp"
SOURCES = ["sp_api.cu", "sp_stages.cu", "sp_logits_tc.cu", "sp_logits_simt.cu", "sp_noalloc.cu", "sp_post.cu",
           "sp_rows.cu", "sp_head_pool.cu", "sp_cache.cu", "sp_attn.cu", "sp_paged_api.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-I", INCLUDE, "-I", CSRC]


def _nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def _inputs():
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    files += [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE)]
    files.append(os.path.abspath(__file__))  # a changed source list rebuilds too
    return files


def up_to_date() -> bool:
    if not os.path.exists(LIB) or not os.path.exists(TORCH_LIB):
        return False
    t = min(os.path.getmtime(LIB), os.path.getmtime(TORCH_LIB))
    return all(os.path.getmtime(f) <= t for f in _inputs())


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    if not force and up_to_date():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    nvcc = _nvcc()

    def compile_one(src):
        obj = os.path.join(BUILD, src.replace(".cu", ".o"))
        cmd = [nvcc, *ARCH, *FLAGS, *extra_flags, "-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if verbose or r.returncode != 0:
            sys.stderr.write(" ".join(cmd) + "\n" + r.stdout + r.stderr)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}")
        return obj

    def compile_torch_side():
        import sysconfig

        import torch
        root = os.path.dirname(torch.__file__)
        cuda = os.path.dirname(os.path.dirname(nvcc)) if os.path.isabs(nvcc) else "/usr/local/cuda"
        obj = os.path.join(BUILD, TORCH_SOURCE.replace(".cpp", ".o"))
        cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-I", INCLUDE, "-I", os.path.join(root, "include"),
               "-I", os.path.join(root, "include", "torch", "csrc", "api", "include"),
               "-I", sysconfig.get_paths()["include"], "-I", os.path.join(cuda, "include"),
               "-c", os.path.join(CSRC, TORCH_SOURCE), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if verbose or r.returncode != 0:
            sys.stderr.write(" ".join(cmd) + "\n" + r.stdout + r.stderr)
        if r.returncode != 0:
            raise RuntimeError(f"g++ failed on {TORCH_SOURCE}")
        return obj, os.path.join(root, "lib")

    with ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        torch_side = ex.submit(compile_torch_side)
        objs = list(ex.map(compile_one, SOURCES))
        torch_obj, torch_libs = torch_side.result()
    tmp = LIB + ".tmp"
    cmd = [nvcc, *ARCH, "-shared", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(" ".join(cmd) + "\n" + r.stdout + r.stderr)
        raise RuntimeError("link failed")
    os.replace(tmp, LIB)
    # (the library is found beside it, torch's libraries are loaded already)
    tmp = TORCH_LIB + ".tmp"
    cmd = ["g++", "-shared", "-o", tmp, torch_obj, "-L", HERE, "-l:libspecprefill.so", "-L", torch_libs, "-ltorch_python", "-ltorch_cpu", "-lc10",
           "-lc10_cuda", "-Wl,-rpath,$ORIGIN"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(" ".join(cmd) + "\n" + r.stdout + r.stderr)
        raise RuntimeError("link of the torch side failed")
    os.replace(tmp, TORCH_LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
