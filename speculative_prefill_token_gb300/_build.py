"""In-tree build of libspecprefill.so for sm_103a (nvcc, no cmake) and of the
torch side of its paged operators (g++ against torch's headers).

Translation units compile in parallel; both shared objects land next to
this file. Rebuilds only when a source or header is newer than they are, the
torch side also when it was compiled against another torch or Python. Without
torch the library alone is built (for callers of the C ABI).
"""

import os
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libspecprefill.so")
TORCH_LIB = os.path.join(HERE, "_paged_torch.so")
TORCH_SOURCE = "sp_paged_torch.cpp"
TORCH_STAMP = os.path.join(BUILD, "paged_torch.stamp")
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


def _fresh(path) -> bool:
    if not os.path.exists(path):
        return False
    t = os.path.getmtime(path)
    return all(os.path.getmtime(f) <= t for f in _inputs())


def torch_stamp():
    """What the torch side is compiled against (its headers are inlined into
    it), or None without torch."""
    try:
        import torch
    except (ImportError, OSError):
        return None
    return f"torch {torch.__version__} cxx11_abi {int(torch._C._GLIBCXX_USE_CXX11_ABI)} {sysconfig.get_config_var('SOABI')}"


def torch_side_fits() -> bool:
    """Whether the torch side was compiled against the torch and Python here."""
    if not os.path.exists(TORCH_LIB) or not os.path.exists(TORCH_STAMP):
        return False
    with open(TORCH_STAMP) as f:
        return f.read() == torch_stamp()


def torch_side_up_to_date() -> bool:
    # (without torch there is nothing to build it against)
    return torch_stamp() is None or (_fresh(TORCH_LIB) and torch_side_fits())


def up_to_date() -> bool:
    return _fresh(LIB) and torch_side_up_to_date()


def _run(cmd, verbose, what):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if verbose or r.returncode != 0:
        sys.stderr.write(" ".join(cmd) + "\n" + r.stdout + r.stderr)
    if r.returncode != 0:
        raise RuntimeError(f"{os.path.basename(cmd[0])} failed on {what}")


def _compile_torch_side(nvcc, verbose):
    import torch
    root = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(nvcc)) if os.path.isabs(nvcc) else "/usr/local/cuda"
    obj = os.path.join(BUILD, TORCH_SOURCE.replace(".cpp", ".o"))
    _run(["g++", "-O2", "-std=c++17", "-fPIC", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
          "-I", INCLUDE, "-I", os.path.join(root, "include"),
          "-I", os.path.join(root, "include", "torch", "csrc", "api", "include"),
          "-I", sysconfig.get_paths()["include"], "-I", os.path.join(cuda, "include"),
          "-c", os.path.join(CSRC, TORCH_SOURCE), "-o", obj], verbose, TORCH_SOURCE)
    return obj, os.path.join(root, "lib")


def _link_torch_side(obj, torch_libs, verbose):
    # (the library is found beside it, torch's libraries are loaded already)
    tmp = TORCH_LIB + ".tmp"
    _run(["g++", "-shared", "-o", tmp, obj, "-L", HERE, "-l:libspecprefill.so", "-L", torch_libs, "-ltorch_python",
          "-ltorch_cpu", "-lc10", "-lc10_cuda", "-Wl,-rpath,$ORIGIN"], verbose, "the link of the torch side")
    os.replace(tmp, TORCH_LIB)
    with open(TORCH_STAMP, "w") as f:
        f.write(torch_stamp())


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    os.makedirs(BUILD, exist_ok=True)
    nvcc = _nvcc()
    with_library = force or not _fresh(LIB)
    with_torch_side = torch_stamp() is not None and (force or with_library or not torch_side_up_to_date())

    def compile_one(src):
        obj = os.path.join(BUILD, src.replace(".cu", ".o"))
        _run([nvcc, *ARCH, *FLAGS, *extra_flags, "-c", os.path.join(CSRC, src), "-o", obj], verbose, src)
        return obj

    with ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        torch_side = ex.submit(_compile_torch_side, nvcc, verbose) if with_torch_side else None
        objs = list(ex.map(compile_one, SOURCES)) if with_library else []
        if with_library:
            # the library is in place also when the torch side fails
            tmp = LIB + ".tmp"
            _run([nvcc, *ARCH, "-shared", "-o", tmp, *objs], False, "the link")
            os.replace(tmp, LIB)
        if with_torch_side:
            _link_torch_side(*torch_side.result(), verbose)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
