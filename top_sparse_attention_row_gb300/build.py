"""Builds libqsa.so (the C-ABI library) in-tree with nvcc for sm_103a, and the Python extension
_serving (argument checks of the serving-step calls, csrc/torch_serving.cpp) with the host compiler.
The library needs nvcc alone; where PyTorch is not installed, the extension is left out.

Usage: ``python -m top_sparse_attention_row_gb300.build`` or ``build()`` from Python.
Translation units compile in parallel; objects go to ``_build/`` next to this file.
"""
from __future__ import annotations

import concurrent.futures as cf
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig
from typing import Optional

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libqsa.so")
SOURCES = ["prefill.cu", "mla.cu", "union.cu", "api.cpp", "noalloc.cu", "probe.cu", "pages.cu",
           "serving.cpp", "plan.cu", "rope.cu", "window.cu", "window_d64.cu", "window_d128.cu",
           "window_d256.cu", "listed.cu", "listed_d64.cu", "listed_d128.cu",
           "listed_d256.cu", "bounds.cu", "score.cu",
           "select_d64.cu", "select_d128.cu", "select_d256.cu"]

EXT_SOURCE = "torch_serving.cpp"
EXT = os.path.join(PKG, "_serving" + (sysconfig.get_config_var("EXT_SUFFIX") or ".so"))

EXT_STAMP = os.path.join(BUILD, "_serving.made_for")       # beside the objects: what EXT was built against

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
COMMON = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-I", os.path.join(ROOT, "include")]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def torch_root() -> Optional[str]:
    """PyTorch's folder, or None where it is not installed."""
    try:
        spec = importlib.util.find_spec("torch")
    except (ImportError, ValueError):
        return None
    return os.path.dirname(spec.origin) if spec is not None and spec.origin else None


def _made_for(root: str) -> str:
    """What an extension is compiled against beside the sources: PyTorch's place and version, and the interpreter."""
    with open(os.path.join(root, "version.py")) as f:
        return f"{root}\n{f.read()}\n{sys.version}\n{sysconfig.get_config_var('EXT_SUFFIX')}\n"


def _extension_is_for(root: str) -> bool:
    try:
        with open(EXT_STAMP) as f:
            return f.read() == _made_for(root)
    except OSError:
        return False


def _compile(nvcc: str, src: str, verbose_ptxas: bool) -> str:
    obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
    cmd = [nvcc, *ARCH, *COMMON, "-c", os.path.join(CSRC, src), "-o", obj]
    if verbose_ptxas and src.endswith(".cu"):
        cmd += ["-Xptxas", "-v"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
    if verbose_ptxas and r.stderr:
        sys.stderr.write(r.stderr)
    return obj


def _compile_extension() -> str:
    """The extension's object file; it is linked against libqsa.so once that is there."""
    import torch
    inc = os.path.join(os.path.dirname(torch.__file__), "include")
    cuda = os.path.dirname(os.path.dirname(_nvcc()))
    obj = os.path.join(BUILD, "torch_serving.o")
    abi = int(getattr(torch._C, "_GLIBCXX_USE_CXX11_ABI", True))
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", f"-D_GLIBCXX_USE_CXX11_ABI={abi}",
           "-isystem", inc, "-isystem", os.path.join(inc, "torch", "csrc", "api", "include"),
           "-isystem", sysconfig.get_paths()["include"], "-isystem", os.path.join(cuda, "include"),
           "-I", os.path.join(ROOT, "include"), "-c", os.path.join(CSRC, EXT_SOURCE), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{cmd[0]} failed on {EXT_SOURCE}:\n{r.stdout}\n{r.stderr}")
    return obj


def _link_extension(obj: str):
    import torch
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = EXT + ".tmp"
    cmd = [os.environ.get("CXX", "g++"), "-shared", "-o", tmp, obj, "-L", PKG, "-lqsa", "-L", lib, "-ltorch_python",
           "-ltorch_cpu", "-lc10_cuda", "-lc10", "-Wl,-rpath,$ORIGIN"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link of {os.path.basename(EXT)} failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, EXT)


def build(verbose_ptxas: bool = False, force: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    srcs = [os.path.join(CSRC, s) for s in SOURCES + [EXT_SOURCE]] + [
        os.path.join(CSRC, h) for h in os.listdir(CSRC) if h.endswith((".h", ".cuh"))
    ] + [os.path.join(ROOT, "include", "qsa.h")]
    newest = max(os.path.getmtime(s) for s in srcs)
    root = torch_root()
    with_ext = root is not None
    targets = (LIB, EXT) if with_ext else (LIB,)
    current = all(os.path.exists(f) and os.path.getmtime(f) >= newest for f in targets)
    if not force and current and (not with_ext or _extension_is_for(root)):
        return LIB
    nvcc = _nvcc()
    with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        ext_obj = ex.submit(_compile_extension) if with_ext else None
        objs = list(ex.map(lambda s: _compile(nvcc, s, verbose_ptxas), SOURCES))
    tmp = LIB + ".tmp"
    cmd = [nvcc, *ARCH, "-shared", "-o", tmp, *objs, "-lrt", "-ldl", "-lpthread"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    if ext_obj is None:
        sys.stderr.write("PyTorch is not installed: the _serving extension (binding.py's serving-step calls) is not built\n")
    else:
        _link_extension(ext_obj.result())
        with open(EXT_STAMP, "w") as f:
            f.write(_made_for(root))
    return LIB


if __name__ == "__main__":
    print(build(verbose_ptxas="-v" in sys.argv, force="-f" in sys.argv))
