"""Builds the CUDA library ``libfg.so`` in-tree for sm_103a with nvcc, and beside it, where torch is installed,
``fg_bind.so``, the Python module of the calls whose marshalling has to be short.  The library needs nvcc only; a
module that does not compile (no Python headers, no g++) is a warning.

The translation units compile in parallel; ``-Xptxas -v`` output goes to
``_build/ptxas.log`` and the build fails if any kernel spills registers or uses local
memory."""
from __future__ import annotations

import hashlib
import importlib.util
import os
import re
import shutil
import subprocess
import sysconfig
import warnings
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libfg.so")
SOURCES = ["fg_api.cu", "fg_gemm_nt.cu", "fg_gemm_split.cu", "fg_gemm_tn.cu", "fg_gemm_layouts.cu",
           "fg_gemm_sepc.cu", "fg_gemm_dense.cu", "fg_gemm_swiglu.cu", "fg_gemm_fp4.cu", "fg_gemm_fp4_grouped.cu",
           "fg_mqa.cu", "fg_quant.cu", "fg_moe.cu", "fg_lora.cu", "fg_route.cu",
           "fg_pages.cu", "fg_rope.cu", "fg_kv.cu", "fg_attn.cu", "fg_attn_prompt.cu", "fg_call.cu"]
BIND = os.path.join(HERE, "fg_bind.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def _nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _flags() -> list[str]:
    return ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
                   "-I", os.path.join(ROOT, "include"), "-I", CSRC]


def _stale(target: str) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    deps = [os.path.join(CSRC, f) for f in os.listdir(CSRC)] + [os.path.join(ROOT, "include", "fg.h"),
                                                                 os.path.abspath(__file__)]
    return any(os.path.getmtime(f) > t for f in deps)


def _torch() -> str | None:
    """The directory of the installed torch."""
    spec = importlib.util.find_spec("torch")
    return spec.submodule_search_locations[0] if spec and spec.submodule_search_locations else None


def bind_abi() -> str | None:
    """What fg_bind.so is built for, as its docstring says: torch's version file and Python's binary interface."""
    torch = _torch()
    if torch is None:
        return None
    with open(os.path.join(torch, "version.py"), "rb") as f:
        text = f.read()
    return "fg_bind for " + hashlib.sha1(text + str(sysconfig.get_config_var("SOABI")).encode()).hexdigest()


def bind_fits() -> bool:
    """Whether the fg_bind.so that is there was built for the torch and the Python that are there now."""
    abi = bind_abi()
    if abi is None or not os.path.exists(BIND):
        return False
    with open(BIND, "rb") as f:
        return abi.encode() in f.read()


def _compile(src: str) -> tuple[str, str]:
    obj = os.path.join(BUILD, src.replace(".cu", ".o"))
    cmd = [_nvcc()] + _flags() + ["-Xptxas", "-v", "-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{r.stderr[-4000:]}")
    return obj, r.stderr


def _compile_bind() -> str:
    obj = os.path.join(BUILD, "fg_bind.o")
    torch = _torch()
    include = [sysconfig.get_paths()["include"], os.path.join(torch, "include"), os.path.join(torch, "include/torch/csrc/api/include"),
               os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(_nvcc()))), "include")]
    cmd = [shutil.which("g++") or "g++", "-O2", "-std=c++17", "-fPIC", "-I", os.path.join(ROOT, "include"),
           f'-DFG_BIND_ABI="{bind_abi()}"']
    cmd += [x for path in include for x in ("-isystem", path)] + ["-c", os.path.join(CSRC, "fg_bind.cpp"), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for fg_bind.cpp:\n{r.stderr[-4000:]}")
    return obj


def _link_bind(obj: str) -> None:
    torch = os.path.join(_torch(), "lib")
    cmd = [shutil.which("g++") or "g++", "-shared", obj, "-o", BIND + ".tmp", "-L", HERE, "-l:libfg.so", "-L", torch, "-ltorch_python",
           "-ltorch_cpu", "-lc10", "-lc10_cuda", "-Wl,-rpath,$ORIGIN"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link of fg_bind.so failed:\n{r.stderr[-4000:]}")
    os.replace(BIND + ".tmp", BIND)


def check_ptxas(log: str) -> None:
    bad = []
    for m in re.finditer(r"(\d+) bytes stack frame, (\d+) bytes spill stores, (\d+) bytes spill loads", log):
        if any(int(x) for x in m.groups()):
            bad.append(m.group(0))
    if bad:
        raise RuntimeError("register spills / local memory in kernels: " + "; ".join(bad))


def _link(objs: list[str]) -> None:
    tmp = LIB + ".tmp"
    cmd = [_nvcc()] + ARCH + ["-shared", "-o", tmp] + objs
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr[-4000:]}")
    os.replace(tmp, LIB)


def build(force: bool = False, verbose: bool = False) -> str:
    lib = force or _stale(LIB)
    bind = _torch() is not None and (force or _stale(BIND) or not bind_fits())
    os.makedirs(BUILD, exist_ok=True)
    with ThreadPoolExecutor(len(SOURCES) + 1) as ex:
        bind_obj = ex.submit(_compile_bind) if bind else None
        results = list(ex.map(_compile, SOURCES)) if lib else []
    if lib:
        log = "\n".join(r[1] for r in results)
        with open(os.path.join(BUILD, "ptxas.log"), "w") as f:
            f.write(log)
        check_ptxas(log)
        _link([r[0] for r in results])
        if verbose:
            print(log)
    if bind:
        try:
            _link_bind(bind_obj.result())
        except (RuntimeError, OSError) as e:
            if os.path.exists(BIND):                        # of other sources
                os.remove(BIND)
            warnings.warn(f"fg_bind.so is not built: {e}", RuntimeWarning, stacklevel=2)
    return LIB


if __name__ == "__main__":
    build(force=True, verbose=True)
