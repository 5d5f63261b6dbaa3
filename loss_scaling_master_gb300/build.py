"""Build libampfp8.so (the CUDA kernels + C ABI) in-tree for sm_103a.

    python -m loss_scaling_master_gb300.build

Each .cu file is compiled in parallel with nvcc, then linked into one shared
library next to this file; the operators' Python argument marshalling
(``csrc/ops_bind.cpp``) is compiled beside them with g++ into ``_ops_bind.so``.
Objects go to ``_build/`` (git-ignored), and with them a stamp of what
``_ops_bind.so`` was compiled for: it reads torch's tensors through torch's own
inline accessors, so another torch or Python needs another one.
"""
from __future__ import annotations

import importlib.metadata
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libampfp8.so")
BIND_SRC = os.path.join(CSRC, "ops_bind.cpp")
BIND = os.path.join(PKG, "_ops_bind.so")
BIND_STAMP = os.path.join(BUILD, "ops_bind.stamp")
SOURCES = ["api.cu", "unscale_check.cu", "adamw_master.cu", "adamw_noalloc.cu", "emit_bf16.cu",
           "fp8_quant.cu",
           "fp8_rowwise.cu", "fp8_groupwise.cu", "update_scale.cu",
           "ops_api.cu", "fp4_mx.cu", "fp4_product.cu", "layer_norm_fwd.cu", "layer_norm_bwd.cu",
           "act_mx8.cu", "fp4_linear.cu", "fp4_linear_pair.cu", "bias_grad.cu", "dropout.cu", "token_logprobs.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
# --fmad=false: no multiply-add is fused behind the code's back; the kernels
# spell out the rounding of every operation.  IEEE division and square root
# (the defaults) stay on; no fast-math.
FLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "--fmad=false", "-Xcompiler", "-fPIC,-O2",
                "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA 13 toolkit is required to build libampfp8")


def _bind_command(target: str):
    """g++ on the operators' argument marshalling, a Python extension against torch's headers
    (found without importing torch)."""
    torch = importlib.util.find_spec("torch").submodule_search_locations[0]
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    return ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-DNDEBUG",
            "-I", sysconfig.get_paths()["include"], "-I", INCLUDE,
            "-isystem", os.path.join(torch, "include"),
            "-isystem", os.path.join(torch, "include", "torch", "csrc", "api", "include"),
            "-isystem", os.path.join(cuda, "include"), BIND_SRC, "-o", target,
            "-L", os.path.join(torch, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10_cuda", "-lc10"]


def _bind_stamp() -> str:
    """What _ops_bind.so depends on besides its sources: torch, Python and the command."""
    return "\n".join([importlib.metadata.version("torch"), sysconfig.get_config_var("SOABI") or sys.version,
                      *_bind_command(BIND)])


def _bind_stale(deps) -> bool:
    try:
        with open(BIND_STAMP) as f:
            same = f.read() == _bind_stamp()
    except OSError:
        same = False
    return not same or _stale(BIND, deps)


def _stale(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    headers = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".h", ".cuh"))]
    headers += [os.path.join(INCLUDE, f) for f in ("ampfp8.h", "ampops.h")]
    cc = nvcc()
    procs, objs = [], []
    for src in SOURCES:
        s = os.path.join(CSRC, src)
        o = os.path.join(BUILD, src.replace(".cu", ".o"))
        objs.append(o)
        if force or _stale(o, [s] + headers):
            cmd = [cc] + FLAGS + (["-Xptxas", "-v"] if ptxas_info else []) + ["-c", s, "-o", o]
            if verbose:
                print(" ".join(cmd), flush=True)
            procs.append((src, subprocess.Popen(cmd, stdout=subprocess.PIPE,
                                                stderr=subprocess.STDOUT, text=True)))
    bind_tmp = BIND + f".tmp{os.getpid()}"
    bind = None
    if force or _bind_stale([BIND_SRC] + headers):
        cmd = _bind_command(bind_tmp)
        if verbose:
            print(" ".join(cmd), flush=True)
        bind = subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    failed = []
    for src, p in procs + ([("ops_bind.cpp", bind)] if bind else []):
        out, _ = p.communicate()
        if verbose or ptxas_info or p.returncode:
            sys.stdout.write(out)
        if p.returncode:
            failed.append(src)
    if failed:
        raise RuntimeError(f"compilation failed for {failed}")
    if bind:
        os.replace(bind_tmp, BIND)
        with open(bind_tmp + ".stamp", "w") as f:
            f.write(_bind_stamp())
        os.replace(bind_tmp + ".stamp", BIND_STAMP)
    if force or procs or _stale(LIB, objs):
        tmp = LIB + f".tmp{os.getpid()}"
        cmd = [cc] + ARCH + ["-shared", "-o", tmp] + objs + ["-cudart", "static"]
        if verbose:
            print(" ".join(cmd), flush=True)
        subprocess.check_call(cmd)
        os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True, ptxas_info="--ptxas" in sys.argv))
