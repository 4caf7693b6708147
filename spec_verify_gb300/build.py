"""Builds libsmp.so in-tree with nvcc for sm_103a.

    python -m spec_verify_gb300.build          # incremental
    python -m spec_verify_gb300.build --force  # from scratch

Translation units compile in parallel; the library links the CUDA runtime
statically, so it loads next to any PyTorch build.  The native marshalling of
the cached step (csrc/step_binding.cpp) is a separate extension module, built
against the PyTorch that is installed; a machine without what that takes gets
libsmp.so alone.
"""

import argparse
import concurrent.futures
import importlib.util
import os
import re
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(BUILD, "libsmp.so")
STEP_SOURCE = os.path.join(CSRC, "step_binding.cpp")
STEP_LIB = os.path.join(BUILD, "smp_step_binding.so")

SOURCES = ["api.cu", "sample.cu", "verify.cu", "prepass.cu", "beam.cu", "verify_probs.cu", "block_plan.cu",
           "norm_rope.cu", "cache_append.cu", "cache_attention.cu", "attention_e4m3_bf16.cu",
           "attention_e4m3_f32.cu", "attention_i8_bf16.cu", "attention_i8_f32.cu", "token_logprobs.cu", "distill.cu"]
HEADERS = ["common.cuh", "row_ops.cuh", "select.cuh", "general.cuh", "launch.h", "exp_table.h", "tma.cuh", "general_bf16.cuh",
           "cache.cuh", "cache_attention.cuh", "attention_rows.h", "scores.cuh", "row_grad.cuh"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
         "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC]


def nvcc():
    exe = shutil.which("nvcc")
    if exe is None:
        cand = "/usr/local/cuda/bin/nvcc"
        if os.path.exists(cand):
            exe = cand
    if exe is None:
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libsmp")
    return exe


def _newest_input():
    paths = [os.path.join(CSRC, f) for f in SOURCES + HEADERS]
    paths += [os.path.join(INCLUDE, f) for f in ("smp.h", "smp_cache.h", "smp_scores.h")]
    paths += [os.path.abspath(__file__), STEP_SOURCE]
    return max(os.path.getmtime(p) for p in paths)


def step_lacks():
    """What the extension module needs and this machine lacks, or None."""
    spec = importlib.util.find_spec("torch")
    if spec is None or not spec.submodule_search_locations:
        return "PyTorch"
    torch = spec.submodule_search_locations[0]
    if not os.path.exists(os.path.join(torch, "include", "torch", "csrc", "autograd", "python_variable.h")):
        return "PyTorch's headers"
    if not os.path.exists(os.path.join(torch, "lib", "libc10_cuda.so")):
        return "a PyTorch built for CUDA"
    if not os.path.exists(os.path.join(sysconfig.get_paths()["include"], "Python.h")):
        return "Python's headers"
    return None if shutil.which("g++") else "g++"


def _torch_version():
    """The installed PyTorch's version, where it can be had without importing it."""
    where = importlib.util.find_spec("torch").submodule_search_locations[0]
    with open(os.path.join(where, "version.py")) as f:
        found = re.search(r"^__version__ = ['\"](.+)['\"]", f.read(), re.M)
    if found:
        return found.group(1)
    import torch
    return str(torch.__version__)


def step_version():
    """The PyTorch that the extension module was built against, or None."""
    try:
        with open(STEP_LIB + ".torch") as f:
            return f.read()
    except FileNotFoundError:
        return None


def up_to_date():
    newest = _newest_input()
    wanted = (LIB,) if step_lacks() else (LIB, STEP_LIB)
    if not all(os.path.exists(p) and os.path.getmtime(p) >= newest for p in wanted):
        return False
    return STEP_LIB not in wanted or step_version() == _torch_version()


def _compile(src, extra):
    obj = os.path.join(BUILD, src.replace(".cu", ".o"))
    cmd = [nvcc(), *ARCH, *FLAGS, *extra, "-c", os.path.join(CSRC, src), "-o", obj]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"nvcc failed on {src}:\n{' '.join(cmd)}\n{res.stdout}\n{res.stderr}")
    return obj, res.stderr


def _compile_step():
    """Object file of the extension module, against the installed PyTorch."""
    from torch.utils import cpp_extension

    obj = os.path.join(BUILD, "step_binding.o")
    includes = [INCLUDE, sysconfig.get_paths()["include"], *cpp_extension.include_paths("cuda")]
    cmd = ["g++", "-O1", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-DTORCH_API_INCLUDE_EXTENSION_H",
           *[f"-isystem{p}" if p != INCLUDE else f"-I{p}" for p in includes], "-c", STEP_SOURCE, "-o", obj]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"g++ failed on {STEP_SOURCE}:\n{' '.join(cmd)}\n{res.stdout}\n{res.stderr}")
    return obj


def _link_step(obj):
    from torch.utils import cpp_extension

    tmp = STEP_LIB + ".tmp"
    libs = [p for p in cpp_extension.library_paths() if os.path.isdir(p)]
    cmd = ["g++", "-shared", obj, "-o", tmp, f"-L{BUILD}", "-lsmp", "-Wl,-rpath,$ORIGIN",
           *[f"-L{p}" for p in libs], *[f"-Wl,-rpath,{p}" for p in libs],
           "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"link failed:\n{' '.join(cmd)}\n{res.stdout}\n{res.stderr}")
    os.replace(tmp, STEP_LIB)
    with open(STEP_LIB + ".torch", "w") as f:
        f.write(_torch_version())


def build(force=False, verbose=False, extra=()):
    """Compile every CUDA source and link libsmp.so, and the extension module
    where this machine has what it takes; returns libsmp.so's path."""
    if not force and up_to_date():
        return LIB
    lacks = step_lacks()
    os.makedirs(BUILD, exist_ok=True)
    extra = list(extra)
    if verbose:
        extra += ["-Xptxas", "-v"]
    with concurrent.futures.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as pool:
        step = None if lacks else pool.submit(_compile_step)
        results = list(pool.map(lambda s: _compile(s, extra), SOURCES))
    if verbose:
        for (_, log), src in zip(results, SOURCES):
            sys.stderr.write(f"--- {src}\n{log}")
    objs = [obj for obj, _ in results]
    tmp = LIB + ".tmp"
    cmd = [nvcc(), *ARCH, "-shared", "-cudart", "static", *objs, "-o", tmp]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"link failed:\n{' '.join(cmd)}\n{res.stdout}\n{res.stderr}")
    os.replace(tmp, LIB)
    if lacks:
        sys.stderr.write(f"smp_step_binding.so is not built: this machine lacks {lacks} (libsmp.so does not need it)\n")
    else:
        _link_step(step.result())
    return LIB


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose", action="store_true", help="print ptxas register/spill reports")
    args = ap.parse_args()
    print(build(force=args.force, verbose=args.verbose))


if __name__ == "__main__":
    main()
