"""Build libzero.so (the C-ABI library) in-tree with nvcc for sm_103a.

Each translation unit is compiled in parallel, then linked into
zero_sharded_optimizer_flatten_gb300/libzero.so.  No cmake, no torch
extension machinery: the library has a plain C ABI and no torch types.
_train_ops.so beside it is the compiled part of the Python binding of the
training-step operators (csrc/train_ops_binding.cpp): it is linked against the
library and the installed torch, and holds no arithmetic.  Without torch the
library is built alone.
"""
from __future__ import annotations

import concurrent.futures as cf
import importlib.metadata
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libzero.so")
BINDING = os.path.join(HERE, "_train_ops.so")
BINDING_SOURCE = "train_ops_binding.cpp"

SOURCES = ["zero_plan.cpp", "zero_capi.cpp", "zero_launch.cu", "zero_kernels_fp16.cu",
           "zero_kernels_bf16.cu", "zero_noalloc.cu", "zero_cpu_adam.cpp", "zero_gradnorm.cu",
           "zero_join.cu", "zero_join_ff.cu", "zero_join_hh.cu", "zero_join_hf.cu",
           "zero_join_bb.cu", "zero_join_bf.cu", "zero_experts.cu", "zero_loss.cu",
           "zero_embed.cu", "zero_route.cu"]
# extra host-compiler flags per source: the host AdamW loop is vectorised at
# -O3; -fno-math-errno lets sqrtf be the plain instruction (results unchanged)
EXTRA = {"zero_cpu_adam.cpp": ["-Xcompiler", "-O3,-fno-math-errno"]}
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
# IEEE division and square root, no flush-to-zero, no FMA contraction of the
# explicitly rounded arithmetic (the kernels use __f*_rn intrinsics anyway).
CUDA_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-prec-div=true", "-prec-sqrt=true",
              "-ftz=false", "-fmad=false", "-Xcompiler", "-fPIC,-O2,-ffp-contract=off",
              "--expt-relaxed-constexpr"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libzero.so")


def _deps_mtime() -> float:
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    files.append(os.path.join(INCLUDE, "zero.h"))
    files.append(os.path.abspath(__file__))
    return max(os.path.getmtime(f) for f in files)


def _wanted() -> list:
    """What is built: the binding only where there is a torch to bind to."""
    return [LIB, BINDING] if importlib.util.find_spec("torch") else [LIB]


def _torch_version() -> str:
    try:
        return importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:  # on the path without its record
        import torch
        return torch.__version__


def _bound_to() -> str:
    """What a binding built now belongs to: torch and Python keep no binary
    interface from one version to the next."""
    spec = importlib.util.find_spec("torch")
    return f"torch {_torch_version()} {spec.origin} {sysconfig.get_config_var('SOABI')}"


def _bound_to_file() -> str:
    return os.path.join(BUILD, BINDING_SOURCE + ".for")


def binding_problem():
    """Why the binding cannot be loaded, None when it can."""
    if not os.path.exists(BINDING):
        return f"{BINDING} is not built"
    try:
        with open(_bound_to_file()) as f:
            same = f.read() == _bound_to()
    except FileNotFoundError:
        same = False
    return None if same else f"{BINDING} was built for another torch or Python"


def up_to_date() -> bool:
    newest, wanted = _deps_mtime(), _wanted()
    return (all(os.path.exists(f) and os.path.getmtime(f) >= newest for f in wanted)
            and (BINDING not in wanted or binding_problem() is None))


def _compile_binding() -> str:
    """Object file of the binding (the host compiler, torch's headers)."""
    import torch
    root = os.path.join(os.path.dirname(torch.__file__), "include")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include")
    obj = os.path.join(BUILD, BINDING_SOURCE + ".o")
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-Wall", "-Wextra", "-I", INCLUDE]
    for path in (sysconfig.get_paths()["include"], root,
                 os.path.join(root, "torch", "csrc", "api", "include"), cuda):
        cmd += ["-isystem", path]  # their warnings are not this file's
    cmd += ["-c", os.path.join(CSRC, BINDING_SOURCE), "-o", obj]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"g++ failed on {BINDING_SOURCE}:\n{' '.join(cmd)}\n{res.stderr}")
    sys.stderr.write(res.stderr)
    return obj


def _link_binding(obj: str):
    import torch
    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = BINDING + f".{os.getpid()}.tmp"
    cmd = ["g++", "-shared", "-o", tmp, obj, "-L", HERE, "-l:libzero.so", "-L", libs,
           "-ltorch_python", "-ltorch_cpu", "-lc10_cuda", "-lc10", "-Wl,-rpath,$ORIGIN",
           f"-Wl,-rpath,{libs}"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"link failed:\n{' '.join(cmd)}\n{res.stderr}")
    os.replace(tmp, BINDING)
    with open(_bound_to_file(), "w") as f:
        f.write(_bound_to())


def build(force: bool = False, verbose: bool = False, extra: list | None = None) -> str:
    if not force and up_to_date():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()
    extra = list(extra or [])

    def compile_one(src: str) -> str:
        obj = os.path.join(BUILD, src + ".o")
        cmd = [cc, *ARCH, *CUDA_FLAGS, *EXTRA.get(src, []), *extra, "-I", INCLUDE, "-I", CSRC, "-c",
               os.path.join(CSRC, src), "-o", obj]
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{' '.join(cmd)}\n{res.stdout}\n{res.stderr}")
        if verbose and (res.stdout or res.stderr):
            sys.stderr.write(res.stdout + res.stderr)
        return obj

    with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        binding = ex.submit(_compile_binding) if BINDING in _wanted() else None
        objs = list(ex.map(compile_one, SOURCES))
        if binding:
            binding = binding.result()
    tmp = LIB + f".{os.getpid()}.tmp"
    cmd = [cc, *ARCH, "-shared", "-o", tmp, *objs, "-Xcompiler", "-fPIC"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"link failed:\n{' '.join(cmd)}\n{res.stdout}\n{res.stderr}")
    os.replace(tmp, LIB)
    if binding:
        _link_binding(binding)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True,
                extra=["-Xptxas", "-v"] if "--ptxas" in sys.argv else None))
