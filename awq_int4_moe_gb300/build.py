"""Build the CUDA library ``libawqmoe.so`` in-tree for sm_103a.

Each ``csrc/*.cu`` is compiled to an object in parallel with nvcc, then the
objects are linked into one shared library next to this file. No CMake, no
torch extension machinery: the library is plain C ABI over the CUDA runtime.
Beside it goes ``_bind.so`` (``csrc/awq_bind.cpp``, host code), the CPython
module that takes the tensors of the decoder operators' calls apart; where
torch is not installed the library is built alone.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libawqmoe.so")
BIND = os.path.join(HERE, "_bind.so")
SOURCES = ["awq_moe_api.cu", "awq_moe_route.cu", "awq_moe_gemm.cu", "awq_moe_fused.cu", "awq_moe_prepare.cu",
           "awq_moe_sliced.cu", "awq_moe_tc.cu",
           "awq_moe_floor.cu", "awq_decoder_api.cu", "awq_norm.cu", "awq_rope.cu", "awq_attn.cu",
           "awq_fp8_gemm.cu", "awq_prompt_api.cu", "awq_qk_norm.cu", "awq_prompt_attn_f16.cu", "awq_prompt_attn_bf16.cu",
           "awq_prompt_attn_f16_e4m3.cu", "awq_prompt_attn_bf16_e4m3.cu"]
HEADERS = ["awq_ptx.cuh", "awq_moe_kernels.cuh", "awq_launch.cuh", "awq_dequant.cuh", "awq_route.cuh",
           "awq_router.cuh", "awq_split.cuh", "awq_tc.cuh", "awq_nvfp4.cuh",
           "awq_decoder_kernels.cuh", "awq_decoder_checks.cuh", "awq_rope.cuh", "awq_prompt_kernels.cuh",
           "awq_prompt_attn.cuh", "awq_prompt_units.cuh"]

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-std=c++17", "-O3", "-lineinfo", "--expt-relaxed-constexpr", "-Xcompiler", "-fPIC",
              "-Xcompiler", "-fvisibility=hidden", "-I", os.path.join(ROOT, "include")]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _bind_command(obj: str, src: str):
    """g++ compile and link of the binding module against the installed torch;
    None where there is none."""
    import importlib.util
    import sysconfig
    spec = importlib.util.find_spec("torch")
    if spec is None:
        return None
    torch_dir = os.path.dirname(spec.origin)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    include = os.path.join(torch_dir, "include")
    dirs = [include, os.path.join(include, "torch", "csrc", "api", "include"), os.path.join(cuda, "include"),
            sysconfig.get_paths()["include"]]
    cmd = ["g++", "-std=c++17", "-O2", "-fPIC", "-fvisibility=hidden", "-Wall"]
    for d in dirs:
        cmd += ["-isystem", d]
    link = ["g++", "-shared", "-L", os.path.join(torch_dir, "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python",
            "-L", HERE, "-l:libawqmoe.so", "-Wl,-rpath,$ORIGIN"]
    return cmd + ["-c", src, "-o", obj], link


def _torch_identity() -> str:
    """The installed torch, whose C++ libraries the binding is linked to."""
    import importlib.metadata
    import importlib.util
    try:
        version = importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:
        version = "unknown"
    return f"{version} {importlib.util.find_spec('torch').origin}\n"


def _read(path: str) -> str:
    if not os.path.exists(path):
        return ""
    with open(path) as f:
        return f.read()


def _stale(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _link(cmd, inputs, target: str) -> None:
    tmp = target + f".tmp{os.getpid()}"
    r = subprocess.run(cmd + ["-o", tmp] + inputs, capture_output=True, text=True)
    if r.returncode:
        raise RuntimeError("link failed: " + r.stdout + r.stderr)
    os.replace(tmp, target)


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    os.makedirs(BUILD, exist_ok=True)
    deps_common = [os.path.join(CSRC, h) for h in HEADERS] + [
        os.path.join(ROOT, "include", "awq_moe.h"), os.path.join(ROOT, "include", "awq_decoder.h"),
        os.path.join(ROOT, "include", "awq_prompt.h"),
        os.path.abspath(__file__)]
    objs, jobs = [], []
    for src in SOURCES:
        s = os.path.join(CSRC, src)
        o = os.path.join(BUILD, src.replace(".cu", ".o"))
        objs.append(o)
        if force or _stale(o, [s] + deps_common):
            cmd = [nvcc()] + ARCH + NVCC_FLAGS + list(extra_flags) + ["-c", s, "-o", o]
            if verbose:
                cmd += ["-Xptxas", "-v"]
            jobs.append(cmd)
    bind_src, bind_obj = os.path.join(CSRC, "awq_bind.cpp"), os.path.join(BUILD, "awq_bind.o")
    bind = _bind_command(bind_obj, bind_src)
    if bind is None:
        sys.stderr.write("torch is not installed: the library is built without its torch binding\n")
    bind_of = os.path.join(BUILD, "awq_bind.torch")          # which torch the binding was built against
    bind_stale = bind is not None and (force or _stale(bind_obj, [bind_src] + deps_common) or _read(bind_of) != _torch_identity())
    lib_jobs = bool(jobs)
    if bind_stale:
        jobs.append(bind[0])
    if jobs:
        with cf.ThreadPoolExecutor(max_workers=len(jobs)) as ex:
            res = list(ex.map(lambda c: subprocess.run(c, capture_output=True, text=True), jobs))
        for cmd, r in zip(jobs, res):
            if verbose or r.returncode:
                sys.stderr.write(r.stdout + r.stderr)
            if r.returncode:
                raise RuntimeError("compilation failed: " + " ".join(cmd))
    if force or lib_jobs or _stale(LIB, objs):
        _link([nvcc()] + ARCH + ["-shared", "-cudart", "shared"], objs, LIB)
    if bind is not None and (bind_stale or _stale(BIND, [bind_obj])):
        _link(bind[1][:2], [bind_obj] + bind[1][2:], BIND)
        with open(bind_of, "w") as f:
            f.write(_torch_identity())
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose="-v" in sys.argv)
    print(LIB)
