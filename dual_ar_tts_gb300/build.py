"""Build ``libs2frame.so`` in-tree with nvcc for sm_103a (one -gencode, TUs compiled in parallel), and ``_calls.so``, the
8-bit operators' calls on torch tensors, with g++ against the installed torch."""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
OUT = os.path.join(HERE, "libs2frame.so")
CALLS = os.path.join(HERE, "_calls.so")
BUILD = os.path.join(HERE, "_build")
SOURCES = ["fk_bf16_h128.cu", "fk_bf16_h64.cu", "fk_f32_h128.cu", "fk_f32_h64.cu", "frame_launch.cu", "prefill.cu",
           "engine.cu", "batch.cu", "codec.cu", "draw.cu", "q4.cu", "kv4.cu", "kv4_attn.cu", "adjust.cu", "q8.cu",
           "q8_matmul.cu"]
HEADERS = ["s2_internal.h", "ptx.cuh", "frame_kernel.cuh", "sampler.cuh", "tc05.cuh",
           "convert.cuh", "kv4.cuh", "q8.cuh", os.path.join("..", "..", "include", "s2frame.h")]

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr"]


def nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _stale() -> bool:
    if not os.path.exists(OUT) or not os.path.exists(CALLS):
        return True
    t = min(os.path.getmtime(OUT), os.path.getmtime(CALLS))
    deps = [os.path.join(CSRC, s) for s in SOURCES + ["calls.cpp"]] + [os.path.join(CSRC, h) for h in HEADERS]
    return any(os.path.getmtime(p) > t for p in deps)


def _torch_flags() -> tuple[list[str], list[str]]:
    """What compiling and linking against the installed torch takes."""
    import torch
    t = os.path.dirname(torch.__file__)
    cuda = os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")
    dirs = [os.path.join(t, "include"), os.path.join(t, "include", "torch", "csrc", "api", "include"),
            sysconfig.get_paths()["include"], cuda]
    lib = os.path.join(t, "lib")
    return ["-O2", "-std=c++17", "-fPIC", *["-isystem" + d for d in dirs]], \
        ["-L" + lib, "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_cuda", "-Wl,-rpath," + lib]


def build(force: bool = False, verbose: bool = False, extra: list[str] | None = None) -> str:
    if not force and not _stale():
        return OUT
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()
    extra = list(extra or [])

    def compile_one(src):
        obj = os.path.join(BUILD, src.replace(".cu", ".o"))
        cmd = [cc, *ARCH, *FLAGS, *extra, "-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stderr}")
        if verbose and r.stderr:
            sys.stderr.write(r.stderr)
        return obj

    flags, libs = _torch_flags()

    def compile_calls():
        obj = os.path.join(BUILD, "calls.o")
        r = subprocess.run(["g++", *flags, "-c", os.path.join(CSRC, "calls.cpp"), "-o", obj], capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"g++ failed for calls.cpp:\n{r.stderr}")
        return obj

    with cf.ThreadPoolExecutor(len(SOURCES) + 1) as ex:
        calls = ex.submit(compile_calls)
        objs = list(ex.map(compile_one, SOURCES))
        calls = calls.result()
    tmp = OUT + f".tmp{os.getpid()}"
    r = subprocess.run([cc, *ARCH, "-shared", "-o", tmp, *objs], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, OUT)
    tmp = CALLS + f".tmp{os.getpid()}"
    r = subprocess.run(["g++", "-shared", "-o", tmp, calls, "-L" + HERE, "-l:libs2frame.so", "-Wl,-rpath,$ORIGIN", *libs],
                       capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, CALLS)
    return OUT


if __name__ == "__main__":
    v = "-v" in sys.argv
    extra = ["-Xptxas", "-v"] if v else None
    print(build(force=True, verbose=v, extra=extra))
