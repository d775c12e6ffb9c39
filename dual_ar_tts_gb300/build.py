"""Build ``libs2frame.so`` in-tree with nvcc for sm_103a (one -gencode, TUs compiled in parallel), and, where torch and Python's
headers are installed, ``_calls.so``, the 8-bit operators' calls on torch tensors, with g++ against that torch."""
from __future__ import annotations

import concurrent.futures as cf
import importlib.util
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
AGAINST = "calls.against"    # in BUILD: the torch and Python that _calls.so was built against
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


def _older(out: str, deps: list[str]) -> bool:
    return not os.path.exists(out) or any(os.path.getmtime(p) > os.path.getmtime(out) for p in deps)


def _stale() -> bool:
    return _older(OUT, [os.path.join(CSRC, s) for s in SOURCES] + [os.path.join(CSRC, h) for h in HEADERS])


def _torch() -> str | None:
    """Where the installed torch is (it is not imported); None where there is none, or no Python.h."""
    spec = importlib.util.find_spec("torch")
    if spec is None or not spec.origin or not os.path.exists(os.path.join(sysconfig.get_paths()["include"], "Python.h")):
        return None
    return os.path.dirname(spec.origin)


def _against(torch: str) -> str:
    with open(os.path.join(torch, "version.py")) as f:
        return f"{sys.version}\n{torch}\n{f.read()}"


def _calls_stale(torch: str) -> bool:
    if _older(CALLS, [os.path.join(CSRC, "calls.cpp"), os.path.join(CSRC, HEADERS[-1])]):
        return True
    try:
        with open(os.path.join(BUILD, AGAINST)) as f:
            return f.read() != _against(torch)
    except OSError:
        return True


def _torch_flags(torch: str) -> tuple[list[str], list[str]]:
    """What compiling and linking against it takes."""
    cuda = os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")
    dirs = [os.path.join(torch, "include"), os.path.join(torch, "include", "torch", "csrc", "api", "include"),
            sysconfig.get_paths()["include"], cuda]
    lib = os.path.join(torch, "lib")
    return ["-O2", "-std=c++17", "-fPIC", *["-isystem" + d for d in dirs]], \
        ["-L" + lib, "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_cuda", "-Wl,-rpath," + lib]


def _run(cmd: list[str], what: str) -> str:
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what}:\n{r.stderr}")
    return r.stderr


def build(force: bool = False, verbose: bool = False, extra: list[str] | None = None) -> str:
    """Builds what is older than its sources, or than the torch that it goes with (or everything); the library's path.  The
    library is in place before a failure of the other is raised."""
    torch = _torch()
    lib, calls = force or _stale(), torch is not None and (force or _calls_stale(torch))
    if not lib and not calls:
        return OUT
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()
    extra = list(extra or [])

    def compile_one(src):
        obj = os.path.join(BUILD, src.replace(".cu", ".o"))
        said = _run([cc, *ARCH, *FLAGS, *extra, "-c", os.path.join(CSRC, src), "-o", obj], f"nvcc failed for {src}")
        if verbose and said:
            sys.stderr.write(said)
        return obj

    def compile_calls():
        obj = os.path.join(BUILD, "calls.o")
        _run(["g++", *_torch_flags(torch)[0], "-c", os.path.join(CSRC, "calls.cpp"), "-o", obj], "g++ failed for calls.cpp")
        return obj

    with cf.ThreadPoolExecutor(len(SOURCES) + 1) as ex:
        calls_obj = ex.submit(compile_calls) if calls else None
        objs = list(ex.map(compile_one, SOURCES)) if lib else []
    if lib:
        tmp = OUT + f".tmp{os.getpid()}"
        _run([cc, *ARCH, "-shared", "-o", tmp, *objs], "link failed")
        os.replace(tmp, OUT)
    if calls:
        tmp = CALLS + f".tmp{os.getpid()}"
        _run(["g++", "-shared", "-o", tmp, calls_obj.result(), "-L" + HERE, "-l:libs2frame.so", "-Wl,-rpath,$ORIGIN",
              *_torch_flags(torch)[1]], "link failed")
        os.replace(tmp, CALLS)
        with open(os.path.join(BUILD, AGAINST), "w") as f:
            f.write(_against(torch))
    return OUT


if __name__ == "__main__":
    v = "-v" in sys.argv
    extra = ["-Xptxas", "-v"] if v else None
    print(build(force=True, verbose=v, extra=extra))
