"""Build libmk.so in-tree with nvcc for sm_100a (B200), and _tensors.so, the
module behind the serving operators' tensor calls, with the host compiler.

``python -m event_tensor_task_b200.build`` or ``build()`` from Python.  A
source is compiled again when it, or any header under ``csrc/`` or
``include/``, is newer than its object (kept under ``_build/``); the sources
compile side by side.
"""
import glob
import os
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
LIB = os.path.join(HERE, "libmk.so")
TENSORS = os.path.join(HERE, "_tensors.so")
OBJ = os.path.join(HERE, "_build")
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
CXX = os.environ.get("CXX", "g++")

SOURCES = ["csrc/megakernel.cu", "csrc/plan.cpp", "csrc/api.cpp", "csrc/serve_checks.cpp", "csrc/append_kv.cu",
           "csrc/prompt_attn.cu", "csrc/paged_attn.cu", "csrc/logits.cu"]
TENSORS_SOURCE = "csrc/tensors.cpp"
FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a", "-lineinfo", "-O3", "-std=c++17",
    "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall", "--expt-relaxed-constexpr",
]


def _newer(path, than) -> bool:
    return not os.path.exists(than) or os.path.getmtime(path) > os.path.getmtime(than)


def _headers():
    found = [os.path.join(HERE, "build.py")] + glob.glob(os.path.join(ROOT, "include", "*.h"))
    for ext in ("*.h", "*.hpp", "*.cuh"):
        found += glob.glob(os.path.join(HERE, "csrc", ext))
    return found


def _stale() -> bool:
    headers = _headers()
    return (any(_newer(d, LIB) for d in [os.path.join(HERE, s) for s in SOURCES] + headers) or
            any(_newer(d, TENSORS) for d in [os.path.join(HERE, TENSORS_SOURCE)] + headers))


def _tensors_command():
    import sysconfig

    import torch
    root = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(NVCC))
    include = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
               sysconfig.get_paths()["include"], os.path.join(cuda, "include")]
    return [CXX, "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-o", TENSORS,
            os.path.join(HERE, TENSORS_SOURCE)] + ["-I" + i for i in include] + [
                "-L" + os.path.join(root, "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"]


def _run(cmd, verbose):
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, cwd=HERE, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{cmd[0]} failed:\n" + r.stdout + r.stderr)
    if verbose and (r.stdout or r.stderr):
        print(r.stdout + r.stderr)


def build(force: bool = False, verbose: bool = False, extra=None) -> str:
    if not force and not _stale():
        return LIB
    os.makedirs(OBJ, exist_ok=True)
    headers = _headers()
    todo, objects = [], []
    for s in SOURCES:
        src, obj = os.path.join(HERE, s), os.path.join(OBJ, os.path.basename(s) + ".o")
        objects.append(obj)
        if force or any(_newer(d, obj) for d in [src] + headers):
            todo.append([NVCC] + FLAGS + (extra or []) + ["-c", "-o", obj, src])
    if force or any(_newer(d, TENSORS) for d in [os.path.join(HERE, TENSORS_SOURCE)] + headers):
        todo.append(_tensors_command())
    with ThreadPoolExecutor(max_workers=max(1, min(len(todo), os.cpu_count() or 1))) as pool:
        list(pool.map(lambda cmd: _run(cmd, verbose), todo))
    _run([NVCC] + FLAGS + ["-shared", "-lcudart", "-o", LIB] + objects, verbose)
    return LIB


if __name__ == "__main__":
    force = "--force" in sys.argv
    extra = ["-Xptxas", "-v"] if "--ptxas-v" in sys.argv else None
    print(build(force=force, verbose=True, extra=extra))
