"""Build libmk.so in-tree with nvcc for sm_100a (B200), and _tensors.so, the
module behind the serving operators' tensor calls, with the host compiler.

``python -m event_tensor_task_b200.build`` or ``build()`` from Python.  A
source is compiled again when it, or any header under ``csrc/`` or
``include/``, is newer than its object (kept under ``_build/``), or when the
object was made another way: with other flags or, for the module, against
another torch or Python.  What made an object stands beside it.  The sources
compile side by side.
"""
import glob
import importlib.metadata
import os
import subprocess
import sys
import sysconfig
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
TENSORS_FLAGS = ["-O2", "-std=c++17", "-fPIC", "-shared", "-Wall"]


def _newer(path, than) -> bool:
    return not os.path.exists(than) or os.path.getmtime(path) > os.path.getmtime(than)


def _headers():
    found = [os.path.join(HERE, "build.py")] + glob.glob(os.path.join(ROOT, "include", "*.h"))
    for ext in ("*.h", "*.hpp", "*.cuh"):
        found += glob.glob(os.path.join(HERE, "csrc", ext))
    return found


def _object(source) -> str:
    return os.path.join(OBJ, os.path.basename(source) + ".o")


def _made_by(out, how=None) -> str:
    """What made an output, as noted beside its object; with `how`, notes it."""
    note = os.path.join(OBJ, os.path.basename(out) + ".how")
    if how is not None:
        with open(note, "w") as f:
            f.write(how)
        return how
    if not os.path.exists(note):
        return ""
    with open(note) as f:
        return f.read()


def _object_how(extra) -> str:
    return " ".join([NVCC] + FLAGS + list(extra or []))


def _tensors_how() -> str:
    return " ".join([CXX] + TENSORS_FLAGS + ["torch", importlib.metadata.version("torch"), sysconfig.get_config_var("SOABI"),
                                             sysconfig.get_paths()["include"]])


def _due(extra=None):
    """(sources whose objects are stale, is the module stale, is the library)"""
    headers = _headers()
    objects = [s for s in SOURCES if any(_newer(d, _object(s)) for d in [os.path.join(HERE, s)] + headers) or
               _made_by(_object(s)) != _object_how(extra)]
    tensors = any(_newer(d, TENSORS) for d in [os.path.join(HERE, TENSORS_SOURCE)] + headers) or \
        _made_by(TENSORS) != _tensors_how()
    return objects, tensors, bool(objects) or any(_newer(_object(s), LIB) for s in SOURCES)


def _tensors_command():
    import torch
    root = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(NVCC))
    include = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
               sysconfig.get_paths()["include"], os.path.join(cuda, "include")]
    return [CXX] + TENSORS_FLAGS + [
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
    objects, tensors, library = (SOURCES, True, True) if force else _due(extra)
    os.makedirs(OBJ, exist_ok=True)
    todo = [([NVCC] + FLAGS + list(extra or []) + ["-c", "-o", _object(s), os.path.join(HERE, s)], _object(s),
             _object_how(extra)) for s in objects]
    if tensors:
        todo.append((_tensors_command(), TENSORS, _tensors_how()))

    def make(command, out, how):
        _made_by(out, "")  # (nothing, should this fail)
        _run(command, verbose)
        _made_by(out, how)

    with ThreadPoolExecutor(max_workers=max(1, min(len(todo), os.cpu_count() or 1))) as pool:
        list(pool.map(lambda t: make(*t), todo))
    if library:
        _run([NVCC] + FLAGS + ["-shared", "-lcudart", "-o", LIB] + [_object(s) for s in SOURCES], verbose)
    return LIB


if __name__ == "__main__":
    force = "--force" in sys.argv
    extra = ["-Xptxas", "-v"] if "--ptxas-v" in sys.argv else None
    print(build(force=force, verbose=True, extra=extra))
