"""Build libmptp.so and the Python extension beside it in-tree (nvcc for sm_103a, g++; no CMake, parallel compiles).

    python -m tensor_transformer_layer_gb300.build

Compiles every ``csrc/*.cu`` with ``-gencode arch=compute_103a,code=sm_103a``
into ``_lib/`` and links ``_lib/libmptp.so`` (CUDA runtime linked statically;
the driver's tensor-map encoder is reached through the runtime's entry-point
query, so no libcuda link is needed at build time). ``csrc/mptp_bind.cpp``, which reads torch
tensors, becomes ``_lib/_mptp_bind.so``: it links libmptp.so and the installed torch, whose classes' layout it holds. So
``_lib/_mptp_bind.for`` says what it was built for, and it is built again for any other. libmptp.so needs neither
Python's headers nor torch's, and is linked before the extension.
"""
from __future__ import annotations

import glob
import importlib.util
import os
import runpy
import shutil
import subprocess
import sys
import sysconfig

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(PKG_DIR, "csrc")
LIB_DIR = os.path.join(PKG_DIR, "_lib")
LIB_PATH = os.path.join(LIB_DIR, "libmptp.so")
BIND_SRC = os.path.join(CSRC, "mptp_bind.cpp")
BIND_PATH = os.path.join(LIB_DIR, "_mptp_bind.so")
BIND_FOR_PATH = os.path.join(LIB_DIR, "_mptp_bind.for")
REPO = os.path.dirname(PKG_DIR)

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
              f"-I{os.path.join(REPO, 'include')}"]


def nvcc_path() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _torch_dir() -> str:
    return importlib.util.find_spec("torch").submodule_search_locations[0]


def bind_for() -> str:
    """The interpreter and the torch that are installed: an extension built for others must not be loaded."""
    v = runpy.run_path(os.path.join(_torch_dir(), "version.py"))
    return f"{sys.implementation.cache_tag}, torch {v['__version__']} {v['git_version']}"


def bind_built_for() -> str | None:
    """What the extension there is was built for."""
    try:
        with open(BIND_FOR_PATH) as f:
            return f.read()
    except OSError:
        return None


def bind_command(target: str, obj: bool):
    """Compiles the extension's object, or links it."""
    torch_dir = _torch_dir()
    out = target[:-3] + ".o"
    if obj:
        inc = [os.path.join(torch_dir, "include"), os.path.join(torch_dir, "include", "torch", "csrc", "api", "include"),
               os.path.join(os.path.dirname(os.path.dirname(nvcc_path())), "include"), sysconfig.get_paths()["include"],
               os.path.join(REPO, "include")]
        return ["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", *(f"-I{p}" for p in inc), "-c", BIND_SRC, "-o", out]
    lib = os.path.join(torch_dir, "lib")
    return ["g++", "-shared", out, "-o", target + ".tmp", f"-L{LIB_DIR}", "-lmptp", f"-L{lib}", "-lc10", "-lc10_cuda",
            "-ltorch_cpu", "-ltorch_python", "-Wl,-rpath,$ORIGIN", f"-Wl,-rpath,{lib}"]


def _stale(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def build(verbose: bool = False, force: bool = False) -> str:
    os.makedirs(LIB_DIR, exist_ok=True)
    nvcc = nvcc_path()
    headers = glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + \
        glob.glob(os.path.join(REPO, "include", "*.h"))
    objs, procs = [], []
    for src in sources():
        obj = os.path.join(LIB_DIR, os.path.basename(src)[:-3] + ".o")
        objs.append(obj)
        if force or _stale(obj, [src] + headers):
            cmd = [nvcc, *ARCH, *NVCC_FLAGS, "-c", src, "-o", obj]
            if verbose:
                print(" ".join(cmd), flush=True)
            procs.append((cmd, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
    bind_obj, bind = BIND_PATH[:-3] + ".o", None
    if force or bind_built_for() != bind_for() or _stale(bind_obj, [BIND_SRC, os.path.join(REPO, "include", "mptp.h")]):
        if os.path.exists(BIND_FOR_PATH):
            os.remove(BIND_FOR_PATH)
        bind = bind_command(BIND_PATH, True)
        bind = bind, subprocess.Popen(bind, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)
    failed = []
    for cmd, p in procs:
        out, _ = p.communicate()
        if p.returncode != 0:
            failed.append((cmd, out.decode(errors="replace")))
        elif verbose and out:
            print(out.decode(errors="replace"))
    if bind is not None:
        out, _ = bind[1].communicate()
    if failed:
        msg = "\n".join(f"$ {' '.join(c)}\n{o}" for c, o in failed)
        raise RuntimeError(f"nvcc failed:\n{msg}")
    if force or _stale(LIB_PATH, objs):
        tmp = LIB_PATH + ".tmp"
        cmd = [nvcc, *ARCH, "-shared", "-o", tmp, *objs]
        if verbose:
            print(" ".join(cmd), flush=True)
        r = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout.decode(errors='replace')}")
        os.replace(tmp, LIB_PATH)
    if bind is not None and bind[1].returncode != 0:
        raise RuntimeError(f"the extension's compilation failed:\n$ {' '.join(bind[0])}\n{out.decode(errors='replace')}")
    if bind is not None or _stale(BIND_PATH, [bind_obj, LIB_PATH]):
        cmd = bind_command(BIND_PATH, False)
        r = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n$ {' '.join(cmd)}\n{r.stdout.decode(errors='replace')}")
        os.replace(BIND_PATH + ".tmp", BIND_PATH)
        with open(BIND_FOR_PATH, "w") as f:
            f.write(bind_for())
    return LIB_PATH


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv, force="-f" in sys.argv))
