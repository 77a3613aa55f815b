"""Build the in-tree CUDA library ``libsmla.so`` for sm_103a with nvcc, and the
compiled part of its Python binding (``_smla_torch.so``) with the host compiler.

Each ``csrc/*.cu`` translation unit compiles in its own nvcc process (in
parallel), then nvcc links the shared library next to this file.  A unit is
rebuilt only when it, a header under ``csrc/`` or ``include/smla.h`` is newer
than its object.  The library needs nvcc alone and is linked whatever becomes
of the binding, which compiles beside it against the installed torch's headers,
again when another torch or Python is installed; without a torch there is
none.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG_DIR)
CSRC = os.path.join(PKG_DIR, "csrc")
BUILD_DIR = os.path.join(ROOT, "_build")
LIB_PATH = os.path.join(PKG_DIR, "libsmla.so")
BINDING_SRC = os.path.join(CSRC, "smla_torch.cpp")
BINDING_PATH = os.path.join(PKG_DIR, "_smla_torch.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
                     "--expt-relaxed-constexpr", "-Xptxas", "-v"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"),
                 "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: set NVCC or put CUDA's bin on PATH")


def _headers():
    return (glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh"))
            + [os.path.join(ROOT, "include", "smla.h")])


def _stale(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _read(path: str) -> str:
    if not os.path.exists(path):
        return ""
    with open(path) as f:
        return f.read()


def _compile(nvcc, src, obj, log_dir):
    cmd = [nvcc] + NVCC_FLAGS + ["-c", src, "-o", obj]
    p = subprocess.run(cmd, capture_output=True, text=True)
    with open(os.path.join(log_dir, os.path.basename(src) + ".log"), "w") as f:
        f.write(" ".join(cmd) + "\n" + p.stdout + p.stderr)
    if p.returncode != 0:
        raise RuntimeError(f"nvcc failed on {src}:\n{p.stderr[-6000:]}")
    return obj


def _torch_dir():
    """The installed torch's folder (None without one), not imported."""
    spec = importlib.util.find_spec("torch")
    return list(spec.submodule_search_locations)[0] if spec else None


def _torch_key() -> str:
    """What the binding's object is compiled against."""
    return f"{sys.version}\n{_torch_dir()}\n" + _read(os.path.join(_torch_dir(), "version.py"))


def _compile_binding(obj, log_dir):
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(_nvcc())))
    inc = [os.path.join(_torch_dir(), "include"),
           os.path.join(cuda, "include"), sysconfig.get_paths()["include"]]
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden"]
    cmd += ["-I" + p for p in inc] + ["-c", BINDING_SRC, "-o", obj]
    p = subprocess.run(cmd, capture_output=True, text=True)
    with open(os.path.join(log_dir, "smla_torch.cpp.log"), "w") as f:
        f.write(" ".join(cmd) + "\n" + p.stdout + p.stderr)
    if p.returncode != 0:
        raise RuntimeError(f"the binding failed to compile:\n{p.stderr[-6000:]}")
    return obj


def _link(cmd):
    p = subprocess.run(cmd, capture_output=True, text=True)
    if p.returncode != 0:
        raise RuntimeError(f"link failed:\n{p.stderr[-4000:]}")


def build(verbose: bool = False, force: bool = False) -> str:
    """Compile every CUDA unit and link libsmla.so, then compile and link its
    Python binding; returns the library path."""
    nvcc = _nvcc()
    os.makedirs(BUILD_DIR, exist_ok=True)
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    hdrs = _headers()
    jobs = []
    objs = []
    for src in srcs:
        obj = os.path.join(BUILD_DIR, os.path.basename(src)[:-3] + ".o")
        objs.append(obj)
        if force or _stale(obj, [src] + hdrs):
            jobs.append((src, obj))
    binding_obj = os.path.join(BUILD_DIR, "smla_torch.o")
    header = os.path.join(ROOT, "include", "smla.h")
    with_binding = _torch_dir() is not None
    stamp = os.path.join(BUILD_DIR, "smla_torch.key")
    binding_job = with_binding and (force or _stale(binding_obj, [BINDING_SRC, header])
                                    or _read(stamp) != _torch_key())
    binding = None
    if jobs or binding_job:
        with cf.ThreadPoolExecutor(max_workers=max(1, min(len(jobs) + 1, os.cpu_count() or 4))) as ex:
            if binding_job:
                binding = ex.submit(_compile_binding, binding_obj, BUILD_DIR)
            futs = [ex.submit(_compile, nvcc, s, o, BUILD_DIR) for s, o in jobs]
            for f in futs:
                f.result()
        if verbose:
            for s, _ in jobs:
                with open(os.path.join(BUILD_DIR, os.path.basename(s) + ".log")) as f:
                    sys.stdout.write(f.read())
    if force or jobs or _stale(LIB_PATH, objs):
        _link([nvcc] + ARCH + ["-shared", "-o", LIB_PATH] + objs)
    if binding is not None:
        binding.result()  # the library is there even when this raises
        with open(stamp, "w") as f:
            f.write(_torch_key())
    if with_binding and (force or jobs or binding_job or _stale(BINDING_PATH, [binding_obj, LIB_PATH])):
        _link([os.environ.get("CXX", "g++"), "-shared", "-o", BINDING_PATH, binding_obj,
               "-L" + PKG_DIR, "-l:libsmla.so", "-Wl,-rpath,$ORIGIN",
               "-L" + os.path.join(_torch_dir(), "lib"), "-ltorch_python",
               "-ltorch_cpu", "-lc10_cuda", "-lc10"])
    return LIB_PATH


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv, force="-f" in sys.argv))
