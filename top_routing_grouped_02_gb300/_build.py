"""Builds libmoe.so in-tree from csrc/*.cu with nvcc for sm_103a, and _native.so, the
compiled part of the Python binding, from csrc/binding.cpp.

Each translation unit compiles in parallel into _build/, then one link step
produces top_routing_grouped_02_gb300/libmoe.so (CUDA runtime linked statically,
so the library loads on a machine without a GPU driver). _native.so links against
it and against torch.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libmoe.so")
NATIVE = os.path.join(PKG, "_native.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
              "--expt-relaxed-constexpr", f"-I{os.path.join(ROOT, 'include')}"]


def nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _stale(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _stamp_file() -> str:
    return os.path.join(BUILD, "native.stamp")


def _read(path: str) -> str | None:
    if not os.path.exists(path):
        return None
    with open(path) as f:
        return f.read()


def _torch_dirs():
    import importlib.util
    spec = importlib.util.find_spec("torch")
    if spec is None:
        raise RuntimeError("torch is not installed")
    base = os.path.dirname(spec.origin)
    return os.path.join(base, "include"), os.path.join(base, "lib")


def _native_stamp(commands) -> str:
    """What _native.so is made with: it belongs to one torch."""
    with open(os.path.join(os.path.dirname(_torch_dirs()[0]), "version.py")) as f:
        return "\n".join([*(" ".join(c) for c in commands), f.read()])


def _native_compile(src: str, obj: str) -> list[str]:
    inc, _ = _torch_dirs()
    cuda = os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")
    dirs = [os.path.join(ROOT, "include"), sysconfig.get_paths()["include"], inc,
            os.path.join(inc, "torch", "csrc", "api", "include"), cuda]
    return ["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", *(f"-I{d}" for d in dirs),
            "-c", src, "-o", obj]


def _native_link(obj: str, out: str) -> list[str]:
    _, lib = _torch_dirs()
    return ["g++", "-shared", obj, "-o", out, f"-L{PKG}", "-l:libmoe.so", f"-L{lib}", "-ltorch_python", "-ltorch",
            "-ltorch_cpu", "-ltorch_cuda", "-lc10", "-lc10_cuda", "-Wl,-rpath,$ORIGIN", f"-Wl,-rpath,{lib}"]


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    """Builds both libraries and returns libmoe.so's path. Where _native.so cannot be made (no
    g++, no Python or torch headers) it says why and leaves none: the layer's calls need
    libmoe.so alone, and the sub-block's calls raise."""
    os.makedirs(BUILD, exist_ok=True)
    sources = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    headers = sorted(glob.glob(os.path.join(CSRC, "*.cuh"))) + [
        os.path.join(ROOT, "include", "moe.h")]
    objs = []
    jobs = []
    for src in sources:
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        objs.append(obj)
        if force or _stale(obj, [src] + headers):
            cmd = [nvcc(), *ARCH, *NVCC_FLAGS, *extra_flags, "-c", src, "-o", obj]
            jobs.append(cmd)
    with cf.ThreadPoolExecutor(max_workers=max(1, min(len(jobs) + 1, os.cpu_count() or 4))) as ex:
        native = ex.submit(_native_object, headers[-1], force, verbose)
        results = list(ex.map(lambda c: subprocess.run(c, capture_output=True, text=True), jobs))
    for cmd, r in zip(jobs, results):
        if verbose or r.returncode != 0:
            print(" ".join(cmd))
            print(r.stdout + r.stderr)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {cmd[-3]}")
    if force or _stale(LIB, objs):
        tmp = LIB + f".tmp{os.getpid()}"
        cmd = [nvcc(), *ARCH, "-shared", "-Xcompiler", "-fPIC", *objs, "-o", tmp]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            print(" ".join(cmd))
            print(r.stdout + r.stderr)
            raise RuntimeError("link of libmoe.so failed")
        os.replace(tmp, LIB)
    try:
        _native_finish(native.result())
    except (OSError, RuntimeError) as e:
        print(f"_native.so was not built, the sub-block's calls will raise: {e}")
        if os.path.exists(NATIVE):
            os.remove(NATIVE)
    return LIB


def _run_native(cmd, verbose: bool = False):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if verbose or r.returncode != 0:
        print(" ".join(cmd))
        print(r.stdout + r.stderr)
    if r.returncode != 0:
        raise RuntimeError(f"{cmd[0]} failed for {cmd[-1]}")


def _native_object(header: str, force: bool, verbose: bool):
    """Compiles the binding if it is out of date; what _native_finish links, or the error."""
    try:
        src, obj = os.path.join(CSRC, "binding.cpp"), os.path.join(BUILD, "binding.o")
        compile_cmd, link_cmd = _native_compile(src, obj), _native_link(obj, NATIVE)
        stamp = _native_stamp([compile_cmd, link_cmd])
        old = force or _stale(obj, [src, header]) or _read(_stamp_file()) != stamp
        if old:
            _run_native(compile_cmd, verbose)
        return obj, stamp, old
    except (OSError, RuntimeError) as e:
        return e


def _native_finish(made):
    if isinstance(made, Exception):
        raise made
    obj, stamp, old = made
    if old or _stale(NATIVE, [obj]):
        tmp = NATIVE + f".tmp{os.getpid()}"
        _run_native(_native_link(obj, tmp))
        os.replace(tmp, NATIVE)
        with open(_stamp_file(), "w") as f:
            f.write(stamp)


if __name__ == "__main__":
    print(build(verbose=True))
