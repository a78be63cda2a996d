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


def _read(path: str) -> str | None:
    if not os.path.exists(path):
        return None
    with open(path) as f:
        return f.read()


def _torch_dirs():
    import importlib.util
    base = os.path.dirname(importlib.util.find_spec("torch").origin)
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
    native_src = os.path.join(CSRC, "binding.cpp")
    native_obj = os.path.join(BUILD, "binding.o")
    native_cmds = [_native_compile(native_src, native_obj), _native_link(native_obj, NATIVE)]
    stamp, stamp_file = _native_stamp(native_cmds), os.path.join(BUILD, "native.stamp")
    native_old = _stale(native_obj, [native_src, headers[-1]]) or _read(stamp_file) != stamp
    if force or native_old:
        jobs.append(native_cmds[0])
    with cf.ThreadPoolExecutor(max_workers=max(1, min(len(jobs), os.cpu_count() or 4))) as ex:
        results = list(ex.map(lambda c: subprocess.run(c, capture_output=True, text=True), jobs))
    for cmd, r in zip(jobs, results):
        if verbose or r.returncode != 0:
            print(" ".join(cmd))
            print(r.stdout + r.stderr)
        if r.returncode != 0:
            raise RuntimeError(f"{os.path.basename(cmd[0])} failed for {cmd[-3]}")
    if force or _stale(LIB, objs):
        tmp = LIB + f".tmp{os.getpid()}"
        cmd = [nvcc(), *ARCH, "-shared", "-Xcompiler", "-fPIC", *objs, "-o", tmp]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            print(" ".join(cmd))
            print(r.stdout + r.stderr)
            raise RuntimeError("link of libmoe.so failed")
        os.replace(tmp, LIB)
    if force or native_old or _stale(NATIVE, [native_obj]):
        tmp = NATIVE + f".tmp{os.getpid()}"
        cmd = _native_link(native_obj, tmp)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            print(" ".join(cmd))
            print(r.stdout + r.stderr)
            raise RuntimeError("link of _native.so failed")
        os.replace(tmp, NATIVE)
        with open(stamp_file, "w") as f:
            f.write(stamp)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
