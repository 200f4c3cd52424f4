"""Builds libspecverify.so in-tree with nvcc for sm_103a (GB300).

Each .cu file under csrc/ is compiled in parallel to an object file under
_build/, then linked into a shared library next to this file.  The CUDA
runtime is linked statically, so the library only needs the driver.

_marshal.so, the torch marshalling of the calls that run on every layer
(csrc/sv_torch.cpp), is host code: compiled beside them with g++ against the
installed torch, linked to libspecverify.so.  It uses torch's C++ classes, so it
is built again when torch or Python is another one than it was built with, and
left out where torch is not installed (libspecverify.so does not need it).
"""
from __future__ import annotations

import glob
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
LIB = os.path.join(HERE, "libspecverify.so")
MARSHAL = os.path.join(HERE, "_marshal.so")
MARSHAL_STAMP = os.path.join(BUILD, "sv_torch.stamp")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
              "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libspecverify.so")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _torch_dir():
    """Where torch is installed, without importing it (minutes on a cold machine); None if it is not."""
    spec = importlib.util.find_spec("torch")
    return None if spec is None or not spec.origin else os.path.dirname(spec.origin)


def _marshal_stamp(torch_dir: str) -> str:
    """What _marshal.so depends on beside its sources: torch, by its place and version file, and
    Python, by its extension modules' suffix."""
    try:
        with open(os.path.join(torch_dir, "version.py")) as f:
            version = f.read()
    except OSError:
        version = ""
    return "\n".join((torch_dir, str(sysconfig.get_config_var("EXT_SUFFIX")), version))


def marshal_matches(torch_dir: str) -> bool:
    """Whether _marshal.so was built for this torch and Python."""
    try:
        with open(MARSHAL_STAMP) as f:
            return f.read() == _marshal_stamp(torch_dir)
    except OSError:
        return False


def _marshal_commands(torch_dir: str):
    """(source, object, compile command, link command) of _marshal.so."""
    src, obj = os.path.join(CSRC, "sv_torch.cpp"), os.path.join(BUILD, "sv_torch.o")
    inc = [INCLUDE, os.path.join(torch_dir, "include"),
           os.path.join(torch_dir, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"], os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")]
    lib = os.path.join(torch_dir, "lib")
    compile_ = ["g++", "-O2", "-std=c++17", "-fPIC", *("-I" + i for i in inc), "-c", src, "-o", obj]
    link = ["g++", "-shared", obj, "-o", MARSHAL, "-L" + HERE, "-lspecverify", "-Wl,-rpath,$ORIGIN", "-L" + lib,
            "-Wl,-rpath," + lib, "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    return src, obj, compile_, link


def _stale(out: str, deps) -> bool:
    if not os.path.exists(out):
        return True
    t = os.path.getmtime(out)
    return any(os.path.getmtime(d) > t for d in deps)


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    os.makedirs(BUILD, exist_ok=True)
    headers = glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh")) + \
        glob.glob(os.path.join(INCLUDE, "*.h"))
    objs, procs = [], []
    for src in sources():
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        objs.append(obj)
        if force or _stale(obj, [src] + headers):
            cmd = [nvcc(), *ARCH, *NVCC_FLAGS, *extra_flags, "-c", src, "-o", obj]
            if verbose:
                print(" ".join(cmd), flush=True)
            procs.append((cmd, subprocess.Popen(cmd, stdout=subprocess.PIPE,
                                                stderr=subprocess.STDOUT, text=True)))
    torch_dir = _torch_dir()
    if torch_dir is None:
        print("torch is not installed: _marshal.so, which the cache, attention and log-probability "
              "helpers of the Python package need, is left out", file=sys.stderr)
    else:
        msrc, mobj, mcompile, mlink = _marshal_commands(torch_dir)
        remake = force or not marshal_matches(torch_dir)
    if torch_dir is not None and (remake or _stale(mobj, [msrc, os.path.join(INCLUDE, "spec_verify.h")])):
        if verbose:
            print(" ".join(mcompile), flush=True)
        procs.append((mcompile, subprocess.Popen(mcompile, stdout=subprocess.PIPE,
                                                 stderr=subprocess.STDOUT, text=True)))
    failed = []
    for cmd, p in procs:
        out, _ = p.communicate()
        if verbose and out:
            print(out, flush=True)
        if p.returncode != 0:
            failed.append((cmd, out))
    if failed:
        msg = "\n".join(" ".join(c) + "\n" + o for c, o in failed)
        raise RuntimeError("compilation failed:\n" + msg)
    if force or _stale(LIB, objs):
        tmp = LIB + ".tmp%d" % os.getpid()
        cmd = [nvcc(), *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs]
        if verbose:
            print(" ".join(cmd), flush=True)
        subprocess.run(cmd, check=True)
        os.replace(tmp, LIB)
    if torch_dir is not None and (remake or _stale(MARSHAL, [mobj, LIB])):
        tmp = MARSHAL + ".tmp%d" % os.getpid()
        subprocess.run([tmp if x == MARSHAL else x for x in mlink], check=True)
        os.replace(tmp, MARSHAL)
        with open(MARSHAL_STAMP, "w") as f:
            f.write(_marshal_stamp(torch_dir))
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
