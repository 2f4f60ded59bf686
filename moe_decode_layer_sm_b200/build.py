"""Build step of libmonoffn.so (nvcc, sm_100a only), in-tree next to the
package so that the library travels with the source tree.

The library is rebuilt unless a stamp file beside it records the SHA-256 of
every source it is built from and of the nvcc commands: a binary that merely
has a later modification time than its sources is not trusted.  Each
translation unit keeps an object with a stamp of its own.

_call.so, the compiled part of the attention half's binding, is built beside it
with g++ against the installed torch and has its own stamp.  Where torch or
Python's headers are missing the library is built alone: the C ABI and the FFN
binding need no more, and attn.py then says what it misses."""

import hashlib
import importlib.util
import os
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
INCLUDE = os.path.join(ROOT, "include")
# translation units and what each is built from
UNITS = {
    "mono_ffn": ["mono_ffn.cu", "common.cuh", "cc_kernel.cuh", "tc_kernel.cuh", "ptx.cuh", "route_noalloc.cuh",
                 "tq_kernel.cuh", "mono_ffn.h"],
    "mono_attn": ["mono_attn.cu", "proj.cuh", "kv_attend.cuh", "kv_append.cuh", "rope.cuh", "kv_index.h", "ptx.cuh",
                  "mono_ffn.h", "mono_attn.h"],
}
SO = os.path.join(PKG, "libmonoffn.so")
STAMP = SO + ".sha256"

NVCC_FLAGS = ["-gencode", "arch=compute_100a,code=sm_100a", "-O3", "-lineinfo", "-std=c++17", "-maxrregcount=168",
              "-Xcompiler", "-fPIC",
              "-Xptxas", "-v"]


def _path(name):
    return os.path.join(INCLUDE if name.endswith(".h") and name.startswith("mono_") else os.path.join(PKG, "csrc"), name)


def _object(unit):
    return os.path.join(PKG, unit + ".o")


def compile_command(unit):
    return ["nvcc", *NVCC_FLAGS, "-I", INCLUDE, "-c", "-o", _object(unit), _path(UNITS[unit][0])]


def command():
    """The link step."""
    return ["nvcc", "-gencode", "arch=compute_100a,code=sm_100a", "-shared", "-o", SO, *map(_object, UNITS)]


def unit_hash(unit):
    h = hashlib.sha256()
    for d in UNITS[unit]:
        h.update(d.encode() + b"\0")
        with open(_path(d), "rb") as f:
            h.update(f.read())
    h.update(" ".join(compile_command(unit)).encode())
    return h.hexdigest()


def source_hash():
    """SHA-256 over every unit's sources (name and bytes, in a fixed order) and
    the nvcc commands."""
    h = hashlib.sha256()
    for u in UNITS:
        h.update(unit_hash(u).encode())
    h.update(" ".join(command()).encode())
    return h.hexdigest()


def up_to_date():
    if not (os.path.exists(SO) and os.path.exists(STAMP)):
        return False
    with open(STAMP) as f:
        return f.read().strip() == source_hash()


CALL = os.path.join(PKG, "_call.so")
CALL_SOURCES = ["call.cpp", "mono_attn.h", "mono_ffn.h"]


def call_command():
    import torch
    t = os.path.join(os.path.dirname(torch.__file__))
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    inc = [os.path.join(t, "include"), os.path.join(t, "include", "torch", "csrc", "api", "include"),
           os.path.join(cuda, "include"), sysconfig.get_paths()["include"]]
    return ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-I", INCLUDE, *[f"-isystem{p}" for p in inc],
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-o", CALL, _path("call.cpp"),
            "-L", PKG, "-l:libmonoffn.so", "-L", os.path.join(t, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10_cuda",
            "-lc10", "-Wl,-rpath,$ORIGIN"]


def call_hash():
    import torch
    h = hashlib.sha256()
    for d in CALL_SOURCES:
        with open(_path(d), "rb") as f:
            h.update(f.read())
    h.update(" ".join([torch.__version__, sys.version, *call_command()]).encode())
    return h.hexdigest()


def can_build_call():
    return importlib.util.find_spec("torch") is not None and \
        os.path.exists(os.path.join(sysconfig.get_paths()["include"], "Python.h"))


def build_call(force=False):
    if not can_build_call():
        return None
    stamp = CALL + ".sha256"
    if not force and os.path.exists(CALL) and os.path.exists(stamp):
        with open(stamp) as f:
            if f.read().strip() == call_hash():
                return CALL
    if os.path.exists(stamp):
        os.unlink(stamp)
    _run(call_command())
    with open(stamp, "w") as f:
        f.write(call_hash() + "\n")
    return CALL


def _run(cmd):
    res = subprocess.run(cmd, capture_output=True, text=True)
    log = " ".join(cmd) + "\n" + res.stdout + res.stderr
    if res.returncode != 0:
        raise RuntimeError(f"{cmd[0]} failed:\n" + log[-4000:])
    return log


def _compile(unit, force):
    """One unit's object, unless the stamp beside it records these sources."""
    stamp = _object(unit) + ".sha256"
    if not force and os.path.exists(_object(unit)) and os.path.exists(stamp):
        with open(stamp) as f:
            if f.read().strip() == unit_hash(unit):
                return ""
    if os.path.exists(stamp):
        os.unlink(stamp)
    log = _run(compile_command(unit))
    with open(stamp, "w") as f:
        f.write(unit_hash(unit) + "\n")
    return log


def build(force=False, verbose=False):
    if not force and up_to_date():
        build_call()
        return SO
    if os.path.exists(STAMP):
        os.unlink(STAMP)
    with ThreadPoolExecutor(len(UNITS)) as pool:   # nvcc runs in its own process
        logs = list(pool.map(lambda u: _compile(u, force), UNITS))
    log = "".join(logs) + _run(command())
    with open(os.path.join(PKG, "build.log"), "w") as f:
        f.write(log)
    with open(STAMP, "w") as f:
        f.write(source_hash() + "\n")
    build_call(force)
    if verbose:
        print(log)
    return SO


if __name__ == "__main__":
    build(force=True, verbose=True)
