"""Builds libkvtc.so in-tree for sm_100a (nvcc cross-compiles without a GPU) and _marshal.so,
the binding's compiled half.

python -m bit_quantization_head_b200.build [--verbose]
"""
from __future__ import annotations

import concurrent.futures as cf
import hashlib
import importlib.util
import os
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(HERE, "libkvtc.so")
MARSHAL = os.path.join(HERE, "_marshal.so")
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
         "-I" + os.path.join(ROOT, "include")]

SOURCES = ["host_plan.cpp", "host_calibrate.cpp", "encode_append.cu", "encode_prefill.cu", "decode.cu", "decode_rope.cu", "decode_noalloc.cu", "step_tables.cu", "rope_append.cu", "raw_decode.cu", "raw_cross.cu"] + [f"decode_v{b}.cu" for b in range(2, 9)]


def _deps_hash(src):
    h = hashlib.sha256()
    for name in sorted(os.listdir(CSRC)):
        if name.endswith((".h", ".cuh")):
            h.update(open(os.path.join(CSRC, name), "rb").read())
    h.update(open(os.path.join(ROOT, "include", "kvtc.h"), "rb").read())
    h.update(open(os.path.join(CSRC, src), "rb").read())
    h.update(" ".join(ARCH + FLAGS).encode())
    return h.hexdigest()[:16]


def _compile(src, verbose):
    obj = os.path.join(BUILD, src + "." + _deps_hash(src) + ".o")
    if os.path.exists(obj):
        return obj, ""
    cmd = [NVCC] + ARCH + FLAGS + ["-c", os.path.join(CSRC, src), "-o", obj + ".tmp"]
    if src.endswith(".cu") and verbose:
        cmd += ["-Xptxas", "-v"]
    if src.endswith(".cpp"):
        cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-Wall", "-I" + os.path.join(ROOT, "include"),
               "-I/usr/local/cuda/include", "-c", os.path.join(CSRC, src), "-o", obj + ".tmp"]
    p = subprocess.run(cmd, capture_output=True, text=True)
    if p.returncode != 0:
        raise RuntimeError(f"compile failed: {src}\n{p.stdout}\n{p.stderr}")
    os.replace(obj + ".tmp", obj)
    return obj, p.stdout + p.stderr


def _build_marshal():
    """The binding's compiled half (csrc/marshal.cpp): a CPython module against torch."""
    spec = importlib.util.find_spec("torch")
    if spec is None:
        raise RuntimeError("torch is not installed")
    torch_dir = spec.submodule_search_locations[0]
    src = os.path.join(CSRC, "marshal.cpp")
    h = hashlib.sha256()
    for path in (src, os.path.join(ROOT, "include", "kvtc.h"), os.path.join(torch_dir, "version.py")):
        h.update(open(path, "rb").read())
    h.update(sys.version.encode())
    out = os.path.join(BUILD, f"_marshal.{h.hexdigest()[:16]}.so")
    if not os.path.exists(out):
        inc = os.path.join(torch_dir, "include")
        cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall", "-I" + os.path.join(ROOT, "include"),
               "-I" + sysconfig.get_paths()["include"], "-isystem", inc, "-isystem",
               os.path.join(inc, "torch", "csrc", "api", "include"), "-isystem", "/usr/local/cuda/include", src, "-o",
               out + ".tmp", "-L" + os.path.join(torch_dir, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10_cuda", "-lc10"]
        p = subprocess.run(cmd, capture_output=True, text=True)
        if p.returncode != 0:
            raise RuntimeError(f"compile failed: marshal.cpp\n{p.stdout}\n{p.stderr}")
        os.replace(out + ".tmp", out)
    with open(out, "rb") as f:
        data = f.read()
    with open(MARSHAL + ".tmp", "wb") as f:
        f.write(data)
    os.replace(MARSHAL + ".tmp", MARSHAL)


def build(verbose=False):
    os.makedirs(BUILD, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=max(2, os.cpu_count() or 2)) as ex:
        marshal = ex.submit(_build_marshal)
        results = list(ex.map(lambda s: _compile(s, verbose), SOURCES))
        marshal_error = marshal.exception()
    objs = [r[0] for r in results]
    if verbose:
        for (o, log), s in zip(results, SOURCES):
            if log.strip():
                print(f"--- {s}\n{log}")
    tmp = LIB + ".tmp"
    cmd = [NVCC] + ARCH + ["-shared", "-o", tmp] + objs + ["-lpthread"]
    p = subprocess.run(cmd, capture_output=True, text=True)
    if p.returncode != 0:
        raise RuntimeError(f"link failed\n{p.stdout}\n{p.stderr}")
    os.replace(tmp, LIB)
    if marshal_error is not None:
        # The library stands without it (a user of the C interface needs neither torch's headers
        # nor Python's); one of an earlier build must not be bound to this library.
        if os.path.exists(MARSHAL):
            os.remove(MARSHAL)
        raise RuntimeError("libkvtc.so is built, the binding's compiled half (kvtc_step_tables and the calls "
                           f"after it in kvtc.py) is not: {marshal_error}") from marshal_error
    return LIB


if __name__ == "__main__":
    print(build(verbose="--verbose" in sys.argv))
