"""Build the C-ABI shared library in-tree with nvcc for sm_100a.

    python -m sparse_mla_decode_front_b200.build

compiles every ``csrc/*.cu`` into ``libsparse_mla_decode.so`` next to this
file (cudart linked statically), and ``csrc/bind.cpp`` (g++, against torch's
headers) into ``_bind.so``, the experts binding's native argument checks.
Rebuilds only when a source is newer, and ``_bind.so`` also when torch or
Python is another one than it was built for.
"""
from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
LIB = os.path.join(HERE, "libsparse_mla_decode.so")
BIND = os.path.join(HERE, "_bind.so")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]


def nvcc() -> str:
    for c in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if c and os.path.exists(c):
            return c
    raise RuntimeError("nvcc not found")


def sources():
    return sorted(glob.glob(os.path.join(HERE, "csrc", "*.cu")))


def deps():
    return sources() + glob.glob(os.path.join(HERE, "csrc", "*.cuh")) + \
        glob.glob(os.path.join(HERE, "csrc", "*.h")) + glob.glob(os.path.join(ROOT, "include", "*.h"))


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(f) <= t for f in deps())


def build_bind(force: bool = False, verbose: bool = False) -> str:
    """``_bind.so``: it calls the library through addresses it is given, and links torch only."""
    src = os.path.join(HERE, "csrc", "bind.cpp")
    used = [src, os.path.join(ROOT, "include", "moe_experts.h")]
    from ._lib import bind_tag
    tag, tag_file = bind_tag(), os.path.join(HERE, "_build", "bind.tag")   # what the last _bind.so was built for
    if not force and os.path.exists(BIND) and all(os.path.getmtime(f) <= os.path.getmtime(BIND) for f in used):
        try:
            with open(tag_file) as f:
                if f.read() == tag:
                    return BIND
        except OSError:
            pass
    import torch
    site = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    include = [sysconfig.get_paths()["include"], os.path.join(site, "include"),
               os.path.join(site, "include", "torch", "csrc", "api", "include"), os.path.join(cuda, "include")]
    tmp = BIND + ".tmp"
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", f'-DBIND_TAG="{tag}"', "-I", os.path.join(ROOT, "include"),
           *[a for d in include for a in ("-isystem", d)], src, "-o", tmp, "-L" + os.path.join(site, "lib"),
           "-lc10", "-lc10_cuda", "-ltorch", "-ltorch_cpu", "-ltorch_python"]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    os.replace(tmp, BIND)
    os.makedirs(os.path.dirname(tag_file), exist_ok=True)
    with open(tag_file, "w") as f:
        f.write(tag)
    return BIND


def build(force: bool = False, verbose: bool = False, extra=()) -> str:
    """The library, which needs nvcc alone, and then the Python binding's native part."""
    lib = build_lib(force, verbose, extra)
    build_bind(force, verbose)
    return lib


def build_lib(force: bool = False, verbose: bool = False, extra=()) -> str:
    if not force and up_to_date():
        return LIB
    out_dir = os.path.join(HERE, "_build")
    os.makedirs(out_dir, exist_ok=True)
    objs = []
    common = [nvcc(), *ARCH, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
              "-I", os.path.join(ROOT, "include"), "--expt-relaxed-constexpr", *extra]
    procs = []
    for src in sources():
        obj = os.path.join(out_dir, os.path.basename(src)[:-3] + ".o")
        objs.append(obj)
        cmd = common + ["-c", src, "-o", obj]
        if verbose:
            print(" ".join(cmd), flush=True)
        procs.append((src, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
    failed = []
    for src, p in procs:
        out, _ = p.communicate()
        if out and (verbose or p.returncode):
            sys.stderr.write(out.decode())
        if p.returncode:
            failed.append(src)
    if failed:
        raise RuntimeError("nvcc failed for: " + ", ".join(failed))
    tmp = LIB + ".tmp"
    cmd = [nvcc(), *ARCH, "-shared", "-o", tmp, *objs]
    subprocess.run(cmd, check=True)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
