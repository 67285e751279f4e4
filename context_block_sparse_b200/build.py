"""Build libsplitkv.so in-tree with nvcc for sm_100a (B200).

    python context_block_sparse_b200/build.py [-v] [-f] [--ptxas]

(Run it as a script: importing the package itself needs the built library.)

Objects go to _build/ at the repository root; the shared library lands next
to this file so the Python binding finds it, and beside it the torch extension
_draft_ext.so (the bindings of the rotary and draft-tree calls; left out, with a note, where there is no
torch).  Only splitkv_* symbols are exported.  Nothing here needs a GPU: nvcc cross-compiles.
"""

from __future__ import annotations

import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libsplitkv.so")
EXT_SRC = os.path.join(PKG, "ext", "draft_ext.cpp")   # torch bindings of the rotary and draft-tree calls
EXT = os.path.join(PKG, "_draft_ext.so")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
COMMON = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC,-O3", "-I", INCLUDE, "-I", CSRC]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def sources():
    return sorted(f for f in os.listdir(CSRC) if f.endswith((".cu", ".cpp")))


def build(verbose: bool = False, force: bool = False, ptxas_info: bool = False) -> str:
    nvcc = _nvcc()
    os.makedirs(BUILD, exist_ok=True)
    headers = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".h", ".cuh"))]
    headers.append(os.path.join(INCLUDE, "splitkv.h"))
    newest_header = max(os.path.getmtime(h) for h in headers)
    objs = []
    for src in sources():
        path = os.path.join(CSRC, src)
        obj = os.path.join(BUILD, src + ".o")
        objs.append(obj)
        if (not force and os.path.exists(obj)
                and os.path.getmtime(obj) >= max(os.path.getmtime(path), newest_header)):
            continue
        cmd = [nvcc, *ARCH, *COMMON, "-c", path, "-o", obj]
        if src.endswith(".cu"):
            cmd.insert(1, "-Xptxas=-v")
        if verbose:
            print(" ".join(cmd), flush=True)
        res = subprocess.run(cmd, capture_output=True, text=True)
        if ptxas_info or res.returncode != 0:
            sys.stderr.write(res.stderr)
        if res.returncode != 0:
            raise subprocess.CalledProcessError(res.returncode, cmd)

    link = [nvcc, *ARCH, "-shared", "-o", LIB, *objs,
            "-Xlinker", "--version-script=" + os.path.join(CSRC, "exports.map"), "-lcuda"]
    if verbose:
        print(" ".join(link), flush=True)
    subprocess.run(link, check=True)
    build_ext(verbose, force)
    return LIB


def _torch_version():
    """The installed torch's version, or None (read without importing it)."""
    from importlib import metadata
    try:
        return metadata.version("torch")
    except metadata.PackageNotFoundError:
        return None


def build_ext(verbose: bool = False, force: bool = False):
    """The torch extension _draft_ext.so beside libsplitkv.so, which it links against: built again when its source, the
    header, this file, torch or the interpreter changed.  Without torch there is nothing to bind to: None, and a note."""
    newest = max(os.path.getmtime(f) for f in (EXT_SRC, os.path.join(INCLUDE, "splitkv.h"), os.path.abspath(__file__)))
    stamp = os.path.join(BUILD, "draft_ext.for")       # what the extension that is there was built for
    made_for = f"torch {_torch_version()}, python {sys.version}"
    if not force and os.path.exists(EXT) and os.path.getmtime(EXT) >= newest and os.path.exists(stamp):
        with open(stamp) as f:
            if f.read() == made_for:
                return EXT
    import sysconfig
    try:
        import torch
        from torch.utils import cpp_extension
    except ImportError as e:
        print(f"_draft_ext.so (the rotary and draft-tree calls from torch) is not built: {e}", file=sys.stderr)
        return None
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    cmd = [os.environ.get("CXX") or "g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-I", INCLUDE,
           "-I", sysconfig.get_paths()["include"], "-isystem", os.path.join(os.path.dirname(os.path.dirname(_nvcc())), "include")]
    for path in cpp_extension.include_paths():
        cmd += ["-isystem", path]
    cmd += [EXT_SRC, "-o", EXT, "-L", PKG, "-l:libsplitkv.so", "-Wl,-rpath,$ORIGIN", "-L", lib, "-lc10", "-lc10_cuda",
            "-ltorch_cpu", "-ltorch_python"]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    with open(stamp, "w") as f:
        f.write(made_for)
    return EXT


if __name__ == "__main__":
    build(verbose="-v" in sys.argv, force="-f" in sys.argv, ptxas_info="--ptxas" in sys.argv)
    print(LIB)
