"""Build of libengram.so (gfx950) in-tree with hipcc.

Usage: ``python hashed_gram_memory_tid2eid_amd/build_lib.py`` (run by path: importing
the package loads the library this script builds).  Compiles the single
device translation unit and the host sources to objects under ``_build/`` and
links ``hashed_gram_memory_tid2eid_amd/libengram.so``; beside it the Python binding's
extension module ``_tensor_args`` with g++ against the installed torch, whose object
layouts it inlines.  Always recompiles.

The library carries a hash of what it was built from (every source under
``csrc/`` and ``include/`` plus the compiler flags), readable with
``engram_build_id()``.  ``ensure_built()`` rebuilds whenever that hash differs
from the sources in the tree, so a stale library is never loaded.  The extension
module records its source, flags, torch and Python in the same way.
"""
from __future__ import annotations

import hashlib
import os
import re
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libengram.so")
EXT_SUFFIX = sysconfig.get_config_var("EXT_SUFFIX")  # names the Python it is for
TENSOR_ARGS = os.path.join(PKG, "_tensor_args" + EXT_SUFFIX)

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
ARCH = "gfx950"

COMMON = [
    f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC",
    # packed fp32 VALU ops stay off: the compiler's own scalar/float2 code only
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall", "-Wno-unused-function", "-I", os.path.join(ROOT, "include"),
]

SOURCES = ["engram_device.hip", "abi.cpp", "layout.cpp", "noalloc.cpp", "train.cpp", "serve.cpp"]
INCLUDE = os.path.join(ROOT, "include")
BUILD_ID_PREFIX = "engram-src-sha256:"
TENSOR_ARGS_FLAGS = ["-O2", "-std=c++17", "-fPIC", "-shared", "-Wall"]
TENSOR_ARGS_PREFIX = "tensor-args-sha256:"


def source_hash() -> str:
    """First 16 hex digits of a SHA-256 over every source file under csrc/ and
    include/ (relative path and bytes, in sorted order) and the compiler flags (paths
    inside the tree written relative to it)."""
    h = hashlib.sha256()
    for top in (CSRC, INCLUDE):
        for root, dirs, files in os.walk(top):
            dirs.sort()
            for f in sorted(files):
                if f.endswith((".hip", ".cpp", ".h", ".hpp", ".inc")):
                    path = os.path.join(root, f)
                    h.update(os.path.relpath(path, ROOT).encode())
                    with open(path, "rb") as fh:
                        h.update(fh.read())
    # the flags with the tree's own location taken out, so a copy of the tree elsewhere
    # (same sources, same flags) keeps the identity and its built library
    h.update(" ".join(COMMON).replace(ROOT, ".").encode())
    return h.hexdigest()[:16]


def built_hash(lib: str = LIB):
    """The source hash recorded in a built library, or None (missing, or built
    before the hash existed)."""
    return _recorded(lib, BUILD_ID_PREFIX)


def _recorded(path: str, prefix: str):
    if not os.path.exists(path):
        return None
    with open(path, "rb") as f:
        m = re.search(re.escape(prefix.encode()) + rb"([0-9a-f]{16})", f.read())
    return m.group(1).decode() if m else None


def tensor_args_identity() -> str:
    """First 16 hex digits of a SHA-256 over what _tensor_args is built from and for: its
    source, its flags, the torch and the Python."""
    import torch
    with open(os.path.join(CSRC, "tensor_args.cpp"), "rb") as f:
        h = hashlib.sha256(f.read())
    h.update("\0".join([*TENSOR_ARGS_FLAGS, str(torch.__version__), EXT_SUFFIX]).encode())
    return h.hexdigest()[:16]


def built_tensor_args(path: str = TENSOR_ARGS):
    """The identity recorded in a built _tensor_args, or None."""
    return _recorded(path, TENSOR_ARGS_PREFIX)


def tensor_args_command(out: str):
    """How _tensor_args is built: the torch libraries it names are those that `import torch`
    has loaded by the time it is imported."""
    import torch
    from torch.utils import cpp_extension
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    includes = [x for path in cpp_extension.include_paths() for x in ("-isystem", path)]
    defines = [f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", f'-DTENSOR_ARGS_TORCH="{torch.__version__}"',
               f'-DTENSOR_ARGS_ID="{TENSOR_ARGS_PREFIX}{tensor_args_identity()}"']
    return [os.environ.get("CXX", "g++"), *TENSOR_ARGS_FLAGS, *includes, "-I", sysconfig.get_paths()["include"], *defines,
            os.path.join(CSRC, "tensor_args.cpp"), "-o", out, "-L", lib, "-ltorch_python", "-ltorch_cpu", "-lc10"]


def build(verbose: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    sha = source_hash()
    cmd = tensor_args_command(TENSOR_ARGS + ".tmp")
    procs = [("tensor_args.cpp", subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT))]
    objs = []
    for src in SOURCES:
        obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
        objs.append(obj)
        lang = ["-x", "hip"]
        defs = [f'-DENGRAM_BUILD_ID="{BUILD_ID_PREFIX}{sha}"'] if src == "abi.cpp" else []
        cmd = [HIPCC, *COMMON, *defs, *lang, "-c", os.path.join(CSRC, src), "-o", obj]
        if verbose:
            print(" ".join(cmd), flush=True)
        procs.append((src, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
    failed = []
    for src, p in procs:
        out, _ = p.communicate()
        text = out.decode(errors="replace")
        # hipcc's host pass does not know the device-only target feature; that warning is noise
        lines = [ln for ln in text.splitlines() if "packed-fp32-ops" not in ln and ln.strip()]
        if p.returncode != 0:
            failed.append(src)
            print(text, file=sys.stderr)
        elif verbose and lines:
            print("\n".join(lines))
    if failed:
        raise RuntimeError(f"hipcc failed for {failed}")
    tmp = LIB + ".tmp"
    cmd = [HIPCC, f"--offload-arch={ARCH}", "-shared", "-fPIC", "-o", tmp, *objs]
    subprocess.run(cmd, check=True)
    os.replace(TENSOR_ARGS + ".tmp", TENSOR_ARGS)
    os.replace(tmp, LIB)
    return LIB


MFMA_CEILING_SRC = os.path.join(PKG, "calibrate", "mfma_ceiling.hip")
MFMA_CEILING_BIN = os.path.join(BUILD, "mfma_ceiling")


def build_mfma_ceiling() -> str:
    """Builds the matrix-core ceiling probe (a measurement program beside the
    library, run by `bench.py --mfma-ceiling`) and returns its path."""
    os.makedirs(BUILD, exist_ok=True)
    cmd = [HIPCC, *COMMON, MFMA_CEILING_SRC, "-o", MFMA_CEILING_BIN]
    out = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)
    if out.returncode != 0:
        print(out.stdout.decode(errors="replace"), file=sys.stderr)
        raise RuntimeError("hipcc failed for the matrix-core ceiling probe")
    return MFMA_CEILING_BIN


HBM_REFERENCE_SRC = os.path.join(PKG, "calibrate", "hbm_reference.hip")
HBM_REFERENCE_BIN = os.path.join(BUILD, "hbm_reference")


def build_hbm_reference() -> str:
    """Builds the HBM streaming-reference probe (a measurement program beside the
    library, run by `bench.py --hbm-reference`) and returns its path."""
    os.makedirs(BUILD, exist_ok=True)
    cmd = [HIPCC, *COMMON, HBM_REFERENCE_SRC, "-o", HBM_REFERENCE_BIN]
    out = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)
    if out.returncode != 0:
        print(out.stdout.decode(errors="replace"), file=sys.stderr)
        raise RuntimeError("hipcc failed for the HBM reference probe")
    return HBM_REFERENCE_BIN


def ensure_built() -> str:
    """Builds the library and the binding's extension module when one of them is
    missing or was built from other sources than the tree holds now, or the module
    for another torch or Python (compared by what is embedded in them); otherwise
    leaves the built ones in place."""
    if built_hash() == source_hash() and built_tensor_args() == tensor_args_identity():
        return LIB
    return build()


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
