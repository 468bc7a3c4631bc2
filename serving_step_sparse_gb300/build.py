"""Build the CUDA library in-tree: csrc/*.cu -> _build/libula.so (sm_103a only), and the
binding of the operators on rows: csrc/rows_binding.cpp -> _build/_rows.so.

Translation units compile in parallel, then link into one shared library that
exports the C ABI declared in include/ula.h; the binding (a Python extension module
against torch's headers) links with it.  The library needs no torch: where that or its headers
are missing, the library alone is built.
"""
from __future__ import annotations

import importlib.util
import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
OUT_DIR = os.path.join(HERE, "_build")
LIB = os.path.join(OUT_DIR, "libula.so")
BINDING = os.path.join(OUT_DIR, "_rows.so")
SOURCES = ["ula_kernels.cu", "ula_api.cu", "ula_noalloc.cu", "ula_rows.cu", "ula_attend.cu"]
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
         "--expt-relaxed-constexpr", "-I", os.path.join(ROOT, "include"), "-I", CSRC]


def _deps():
    return [os.path.join(CSRC, f) for f in os.listdir(CSRC)] + [os.path.join(ROOT, "include", "ula.h")]


def _torch_dir() -> str | None:
    """Where torch is installed, if it has what the binding is built from (found without importing it)."""
    spec = importlib.util.find_spec("torch")
    for d in (spec.submodule_search_locations or []) if spec else []:
        if all(os.path.exists(os.path.join(d, *f)) for f in (("include", "ATen", "core", "Tensor.h"),
                                                             ("lib", "libtorch_cuda.so"))):
            return d
    return None


def up_to_date() -> bool:
    made = [LIB] + ([BINDING] if _torch_dir() else [])
    if not all(os.path.exists(f) for f in made):
        return False
    t = min(os.path.getmtime(f) for f in made)
    return all(os.path.getmtime(d) <= t for d in _deps())


CXX = os.environ.get("CXX", "g++")


def _binding_flags() -> list[str]:
    import sysconfig

    import torch
    from torch.utils.cpp_extension import include_paths
    flags = ["-O2", "-std=c++17", "-fPIC", "-Wall",
             f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
             "-I", os.path.join(ROOT, "include"), "-isystem", sysconfig.get_paths()["include"],
             "-isystem", os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(NVCC))), "include")]
    for p in include_paths():
        flags += ["-isystem", p]
    return flags


def _link_binding(obj: str) -> None:
    """Links with the library beside it and with torch's libraries."""
    import torch
    tmp = BINDING + f".{os.getpid()}.tmp"
    subprocess.run([CXX, "-shared", "-o", tmp, obj, "-L", OUT_DIR, "-l:libula.so",
                    "-L", os.path.join(os.path.dirname(torch.__file__), "lib"), "-ltorch_python",
                    "-ltorch_cuda", "-ltorch_cpu", "-ltorch", "-lc10_cuda", "-lc10",
                    "-Wl,-rpath,$ORIGIN"], check=True)
    os.replace(tmp, BINDING)


def build(force: bool = False, verbose: bool = False, extra: list[str] | None = None) -> str:
    if not force and up_to_date():
        return LIB
    os.makedirs(OUT_DIR, exist_ok=True)
    procs, objs = [], []
    for src in SOURCES:
        obj = os.path.join(OUT_DIR, src.replace(".cu", ".o"))
        cmd = [NVCC, *ARCH, *FLAGS, *(extra or []), "-c", os.path.join(CSRC, src), "-o", obj]
        if verbose:
            print(" ".join(cmd), file=sys.stderr)
        procs.append((src, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
        objs.append(obj)
    binding = None
    if _torch_dir():
        binding = os.path.join(OUT_DIR, "rows_binding.o")
        cmd = [CXX, *_binding_flags(), "-c", os.path.join(CSRC, "rows_binding.cpp"), "-o", binding]
        if verbose:
            print(" ".join(cmd), file=sys.stderr)
        procs.append(("rows_binding.cpp", subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
    else:
        print("torch or its headers not found: the binding of the operators on rows is not built", file=sys.stderr)
    failed = {}
    for src, p in procs:
        out, _ = p.communicate()
        if p.returncode:
            failed[src] = out.decode(errors="replace")
        elif verbose and out:
            print(out.decode(errors="replace"), file=sys.stderr)
    if not failed.keys() & set(SOURCES):  # the library does not wait for the binding
        tmp = LIB + f".{os.getpid()}.tmp"
        subprocess.run([NVCC, *ARCH, "-shared", "-cudart", "shared", "-o", tmp, *objs], check=True)
        os.replace(tmp, LIB)
    if failed:
        raise RuntimeError("compilation failed:\n" + "\n".join(f"--- {s}\n{o}" for s, o in failed.items()))
    if binding:
        _link_binding(binding)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True,
                extra=["-Xptxas", "-v"] if "--ptxas" in sys.argv else None))
