"""Build libpkv.so (the C-ABI library) in-tree for sm_103a with nvcc, and
_binding.so, the CPython extension over some of its entries.

Each .cu translation unit is compiled in parallel to an object under
``_build/``, then linked into ``libpkv.so`` next to this file.  The CUDA
runtime is linked statically, so the library depends only on the driver.
``_binding.so`` (csrc/binding.cpp) is compiled beside them with the host
compiler against the installed PyTorch's headers, and links to ``libpkv.so``.

    python -m paged_kv_cache_write_gb300.build [--force] [--verbose]
"""
from __future__ import annotations

import argparse
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libpkv.so")
BINDING = os.path.join(HERE, "_binding.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-O3",
              "--expt-relaxed-constexpr", "-I", INCLUDE]


def nvcc() -> str:
    path = shutil.which("nvcc")
    if path is None:
        cand = "/usr/local/cuda/bin/nvcc"
        if os.path.exists(cand):
            return cand
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libpkv.so")
    return path


def _sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _deps():
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    files += [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE)]
    files.append(os.path.abspath(__file__))
    return files


def up_to_date() -> bool:
    if not os.path.exists(LIB) or not os.path.exists(BINDING):
        return False
    t = min(os.path.getmtime(LIB), os.path.getmtime(BINDING))
    return all(os.path.getmtime(f) <= t for f in _deps())


def _binding_commands():
    """Commands that compile and link _binding.so."""
    torch = importlib.util.find_spec("torch").submodule_search_locations[0]
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    obj = os.path.join(BUILD, "binding.o")
    cxx = os.environ.get("CXX", "g++")
    compile_ = [cxx, "-O2", "-std=c++17", "-fPIC", "-w", "-I", INCLUDE,
                "-isystem", os.path.join(torch, "include"), "-isystem", os.path.join(cuda, "include"),
                "-isystem", sysconfig.get_paths()["include"], "-c", os.path.join(CSRC, "binding.cpp"),
                "-o", obj]
    link = [cxx, "-shared", "-o", BINDING + ".tmp", obj, LIB, "-Wl,-rpath,$ORIGIN",
            "-L", os.path.join(torch, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10_cuda", "-lc10"]
    return compile_, link


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    """Compile and link libpkv.so and _binding.so if any source is newer; return the
    library's path."""
    if not force and up_to_date():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()
    procs = []
    objs = []
    for src in _sources():
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        objs.append(obj)
        cmd = [cc, *ARCH, *NVCC_FLAGS, *extra_flags, "-c", src, "-o", obj]
        if verbose:
            print(" ".join(cmd), flush=True)
        procs.append((src, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
    compile_binding, link_binding = _binding_commands()
    if verbose:
        print(" ".join(compile_binding), flush=True)
    procs.append(("binding.cpp", subprocess.Popen(compile_binding, stdout=subprocess.PIPE,
                                                  stderr=subprocess.STDOUT)))
    failed = []
    for src, p in procs:
        out, _ = p.communicate()
        text = out.decode(errors="replace")
        if p.returncode != 0:
            failed.append((src, text))
        elif verbose and text.strip():
            print(text)
    if failed:
        msg = "\n".join(f"--- {s}\n{t}" for s, t in failed)
        raise RuntimeError(f"compilation failed:\n{msg}")
    tmp = LIB + ".tmp"
    cmd = [cc, *ARCH, "-shared", "-Xlinker", "-soname=libpkv.so", "-o", tmp, *objs]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)
    if r.returncode != 0:
        raise RuntimeError("nvcc link failed:\n" + r.stdout.decode(errors="replace"))
    os.replace(tmp, LIB)
    if verbose:
        print(" ".join(link_binding), flush=True)
    r = subprocess.run(link_binding, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)
    if r.returncode != 0:
        raise RuntimeError("link of the binding failed:\n" + r.stdout.decode(errors="replace"))
    os.replace(BINDING + ".tmp", BINDING)
    return LIB


def main(argv=None):
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose", action="store_true")
    ap.add_argument("--ptxas-info", action="store_true", help="print registers / spills per kernel")
    ap.add_argument("--nvtx", action="store_true",
                    help="push an NVTX range in every entry point (for profiler timelines)")
    a = ap.parse_args(argv)
    extra = ["-Xptxas", "-v"] if a.ptxas_info else []
    if a.nvtx:
        extra.append("-DPKV_NVTX")
    path = build(force=a.force or a.ptxas_info or a.nvtx, verbose=a.verbose or a.ptxas_info,
                 extra_flags=extra)
    print(path)


if __name__ == "__main__":
    sys.exit(main())
