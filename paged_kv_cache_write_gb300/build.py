"""Build libpkv.so (the C-ABI library) in-tree for sm_103a with nvcc, and
_binding, the CPython extension over some of its entries.

Each .cu translation unit is compiled in parallel to an object under
``_build/``, then linked into ``libpkv.so`` next to this file.  The CUDA
runtime is linked statically, so the library depends only on the driver.
``_binding.<ABI>.so`` (csrc/binding.cpp) is compiled beside them with the host
compiler against the installed PyTorch's headers, and links to ``libpkv.so``.  It
holds for that interpreter and that PyTorch only: it is named after the one, knows
the other's version, and is built again when what it was built with has changed.
The library alone, for users of the C ABI, needs neither PyTorch nor Python's
headers: run this file as a script.

    python -m paged_kv_cache_write_gb300.build [--force] [--verbose]
"""
from __future__ import annotations

import argparse
import importlib.util
import os
import re
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libpkv.so")
BINDING = os.path.join(HERE, "_binding" + sysconfig.get_config_var("EXT_SUFFIX"))
BINDING_STAMP = os.path.join(BUILD, "binding.stamp")  # the commands that made it

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
    """What the library is built from, and what the extension is besides it."""
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f != "binding.cpp"]
    files += [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE)]
    files.append(os.path.abspath(__file__))
    return files


def _newer(target, files) -> bool:
    """Whether the target exists and none of the files is newer."""
    if not os.path.exists(target):
        return False
    t = os.path.getmtime(target)
    return all(os.path.getmtime(f) <= t for f in files)


def library_up_to_date() -> bool:
    return _newer(LIB, _deps())


def binding_up_to_date() -> bool:
    torch = _torch()
    if torch is None or not _newer(BINDING, [os.path.join(CSRC, "binding.cpp"), *_deps()]):
        return False
    try:
        with open(BINDING_STAMP) as f:
            return f.read() == _stamp(torch)
    except OSError:
        return False


def up_to_date() -> bool:
    return library_up_to_date() and (_torch() is None or binding_up_to_date())


def _torch():
    """PyTorch's folder, or None where it is not installed."""
    spec = importlib.util.find_spec("torch")
    return spec.submodule_search_locations[0] if spec and spec.submodule_search_locations else None


def _torch_version(torch):
    """torch.__version__, without importing it."""
    with open(os.path.join(torch, "version.py")) as f:
        found = re.search(r"""^__version__\s*=\s*['"]([^'"]*)['"]""", f.read(), re.M)
    if found is None:
        raise RuntimeError(f"no version in {torch}/version.py")
    return found.group(1)


def _stamp(torch):
    return "\n".join([sys.version, *(" ".join(c) for c in _binding_commands(torch))])


def _binding_commands(torch):
    """Commands that compile and link the extension."""
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    obj = os.path.join(BUILD, "binding.o")
    cxx = os.environ.get("CXX", "g++")
    compile_ = [cxx, "-O2", "-std=c++17", "-fPIC", "-w", "-I", INCLUDE,
                f'-DPKV_TORCH_VERSION="{_torch_version(torch)}"',
                "-isystem", os.path.join(torch, "include"), "-isystem", os.path.join(cuda, "include"),
                "-isystem", sysconfig.get_paths()["include"], "-c", os.path.join(CSRC, "binding.cpp"),
                "-o", obj]
    link = [cxx, "-shared", "-o", BINDING + ".tmp", obj, LIB, "-Wl,-rpath,$ORIGIN",
            "-L", os.path.join(torch, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10_cuda", "-lc10"]
    return compile_, link


def _start(cmd, verbose):
    if verbose:
        print(" ".join(cmd), flush=True)
    return subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)


def _finish(p, verbose):
    """The process's return code and output."""
    text = p.communicate()[0].decode(errors="replace")
    if p.returncode == 0 and verbose and text.strip():
        print(text)
    return p.returncode, text


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    """Compile and link libpkv.so, and where PyTorch is installed the extension, if any
    source is newer; return the library's path.  The library needs nvcc alone, and is there
    whatever becomes of the extension: what fails in that is raised after it."""
    library = force or not library_up_to_date()
    torch = _torch()
    if torch is None:
        print("PyTorch is not installed: libpkv.so is built without the Python extension",
              file=sys.stderr)
    binding = torch is not None and (library or not binding_up_to_date())
    if not library and not binding:
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()
    procs = []
    objs = []
    for src in _sources() if library else []:
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        objs.append(obj)
        procs.append((src, _start([cc, *ARCH, *NVCC_FLAGS, *extra_flags, "-c", src, "-o", obj], verbose)))
    if binding:
        compile_binding, link_binding = _binding_commands(torch)
        compiling = _start(compile_binding, verbose)
    done = [(src, *_finish(p, verbose)) for src, p in procs]
    failed = [(src, text) for src, rc, text in done if rc]
    binding_rc, binding_text = _finish(compiling, verbose) if binding else (0, "")
    if failed:
        msg = "\n".join(f"--- {s}\n{t}" for s, t in failed)
        raise RuntimeError(f"compilation failed:\n{msg}")
    if library:
        tmp = LIB + ".tmp"
        cmd = [cc, *ARCH, "-shared", "-Xlinker", "-soname=libpkv.so", "-o", tmp, *objs]
        rc, text = _finish(_start(cmd, verbose), False)
        if rc:
            raise RuntimeError("nvcc link failed:\n" + text)
        os.replace(tmp, LIB)
    if binding and binding_rc == 0:
        binding_rc, binding_text = _finish(_start(link_binding, verbose), False)
    if binding_rc:
        raise RuntimeError(f"{LIB} is built, but its Python extension is not:\n{binding_text}")
    if binding:
        os.replace(BINDING + ".tmp", BINDING)
        with open(BINDING_STAMP, "w") as f:
            f.write(_stamp(torch))
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
