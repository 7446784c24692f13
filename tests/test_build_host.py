"""Building the library and its Python extension, on small sources of their own."""
import os
import shutil
import subprocess
import sys
import sysconfig

import pytest
import torch

from paged_kv_cache_write_gb300 import build as real

LIBRARY = 'extern "C" int pkv_answer() { return 42; }\n'
EXTENSION = """#include <Python.h>
static PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, nullptr};
PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
"""


class Tree:
    """The build script over a package of two files."""

    def __init__(self, root, extension=EXTENSION):
        self.pkg = root / "pkg"
        (self.pkg / "csrc").mkdir(parents=True)
        (root / "include").mkdir()
        (root / "include" / "pkv.h").write_text("")
        shutil.copy(real.__file__, self.pkg / "build.py")
        (self.pkg / "csrc" / "a.cu").write_text(LIBRARY)
        self.extension = self.pkg / "csrc" / "binding.cpp"
        self.extension.write_text(extension)

    def run(self, *flags):
        env = {k: v for k, v in os.environ.items() if k != "PYTHONPATH"}
        return subprocess.run([sys.executable, *flags, str(self.pkg / "build.py")], env=env, cwd=self.pkg,
                              stdout=subprocess.PIPE, stderr=subprocess.PIPE, text=True, timeout=300)

    @property
    def library(self):
        return self.pkg / "libpkv.so"

    def extensions(self):
        return sorted(self.pkg.glob("_binding*.so"))


@pytest.fixture
def tree(tmp_path):
    return Tree(tmp_path)


def test_both_are_built_once(tree):
    r = tree.run()
    assert r.returncode == 0, r.stderr
    assert tree.library.exists() and len(tree.extensions()) == 1
    stamps = [p.stat().st_mtime_ns for p in (tree.library, *tree.extensions())]
    assert tree.run().returncode == 0
    assert [p.stat().st_mtime_ns for p in (tree.library, *tree.extensions())] == stamps
    os.utime(tree.extension, ns=(stamps[1] + 10 ** 9,) * 2)  # the extension's source alone
    assert tree.run().returncode == 0
    assert tree.library.stat().st_mtime_ns == stamps[0]


def test_the_library_needs_no_pytorch(tree):
    """(-S: without the folder that PyTorch is installed in.)"""
    r = tree.run("-S")
    assert r.returncode == 0, r.stderr
    assert tree.library.exists() and not tree.extensions()
    assert "PyTorch is not installed" in r.stderr
    stamp = tree.library.stat().st_mtime_ns
    assert tree.run("-S").returncode == 0 and tree.library.stat().st_mtime_ns == stamp
    r = tree.run()  # PyTorch is there now
    assert r.returncode == 0 and len(tree.extensions()) == 1 and tree.library.stat().st_mtime_ns == stamp


def test_the_library_is_there_when_the_extension_fails(tmp_path):
    tree = Tree(tmp_path, extension="#error no headers for this\n")
    r = tree.run()
    assert r.returncode != 0 and "no headers for this" in r.stderr
    assert tree.library.exists() and not tree.extensions()
    stamp = tree.library.stat().st_mtime_ns
    r = tree.run()
    assert r.returncode != 0 and tree.library.stat().st_mtime_ns == stamp


def test_the_extension_belongs_to_an_interpreter_and_a_pytorch(tree):
    """Named after the one, built again for another version or other flags of the other."""
    assert tree.run().returncode == 0
    (made,) = tree.extensions()
    assert made.name == "_binding" + sysconfig.get_config_var("EXT_SUFFIX")
    library, stamp = tree.library.stat().st_mtime_ns, made.stat().st_mtime_ns
    assert tree.run().returncode == 0 and made.stat().st_mtime_ns == stamp
    kept = tree.pkg / "_build" / "binding.stamp"
    text = kept.read_text()
    assert torch.__version__ in text and sys.version in text
    kept.write_text(text.replace(torch.__version__, "1.0"))
    assert tree.run().returncode == 0
    assert made.stat().st_mtime_ns > stamp and tree.library.stat().st_mtime_ns == library
    assert kept.read_text() == text


def test_an_extension_for_another_pytorch_is_refused():
    """As an import in a process whose PyTorch says that it is another one."""
    real.build()
    code = ("import torch; torch.__version__ = '1.0'\n"
            "import paged_kv_cache_write_gb300 as pkv\n"
            "try:\n    pkv._load_binding()\nexcept ImportError as e:\n    print(e)\n")
    r = subprocess.run([sys.executable, "-c", code], cwd=os.path.dirname(os.path.dirname(real.__file__)),
                       stdout=subprocess.PIPE, stderr=subprocess.PIPE, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    assert f"built for PyTorch {torch.__version__}, this is 1.0" in r.stdout
