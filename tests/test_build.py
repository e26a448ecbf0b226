"""What build.py makes and when, with compilers that only note what they are asked for."""
import os
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
COMPILER = """#!/bin/sh
echo "$(basename "$0") $*" >> "$BUILD_LOG"
[ -e "$BUILD_LOG.fail.$(basename "$0")" ] && exit 1
while [ $# -gt 0 ]; do [ "$1" = -o ] && : > "$2"; shift; done
exit 0
"""
HIDDEN = "import sys; sys.modules['torch'] = None; "


class Tree:
    """A copy of the sources in a folder of its own."""

    def __init__(self, path):
        self.path, self.log = path, str(path / "log")
        package = path / "mla_latent_kv_13_gb300"
        package.mkdir()
        for f in ("__init__.py", "build.py"):
            shutil.copy(os.path.join(ROOT, "mla_latent_kv_13_gb300", f), package)
        shutil.copytree(os.path.join(ROOT, "mla_latent_kv_13_gb300", "csrc"), package / "csrc")
        shutil.copytree(os.path.join(ROOT, "include"), path / "include")
        (path / "bin").mkdir()
        for name in ("nvcc", "g++"):
            (path / "bin" / name).write_text(COMPILER)
            (path / "bin" / name).chmod(0o755)
        self.library, self.binding = package / "libmla.so", package / "_binding.so"

    def fail(self, name):
        open(f"{self.log}.fail.{name}", "w").close()

    def build(self, before=""):
        """Runs the build; returns its exit status and what was compiled or linked."""
        if os.path.exists(self.log):
            os.remove(self.log)
        env = dict(os.environ, BUILD_LOG=self.log, NVCC=str(self.path / "bin" / "nvcc"),
                   PATH=f"{self.path / 'bin'}:{os.environ['PATH']}", PYTHONPATH=str(self.path))
        r = subprocess.run([sys.executable, "-c", before + "from mla_latent_kv_13_gb300 import "
                            "build; build.build()"], env=env, cwd=self.path, capture_output=True,
                           text=True)
        lines = open(self.log).read().splitlines() if os.path.exists(self.log) else []
        made = {os.path.basename(w) for line in lines
                for a, w in zip(line.split(), line.split()[1:]) if a == "-o"}
        return r.returncode, {m.split(".so")[0] + ".so" if ".so." in m else m for m in made}, r.stderr


@pytest.fixture
def tree(tmp_path):
    return Tree(tmp_path)


def test_everything_once(tree):
    rc, made, err = tree.build()
    assert rc == 0, err
    assert tree.library.exists() and tree.binding.exists()
    assert {"libmla.so", "_binding.so", "binding.o", "rows_tc.o"} <= made
    assert tree.build()[:2] == (0, set())


def test_the_library_needs_no_pytorch(tree):
    rc, made, err = tree.build(HIDDEN)
    assert rc == 0, err
    assert tree.library.exists() and not tree.binding.exists()
    assert "_binding.so" in err  # says what is not there
    assert tree.build(HIDDEN)[:2] == (0, set())
    # PyTorch comes later
    rc, made, err = tree.build()
    assert rc == 0, err
    assert tree.binding.exists() and made == {"binding.o", "_binding.so"}


def test_a_binding_that_fails_leaves_the_library(tree):
    tree.fail("g++")
    rc, _, err = tree.build()
    assert rc != 0 and "g++ failed" in err
    assert tree.library.exists() and not tree.binding.exists()


def test_a_library_that_fails_is_told(tree):
    tree.fail("nvcc")
    rc, _, err = tree.build()
    assert rc != 0 and "nvcc failed" in err
    assert not tree.library.exists() and not tree.binding.exists()


@pytest.mark.parametrize("source,want", [("binding.cpp", {"binding.o", "_binding.so"}),
                                         ("pages.cu", {"libmla.so", "pages.o", "rows_tc.o"})])
def test_a_changed_source_is_built_again(tree, source, want):
    assert tree.build()[0] == 0
    src = tree.path / "mla_latent_kv_13_gb300" / "csrc" / source
    later = os.path.getmtime(tree.binding) + 5
    os.utime(src, (later, later))
    rc, made, err = tree.build()
    assert rc == 0 and want <= made, err


def test_another_pytorch_or_python_gets_its_own_binding(tree):
    """The module is tied to the PyTorch that it was compiled against; the library is not."""
    assert tree.build()[0] == 0
    other = "import torch; torch.__version__ = '0.0.1'; "
    rc, made, err = tree.build(other)
    assert rc == 0 and made == {"binding.o", "_binding.so"}, err
    assert tree.build(other)[:2] == (0, set())
    other = "import sysconfig; sysconfig.get_config_vars()['SOABI'] = 'other'; "
    rc, made, err = tree.build(other)
    assert rc == 0 and made == {"binding.o", "_binding.so"}, err
