"""Importing the binding with parts of the build missing."""
import os
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PACKAGE = os.path.join(ROOT, "mla_latent_kv_13_gb300")


@pytest.fixture
def python(tmp_path):
    from mla_latent_kv_13_gb300 import build
    build.build()
    package = tmp_path / "mla_latent_kv_13_gb300"
    package.mkdir()
    for f in ("__init__.py", "mla.py"):
        shutil.copy(os.path.join(PACKAGE, f), package)

    def run(code, library=True, binding=None):
        if library:
            os.symlink(os.path.join(PACKAGE, "libmla.so"), package / "libmla.so")
        if binding is not None:
            (package / "_binding.so").write_bytes(binding)
        return subprocess.run([sys.executable, "-c", code], cwd=tmp_path, capture_output=True,
                              text=True, env=dict(os.environ, PYTHONPATH=str(tmp_path)))

    return run


@pytest.mark.parametrize("binding", [None, b"", b"not a library"])
def test_without_a_binding_the_other_calls_work(python, binding):
    r = python("""
import torch
from mla_latent_kv_13_gb300 import mla
assert mla.decode_plan(200, 128, 8192)[0] == 0
assert mla.decode_workspace_size(2, 16, 100) >= 256
assert mla.chunk_workspace_size(2, 2, 16, 100) >= 256
t = torch.zeros(2, dtype=torch.int32)
for call in (lambda: mla.chunk_attention(t, t, t, t, t, t, 9, 0.1, out=t, lse=t, workspace=t),
             lambda: mla.decode_attention_window(t, t, t, t, t, 9, 3, 0, 0.1, out=t, lse=t, workspace=t),
             lambda: mla.norm_rope_append(t, t, t, t, t, t, t, c_q=t, workspace=t),
             lambda: mla.pages_free(t, t, t, t, workspace=t),
             lambda: mla.pages_compact(t, t, t, [t], live=t, workspace=t)):
    try:
        call()
    except ImportError as e:
        assert "_binding.so" in str(e) and "mla_latent_kv_13_gb300.build" in str(e)
    else:
        raise AssertionError("went through")
""", binding=binding)
    assert r.returncode == 0, r.stderr


def test_without_the_library_nothing_does(python):
    r = python("from mla_latent_kv_13_gb300 import mla", library=False)
    assert r.returncode != 0 and "libmla.so not found" in r.stderr
