"""The C module that some calls pass their arguments through: the interpreter's
own file, and needed by those calls alone.  No GPU."""
from __future__ import annotations

import os
import subprocess
import sys
import sysconfig

import pytest

from paged_kv_cache_355_b200 import build

PKG = os.path.dirname(os.path.abspath(build.__file__))


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()


def test_its_file_belongs_to_this_interpreter():
    from paged_kv_cache_355_b200 import _binding as b

    assert os.path.basename(build.MARSHAL) == "_marshal" + sysconfig.get_config_var("EXT_SUFFIX")
    assert b.MARSHAL_PATH == build.MARSHAL == b._marshal.__file__


@pytest.mark.parametrize("stale", [False, True])
def test_the_other_calls_need_only_the_library(tmp_path, stale):
    """A package without the module, or with one that names no interpreter."""
    pkg = tmp_path / "paged_kv_cache_355_b200"
    pkg.mkdir()
    for name in os.listdir(PKG):
        if not name.startswith("_marshal") and name != "__pycache__":
            os.symlink(os.path.join(PKG, name), pkg / name)
    if stale:
        (pkg / "_marshal.so").write_bytes(b"of another interpreter")
    program = """
import torch, paged_kv_cache_355_b200 as pa
from paged_kv_cache_355_b200.block_manager import BlockManager
assert pa.__file__.startswith({root!r}), pa.__file__
assert BlockManager(4, 8).num_free() == 4
assert pa.pa_paged_attention_workspace_size(2, 8, 2, 128, 100, 16) >= 0
try:
    pa.pa_select_blocks(torch.zeros(1, 1, 1), torch.zeros(1, dtype=torch.int32), 8, 8, torch.zeros(1, 1, 3, dtype=torch.int32))
except ImportError as e:
    assert "_marshal" in str(e) and "is missing" in str(e), e
else:
    raise SystemExit("not refused")
""".format(root=str(tmp_path))
    got = subprocess.run([sys.executable, "-c", program], cwd=tmp_path, capture_output=True, text=True,
                         env=dict(os.environ, PYTHONPATH=str(tmp_path)))
    assert got.returncode == 0, got.stderr


def test_build_without_python_headers(tmp_path, monkeypatch, capsys):
    monkeypatch.setattr(build, "MARSHAL", str(tmp_path / "_marshal.so"))
    monkeypatch.setattr(build.sysconfig, "get_paths", lambda: {"include": str(tmp_path)})
    assert build.build() == build.LIB
    assert "no Python.h" in capsys.readouterr().err and not os.path.exists(build.MARSHAL)
