"""The library's build stands on its own: it imports nothing from tests/."""
from __future__ import annotations

import os
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PKG = "gated_deltanet_linear_20_b200"


@pytest.mark.parametrize("sources", [False, True], ids=["no tests/", "only tests/csrc"])
def test_build_needs_no_test_module(tmp_path, sources):
    """build() of a copy without tests/, or with its CUDA sources alone.  (The built
    libraries are copied with their times, so that nothing is compiled again.)"""
    import __graft_entry__ as entry
    entry.build()
    for name in (PKG, "include", "oracle") + (("tests/csrc",) if sources else ()):
        shutil.copytree(os.path.join(ROOT, name), tmp_path / name)
    shutil.copy2(os.path.join(ROOT, "__graft_entry__.py"), tmp_path)
    code = ("import sys, __graft_entry__ as g; g.build(); "
            "assert not any(m == 'tests' or m.startswith('tests.') for m in sys.modules); "
            f"import {PKG}.gdn as m; print(m.library_path)")
    env = {k: v for k, v in os.environ.items() if k != "PYTHONPATH"}
    out = subprocess.run([sys.executable, "-c", code], cwd=tmp_path, env=env, capture_output=True,
                         text=True, timeout=600)
    assert out.returncode == 0, out.stderr[-2000:]
    assert out.stdout.strip() == str(tmp_path / PKG / "libgdn_b200.so")


def test_smoke_needs_no_test_module():
    with open(os.path.join(ROOT, "__graft_entry__.py")) as f:
        source = f.read()
    assert "from tests" not in source and "import tests" not in source
