"""The library is built and loaded without the Python module, and the module is
built again for another torch or Python."""
import os
import subprocess
import sys

import pytest

from sequence_sharded_mla_gb300 import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

BROKEN = """
import sequence_sharded_mla_gb300 as mla
from sequence_sharded_mla_gb300 import build

def broken(obj):
    raise RuntimeError("no C++ headers")

build.BINDING = build.BINDING + ".missing"
build._binding_object = broken
assert mla.mla_version() > 0
assert mla.mla_workspace_size(2, 1, 16, 2) >= 0
try:
    mla.gqa_shard_combine(None, None)
except RuntimeError as e:
    assert "no C++ headers" in str(e)
else:
    raise AssertionError("answered without its module")
assert mla.mla_version() > 0
"""


def test_library_answers_where_the_module_cannot_be_built():
    build.build()
    r = subprocess.run([sys.executable, "-c", BROKEN], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


def test_module_is_built_again_for_another_torch(monkeypatch, tmp_path):
    build.build_binding()
    assert not build.needs_binding() and not build.needs_build()
    for text in ("torch 1.0 at /elsewhere, python 3", None):
        stamp = tmp_path / "built-for"
        if text is None:
            stamp.unlink()
        else:
            stamp.write_text(text)
        with monkeypatch.context() as m:
            m.setattr(build, "BINDING_STAMP", str(stamp))
            assert build.needs_binding() and not build.needs_build()
    with monkeypatch.context() as m:
        m.setattr(build, "_binding_for", lambda: "another Python")
        assert build.needs_binding()
    assert not build.needs_binding()


@pytest.mark.parametrize("which", ["LIB", "BINDING"])
def test_missing_parts_are_found(monkeypatch, tmp_path, which):
    build.build_binding()
    with monkeypatch.context() as m:
        m.setattr(build, which, str(tmp_path / "missing.so"))
        assert build.needs_build() == (which == "LIB")
        assert build.needs_binding() == (which == "BINDING")
