"""The library and the binding of its rotary and paged calls are built and loaded apart: the calls that do
without the binding need neither it nor what it is built with."""
import os
import subprocess
import sys

import pytest

from sparse_long_context_cca_gb300 import build as cbuild


@pytest.fixture(scope="module")
def built():
    cbuild.build()


def run(code):
    return subprocess.run([sys.executable, "-c", code], cwd=cbuild.ROOT, capture_output=True, text=True, timeout=600)


def test_older_calls_do_without_the_binding(built):
    r = run("""
from sparse_long_context_cca_gb300 import api, build
build.BINDING = "/nowhere/_binding.so"
lib = api.load_library()
assert "invalid" in api.status_string(api.CCA_ERR_INVALID_ARG).lower()
assert api.decode_workspace_size(1, 2, 2, 1024, 128, 16, 64, __import__("torch").bfloat16) > 0
try:
    api.cca_pages_free(None, None, None, None)
except RuntimeError as e:
    assert "build it first" in str(e) and "/nowhere" in str(e), e
else:
    raise SystemExit("no error")
""")
    assert r.returncode == 0, r.stderr


def test_a_binding_for_another_torch_is_not_loaded(built, tmp_path, monkeypatch):
    mark = tmp_path / "binding_for"
    mark.write_text("torch 1.0, Python 3.0")
    monkeypatch.setattr(cbuild, "BINDING_FOR", str(mark))
    assert not cbuild.binding_is_for_this_torch()
    r = run(f"""
from sparse_long_context_cca_gb300 import api, build
build.BINDING_FOR = {str(mark)!r}
api.load_library()
try:
    api.cca_pages_free(None, None, None, None)
except RuntimeError as e:
    assert "another torch" in str(e), e
else:
    raise SystemExit("no error")
import sys
assert "sparse_long_context_cca_gb300._binding" not in sys.modules
""")
    assert r.returncode == 0, r.stderr


def test_it_is_built_again_for_another_torch(tmp_path, monkeypatch):
    """Only the binding: the library is up to date."""
    for name in ("LIB", "BINDING", "BINDING_FOR"):
        monkeypatch.setattr(cbuild, name, str(tmp_path / name))
        (tmp_path / name).write_text("torch 1.0, Python 3.0")
    monkeypatch.setattr(cbuild, "BUILD", str(tmp_path))
    monkeypatch.setattr(cbuild, "_binding_command", lambda out: ["cp", cbuild.LIB, out])
    monkeypatch.setattr(cbuild, "SOURCES", ["no_such_file.cu"])
    cbuild.build()
    assert cbuild.binding_is_for_this_torch() and (tmp_path / "LIB").read_text() == "torch 1.0, Python 3.0"


def test_the_library_is_built_where_the_binding_cannot_be(tmp_path, monkeypatch):
    for name in ("LIB", "BINDING", "BINDING_FOR"):
        monkeypatch.setattr(cbuild, name, str(tmp_path / name))
    monkeypatch.setattr(cbuild, "BUILD", str(tmp_path))
    monkeypatch.setattr(cbuild, "SOURCES", ["pages.cu"])
    monkeypatch.setattr(cbuild, "_binding_command", lambda out: ["false"])
    with pytest.raises(RuntimeError, match="binding failed"):
        cbuild.build()
    assert os.path.exists(cbuild.LIB) and not os.path.exists(cbuild.BINDING) and not cbuild.binding_is_for_this_torch()
