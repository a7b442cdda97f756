"""What build() compiles and when, with the compilers replaced by a recorder: the
library without torch."""
import importlib.util
import os
from types import SimpleNamespace

import pytest

from mxfp4_precision_gb300 import build as mxbuild


@pytest.fixture
def calls(tmp_path, monkeypatch):
    """The outputs of each compiler call, in order of their names; every call creates its output."""
    made = []

    def run(cmd, verbose=False):
        out = cmd[cmd.index("-o") + 1]
        open(out, "w").close()
        made.append(os.path.basename(out).split(".tmp")[0])

    torch = tmp_path / "torch"
    torch.mkdir()
    (torch / "version.py").write_text("__version__ = '1'\n")
    find = importlib.util.find_spec
    where = SimpleNamespace(origin=str(torch / "__init__.py"))
    monkeypatch.setattr(importlib.util, "find_spec", lambda n, *a: made.torch if n == "torch" else find(n, *a))
    for name, value in (("BUILD_DIR", tmp_path), ("LIB", tmp_path / "libmx.so"), ("TORCH_LIB", tmp_path / "mx_torch.so")):
        monkeypatch.setattr(mxbuild, name, str(value))
    monkeypatch.setattr(mxbuild, "_run", run)

    class Made(list):
        pass
    made = Made()
    made.torch, made.version = where, torch / "version.py"
    return made


def _sorted(made):
    out = sorted(made)
    made.clear()
    return out


LIBRARY = sorted([os.path.splitext(s)[0] + ".o" for s in mxbuild.SOURCES] + ["libmx.so"])


def test_the_library_builds_without_torch(calls):
    calls.torch = None
    assert mxbuild.build() == mxbuild.LIB
    assert _sorted(calls) == LIBRARY
    mxbuild.build()
    assert _sorted(calls) == []
