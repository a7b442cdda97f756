"""What build() compiles and when, with the compilers replaced by a recorder: the
library without torch, the torch entry points again for another torch or Python."""
import importlib.util
import os
from types import SimpleNamespace

import pytest

from mxfp4_precision_gb300 import _block
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
    monkeypatch.setattr(mxbuild, "TORCH_STAMP", str(tmp_path / "stamp"), raising=False)
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
ENTRY = ["mx_torch.o", "mx_torch.so"]


def test_the_library_builds_without_torch(calls):
    calls.torch = None
    assert mxbuild.build() == mxbuild.LIB
    assert _sorted(calls) == LIBRARY
    mxbuild.build()
    assert _sorted(calls) == []


def test_entry_points_are_built_again_for_another_torch_or_python(calls, monkeypatch):
    mxbuild.build()
    assert _sorted(calls) == sorted(LIBRARY + ENTRY)
    mxbuild.build()
    assert _sorted(calls) == []
    stamp = os.stat(calls.version).st_mtime
    calls.version.write_text("__version__ = '2'\n")
    os.utime(calls.version, (stamp - 1000, stamp - 1000))       # an older release's older file
    mxbuild.build()
    assert _sorted(calls) == ENTRY
    abi = mxbuild.sysconfig.get_config_var
    monkeypatch.setattr(mxbuild.sysconfig, "get_config_var", lambda n: "cpython-399-none" if n == "SOABI" else abi(n))
    mxbuild.build()
    assert _sorted(calls) == ENTRY
    mxbuild.build()
    assert _sorted(calls) == []


def test_entry_points_of_another_torch_are_not_loaded(calls, monkeypatch):
    mxbuild.build()
    calls.version.write_text("__version__ = '2'\n")
    monkeypatch.setattr(_block, "_calls", None)
    monkeypatch.setattr(_block, "TORCH_LIB", mxbuild.TORCH_LIB)
    with pytest.raises(RuntimeError, match="another torch or Python"):
        _block._load()
