"""What the in-tree build needs and when it runs again."""
import os

import pytest

from non_uniform_paged_gb300 import _build


@pytest.fixture
def compilers(monkeypatch, tmp_path):
    """Compilers that only write their output file; the commands they were given."""
    commands = []

    class Done:
        returncode, stderr, stdout = 0, "", ""

    def run(cmd, **kw):
        commands.append([os.path.basename(cmd[0])] + list(cmd[1:]))
        open(cmd[cmd.index("-o") + 1], "wb").close()
        return Done

    monkeypatch.setattr(_build.subprocess, "run", run)
    monkeypatch.setattr(_build, "LIB", str(tmp_path / "libtg.so"))
    monkeypatch.setattr(_build, "PKG", str(tmp_path))
    monkeypatch.setattr(_build, "BUILD_DIR", str(tmp_path))
    return commands


def test_libtg_needs_no_torch(compilers, monkeypatch):
    """The C library is built, and stays current, without torch and without the module built against it."""
    monkeypatch.setattr(_build.importlib.util, "find_spec", lambda name: None)
    assert not _build.up_to_date()
    assert _build.build() == _build.LIB
    assert compilers and all(cmd[0] == os.path.basename(_build.nvcc()) for cmd in compilers)
    assert _build.up_to_date()
    n = len(compilers)
    _build.build()
    assert len(compilers) == n
    with pytest.raises(RuntimeError, match="torch"):
        _build.build_calls()


def test_calls_are_built_apart(compilers):
    assert not _build.calls_up_to_date()
    _build.build_calls()
    assert len(compilers) == 1 and not os.path.exists(_build.LIB)
    assert _build.calls_up_to_date()
    _build.build_calls()
    assert len(compilers) == 1
    _build.build_calls(force=True)
    assert len(compilers) == 2


def test_calls_belong_to_one_torch_and_one_python(compilers, monkeypatch, tmp_path):
    """Another torch, another place of it or another Python: the module is built for it, beside the first."""
    first = _build.build_calls()
    for version, place in (("9.9.1", "a"), ("9.9.2", "a"), ("9.9.2", "b")):
        where = tmp_path / place / "torch"
        where.mkdir(parents=True, exist_ok=True)
        (where / "version.py").write_text(f"__all__ = ['__version__']\n__version__ = '{version}'\n")
        monkeypatch.setattr(_build, "_torch_dir", lambda: str(where))
        assert not _build.calls_up_to_date()
        assert _build.build_calls() != first and _build.calls_up_to_date()
    config = _build.sysconfig.get_config_var
    monkeypatch.setattr(_build.sysconfig, "get_config_var",
                        lambda name: ".cpython-399-none.so" if name == "EXT_SUFFIX" else config(name))
    assert not _build.calls_up_to_date()
    assert os.path.basename(_build.calls_path()).endswith(".cpython-399-none.so")
    assert len(compilers) == 4 and os.path.exists(first)
