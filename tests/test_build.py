"""The library is built without torch and whatever becomes of the binding; the
binding is built again for another torch or Python."""
import os
import subprocess
import types

import pytest

from paged_kv_cache_06_gb300 import build as b


@pytest.fixture
def fake(tmp_path, monkeypatch):
    """Products in a folder of their own; compilers that only write their output file."""
    monkeypatch.setattr(b, "BUILD_DIR", str(tmp_path / "_build"))
    monkeypatch.setattr(b, "LIB_PATH", str(tmp_path / "libpagedkv.so"))
    monkeypatch.setattr(b, "BINDING_PATH", str(tmp_path / "_binding.so"))
    f = types.SimpleNamespace(ran=[], fails=None)

    def run(cmd, **kw):
        f.ran.append(cmd)
        bad = f.fails and any(f.fails in str(x) for x in cmd)
        if not bad:
            open(cmd[cmd.index("-o") + 1], "w").close()
        return subprocess.CompletedProcess(cmd, int(bool(bad)), "", "no such header" if bad else "")

    monkeypatch.setattr(subprocess, "run", run)
    return f


def compiled(f):
    return {os.path.basename(cmd[cmd.index("-c") + 1]) for cmd in f.ran if "-c" in cmd}


def no_torch(monkeypatch):
    find = __import__("importlib.util").util.find_spec
    monkeypatch.setattr("importlib.util.find_spec", lambda name, *a: None if name == "torch" else find(name, *a))


def test_the_library_needs_no_torch(fake, monkeypatch):
    no_torch(monkeypatch)
    assert b.build() == b.LIB_PATH
    assert os.path.exists(b.LIB_PATH) and not os.path.exists(b.BINDING_PATH)
    assert "binding.cpp" not in compiled(fake) and "tree.cu" in compiled(fake)
    assert not b.is_stale()


def test_a_binding_that_does_not_compile_leaves_the_library(fake):
    fake.fails = "binding.cpp"
    with pytest.raises(RuntimeError, match="binding.cpp"):
        b.build()
    assert os.path.exists(b.LIB_PATH) and not os.path.exists(b.BINDING_PATH)


def test_another_torch_or_python_means_another_binding(fake, monkeypatch):
    b.build()
    assert os.path.exists(b.BINDING_PATH) and not b.is_stale()
    fake.ran.clear()
    b.build()
    assert not fake.ran
    for what, other in (("sys.version", "3.99"), ("sysconfig.get_config_var", lambda name: "other")):
        with monkeypatch.context() as m:
            m.setattr(what, other)
            assert b.is_stale()
    torch_dir = os.path.join(os.path.dirname(b.LIB_PATH), "torch")
    os.makedirs(torch_dir)
    with open(os.path.join(torch_dir, "version.py"), "w") as f:
        f.write("__version__ = '99'\n")
    monkeypatch.setattr(b, "_torch_dir", lambda: torch_dir)
    assert b.is_stale()
    b.build()
    assert compiled(fake) == {"binding.cpp"}          # the library stays
    assert not b.is_stale()
