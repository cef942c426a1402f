"""What the build makes where PyTorch is missing, has no CUDA or changes: the
compilers are replaced by a stand-in that only writes the files asked for."""
import os
import subprocess

import pytest

from attention_backward_sm_gb300 import build as b


class Compilers:
    def __init__(self):
        self.calls, self.fail = [], ()

    def run(self, cmd, **kw):
        self.calls.append(os.path.basename(cmd[0]))
        if any(f in " ".join(cmd) for f in self.fail):
            return subprocess.CompletedProcess(cmd, 1, "", "no such header")
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("made")
        return subprocess.CompletedProcess(cmd, 0, "", "")


@pytest.fixture
def compilers(monkeypatch, tmp_path):
    c = Compilers()
    monkeypatch.setattr(subprocess, "run", c.run)
    for name, path in (("LIB", "libfabwd.so"), ("HOST", "_paged_host.so"), ("BUILD", "build"),
                       ("HOST_TAG", "build/host_torch")):
        monkeypatch.setattr(b, name, str(tmp_path / path))
    return c


def torch_at(monkeypatch, path):
    """Lets the build find a PyTorch in this folder (None: none)."""
    class Spec:
        submodule_search_locations = [str(path)]

    monkeypatch.setattr(b.importlib.util, "find_spec", lambda name: None if path is None else Spec)


def fake_torch(path, version, cuda=True):
    os.makedirs(path / "lib", exist_ok=True)
    (path / "version.py").write_text(version)
    if cuda:
        (path / "lib" / "libc10_cuda.so").write_text("")
    return path


@pytest.mark.parametrize("kind", ["missing", "without CUDA"])
def test_library_alone_without_a_pytorch_that_has_cuda(compilers, monkeypatch, tmp_path, kind):
    torch_at(monkeypatch, None if kind == "missing" else fake_torch(tmp_path / "torch", "1", cuda=False))
    assert b.build() == b.LIB and os.path.exists(b.LIB) and not os.path.exists(b.HOST)
    assert "g++" not in compilers.calls and compilers.calls.count("nvcc") == len(b.SOURCES) + 1
    compilers.calls.clear()
    b.build()
    assert compilers.calls == []


def test_library_is_made_where_the_extension_fails(compilers, monkeypatch, tmp_path):
    torch_at(monkeypatch, fake_torch(tmp_path / "torch", "1"))
    compilers.fail = (b.HOST_SOURCE,)
    with pytest.raises(RuntimeError, match="no such header"):
        b.build()
    assert os.path.exists(b.LIB) and not os.path.exists(b.HOST)
    compilers.fail = ()
    compilers.calls.clear()
    b.build()
    assert os.path.exists(b.HOST) and "nvcc" not in compilers.calls


def test_extension_is_remade_for_another_pytorch_or_python(compilers, monkeypatch, tmp_path):
    torch_at(monkeypatch, fake_torch(tmp_path / "torch", "1"))
    b.build()
    assert os.path.exists(b.LIB) and os.path.exists(b.HOST)
    for change in ("nothing", "torch", "python"):
        compilers.calls.clear()
        if change == "torch":
            fake_torch(tmp_path / "torch", "2")
        if change == "python":
            monkeypatch.setattr(b.sysconfig, "get_config_var", lambda name: ".cpython-399.so")
        b.build()
        assert compilers.calls == ([] if change == "nothing" else ["g++", "g++"]), change


def test_entry_build_imports_the_extension(monkeypatch):
    """An extension that cannot be imported shows at the build."""
    import __graft_entry__ as entry
    from attention_backward_sm_gb300 import paged
    entry.build()
    monkeypatch.setattr(paged, "_native", None)
    monkeypatch.setitem(__import__("sys").modules, "attention_backward_sm_gb300._paged_host", None)
    monkeypatch.delattr("attention_backward_sm_gb300._paged_host", raising=False)
    with pytest.raises(ImportError):
        entry.build()


def test_entry_build_without_the_extension(compilers, monkeypatch, tmp_path):
    """Beside a PyTorch without CUDA the entry builds and loads the library."""
    import __graft_entry__ as entry
    import attention_backward_sm_gb300 as fab
    torch_at(monkeypatch, fake_torch(tmp_path / "torch", "1", cuda=False))
    loaded = []
    monkeypatch.setattr(fab, "lib", lambda: loaded.append(1))
    monkeypatch.setattr(fab.paged, "_host", lambda: pytest.fail("there is none"))
    entry.build()
    assert loaded and not os.path.exists(b.HOST)
