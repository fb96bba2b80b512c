"""The build of the CUDA library depends on neither torch nor the binding's tensor module."""
import os
from types import SimpleNamespace

import pytest

from tile_centric_comm_gb300 import build as tdg_build


@pytest.fixture
def fake(monkeypatch, tmp_path):
    """The build with commands that only write their outputs; `fail` names a command that fails."""
    state = SimpleNamespace(fail=None, ran=[])

    def run(cmd, **kw):
        state.ran.append(os.path.basename(cmd[0]))
        if state.ran[-1] == state.fail:
            return SimpleNamespace(returncode=1, stdout="", stderr="no such header")
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("x")
        return SimpleNamespace(returncode=0, stdout="", stderr="")

    monkeypatch.setattr(tdg_build, "subprocess", SimpleNamespace(run=run))
    monkeypatch.setattr(tdg_build, "nvcc", lambda: "nvcc")
    monkeypatch.setattr(tdg_build, "BUILD", str(tmp_path))
    monkeypatch.setattr(tdg_build, "LIB", str(tmp_path / "libtdg.so"))
    return state


def test_builds_without_torch(fake, monkeypatch):
    find = tdg_build.importlib.util.find_spec
    monkeypatch.setattr(tdg_build.importlib.util, "find_spec", lambda name, *a: None if name == "torch" else find(name, *a))
    for _ in range(2):                     # from nothing, and up to date
        assert os.path.exists(tdg_build.build())
    assert "g++" not in fake.ran and fake.ran.count("nvcc") == len(tdg_build._sources()) + 1


@pytest.mark.parametrize("fail", ["g++", "missing"])
def test_library_is_linked_when_the_tensor_module_fails(fake, monkeypatch, fail):
    pytest.importorskip("torch")
    if fail == "g++":
        fake.fail = "g++"
    else:                                  # no g++ at all
        run = tdg_build.subprocess.run

        def absent(cmd, **kw):
            if cmd[0] == "g++":
                raise FileNotFoundError("g++")
            return run(cmd, **kw)
        monkeypatch.setattr(tdg_build, "subprocess", SimpleNamespace(run=absent))
    with pytest.warns(UserWarning, match="tensor checks were not built"):
        assert os.path.exists(tdg_build.build())
    with pytest.warns(UserWarning, match="tensor checks were not built"):
        tdg_build.build()                  # and says so again


def test_a_failing_kernel_is_an_error(fake):
    fake.fail = "nvcc"
    with pytest.raises(RuntimeError, match="nvcc failed"):
        tdg_build.build()
    assert not os.path.exists(tdg_build.LIB)


def _fresh_binding():
    """A second copy of the binding, which has not looked for the module yet."""
    import importlib.util
    spec = importlib.util.find_spec("tile_centric_comm_gb300.tdg")
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_binding_takes_the_module_of_its_own_torch_and_python():
    torch = pytest.importorskip("torch")
    tdg_build.build()
    path = tdg_build.tensors_path(torch.version.__version__)
    assert os.path.exists(path) and path == tdg_build.build_tensors()
    assert tdg_build.tensors_path("1.0") != path
    b = _fresh_binding()
    b._attn()
    assert b._rows is not b._checked_rows and b._table is not b._checked_table and b._flat is not b._checked_flat


def test_binding_checks_in_python_without_the_module(monkeypatch, tmp_path):
    torch = pytest.importorskip("torch")
    tdg_build.build()
    other = tmp_path / "tdg_tensors.so"                 # one of unknown versions is not touched
    other.write_text("x")
    monkeypatch.setattr(tdg_build, "tensors_path", lambda version: str(tmp_path / ("of-" + version)))
    b = _fresh_binding()
    b._attn()
    assert b._rows is b._checked_rows and b._table is b._checked_table and b._flat is b._checked_flat
    # and the calls go through them
    heap = SimpleNamespace(device=torch.device("cuda", 0), world=1, h=None)
    x = torch.zeros(1, 2, 128)
    with pytest.raises(TypeError, match="k: expected torch.bfloat16"):
        b.rope_append(heap, b.PagedCache(4, 16, 2, 128, 0, 1 << 16), None, x, x, None, None, None, None, None)
