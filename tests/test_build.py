"""The build: the CUDA library by itself, and a binding that belongs to the installed torch."""
import os

import pytest

from recurrent_state_memory_b200 import build, gdr


@pytest.fixture
def commands(monkeypatch, tmp_path):
    """Compiler calls are noted, and leave an empty file; nothing of the package's own is touched."""
    calls = []

    def run(cmd, check):
        calls.append(cmd)
        out = cmd[cmd.index("-o") + 1]
        open(out, "w").close()
        if "-MF" in cmd:
            open(cmd[cmd.index("-MF") + 1], "w").write(out + ":")

    monkeypatch.setattr(build.subprocess, "run", run)
    for name in ("LIB", "LIB_DEBUG", "BINDING"):
        monkeypatch.setattr(build, name, str(tmp_path / name.lower()))
    monkeypatch.setattr(build, "OBJ", str(tmp_path / "obj"))
    if hasattr(build, "BINDING_MADE_FOR"):
        monkeypatch.setattr(build, "BINDING_MADE_FOR", str(tmp_path / "obj" / "binding.txt"))
    return calls


def test_the_library_needs_no_binding(commands, monkeypatch):
    """Without a host compiler, or without torch's headers, libgdr.so is built all the same."""
    from torch.utils import cpp_extension
    before = build.subprocess.run

    def run(cmd, check):
        if cmd[0] == build.CXX:
            raise FileNotFoundError(build.CXX)
        before(cmd, check)

    monkeypatch.setattr(build.subprocess, "run", run)
    with pytest.warns(UserWarning, match="_binding.so is not built"):
        assert build.build() == build.LIB
    assert os.path.exists(build.LIB) and not os.path.exists(build.BINDING)
    os.remove(build.LIB)
    monkeypatch.setattr(cpp_extension, "include_paths", lambda *a, **k: [])
    with pytest.warns(UserWarning, match="torch/extension.h"):
        assert build.build() == build.LIB
    assert os.path.exists(build.LIB)


def test_a_binding_that_does_not_compile_is_an_error(commands, monkeypatch):
    before = build.subprocess.run

    def run(cmd, check):
        if cmd[0] == build.CXX:
            raise build.subprocess.CalledProcessError(1, cmd)
        before(cmd, check)

    monkeypatch.setattr(build.subprocess, "run", run)
    with pytest.raises(build.subprocess.CalledProcessError):
        build.build()
    assert os.path.exists(build.LIB)


def test_another_torch_builds_the_binding_again(commands, monkeypatch):
    import torch
    build.build_binding()
    assert len(commands) == 1
    build.build_binding()
    assert len(commands) == 1                   # fresh
    monkeypatch.setattr(torch, "__version__", "9.9.9")
    build.build_binding()
    assert len(commands) == 2
    build.build_binding()
    assert len(commands) == 2


def test_a_binding_of_another_torch_is_refused(monkeypatch):
    import torch
    build.build()
    monkeypatch.setattr(gdr, "_binding", None)
    monkeypatch.setattr(torch, "__version__", "9.9.9")
    with pytest.raises(RuntimeError, match="9.9.9"):
        gdr._ops()
    monkeypatch.undo()
    assert gdr._ops().torch_version == torch.__version__
