"""The build of the CUDA library does not hang on what only its Python module needs."""
import os

import pytest

from tree_verify_b200 import build as b


def _fake_compiler(monkeypatch, tmp_path):
    """Records the targets that are compiled; nothing is, and nothing is up to date."""
    made = []

    def compile_(cmd, target, verbose):
        made.append((os.path.basename(target), cmd[0]))
        if os.path.basename(target) == "_marshal.so":
            raise RuntimeError("no C++ compiler")

    monkeypatch.setattr(b, "_compile", compile_)
    monkeypatch.setattr(b, "LIB", str(tmp_path / "libeagle_verify.so"))
    monkeypatch.setattr(b, "MARSHAL", str(tmp_path / "_marshal.so"))
    return made


@pytest.mark.parametrize("force", [False, True])
def test_the_library_is_built_where_the_module_cannot_be(monkeypatch, tmp_path, force):
    made = _fake_compiler(monkeypatch, tmp_path)
    with pytest.raises(RuntimeError):
        b.build(force=force)
    assert [name for name, _ in made] == ["libeagle_verify.so", "_marshal.so"]


def test_the_compiler_is_looked_up_at_the_call(monkeypatch, tmp_path):
    made = _fake_compiler(monkeypatch, tmp_path)
    monkeypatch.setenv("NVCC", "/opt/other/bin/nvcc")
    with pytest.raises(RuntimeError):
        b.build()
    assert made[0] == ("libeagle_verify.so", "/opt/other/bin/nvcc")
