"""What build() makes, and when, with the compilers replaced (no GPU needed)."""
import os

import pytest


@pytest.fixture
def made(monkeypatch, tmp_path):
    """build.py with its outputs under tmp_path and compilers that only write their output files; the commands
    that ran, by the kind of file that they made."""
    from top_sparse_attention_row_gb300 import build as b
    ran = []

    def write(path):
        ran.append(os.path.basename(path).removesuffix(".tmp"))
        with open(path, "w") as f:
            f.write("x")
        return path

    class Done:
        returncode, stdout, stderr = 0, "", ""

    def run(cmd, **kw):
        write(cmd[cmd.index("-o") + 1])
        return Done()

    monkeypatch.setattr(b, "BUILD", str(tmp_path / "_build"))
    monkeypatch.setattr(b, "LIB", str(tmp_path / "libqsa.so"))
    monkeypatch.setattr(b, "EXT", str(tmp_path / "_serving.so"))
    monkeypatch.setattr(b, "EXT_STAMP", str(tmp_path / "_build" / "_serving.made_for"), raising=False)
    monkeypatch.setattr(b, "_nvcc", lambda: "/usr/local/cuda/bin/nvcc")
    monkeypatch.setattr(b.subprocess, "run", run)
    b.ran = ran
    yield b
    del b.ran


def test_the_library_is_built_without_torch(made, monkeypatch, capsys):
    """The C library needs nvcc alone; the extension is left out, and said to be."""
    monkeypatch.setitem(__import__("sys").modules, "torch", None)      # an import raises
    assert made.torch_root() is None
    assert made.build() == made.LIB and os.path.exists(made.LIB) and not os.path.exists(made.EXT)
    assert "_serving" in capsys.readouterr().err
    del made.ran[:]
    made.build()
    assert made.ran == []                                              # up to date


def test_both_are_built_with_torch(made):
    made.build()
    assert os.path.exists(made.LIB) and os.path.exists(made.EXT)
    assert "torch_serving.o" in made.ran and "libqsa.so" in made.ran and "_serving.so" in made.ran
    del made.ran[:]
    made.build()
    assert made.ran == []


def test_an_extension_that_does_not_compile_is_an_error(made, monkeypatch):
    def broken():
        raise RuntimeError("g++ failed")
    monkeypatch.setattr(made, "_compile_extension", broken)
    with pytest.raises(RuntimeError, match="g\\+\\+ failed"):
        made.build()
    assert os.path.exists(made.LIB)


def test_the_extension_is_built_again_for_another_torch(made, monkeypatch, tmp_path):
    """It is compiled against PyTorch's headers: another version, or place, needs another extension."""
    made.build()
    del made.ran[:]
    other = tmp_path / "torch"
    other.mkdir()
    (other / "version.py").write_text("__version__ = '0.0.1'")
    monkeypatch.setattr(made, "torch_root", lambda: str(other))
    made.build()
    assert "_serving.so" in made.ran
    del made.ran[:]
    made.build()
    assert made.ran == []
    (other / "version.py").write_text("__version__ = '0.0.2'")
    made.build()
    assert "_serving.so" in made.ran
    os.remove(made.EXT_STAMP)                       # not known what it was built against
    del made.ran[:]
    made.build()
    assert "_serving.so" in made.ran
