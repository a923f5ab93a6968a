"""What the build script makes, where and when; nothing is compiled here."""
import os

import pytest

from tile_signaled_grouped_gb300 import build as B


@pytest.fixture
def made(tmp_path, monkeypatch):
    """The build script with its outputs in a folder of their own and compilers that only write
    their output files; the list of what it linked."""
    linked = []

    def run(cmd, what):
        out = cmd[cmd.index("-o") + 1]
        open(out, "w").close()
        if out.endswith(".tmp"):
            linked.append(os.path.basename(out)[:-4])

    monkeypatch.setattr(B, "LIB", str(tmp_path / "libmoe_tsg.so"))
    monkeypatch.setattr(B, "BINDING", str(tmp_path / "_torch_ops.so"))
    monkeypatch.setattr(B, "BUILD", str(tmp_path / "_build"))
    monkeypatch.setattr(B, "_run", run)
    monkeypatch.setattr(B, "_compile", lambda src, verbose, extra: src + ".o")
    return linked


def test_library_and_binding_are_built_once(made):
    assert B.build() == B.LIB
    assert made == ["libmoe_tsg.so", "_torch_ops.so"]
    B.build()
    assert len(made) == 2
    B.build(force=True)
    assert len(made) == 4


def test_library_is_built_without_torch(made, monkeypatch):
    monkeypatch.setattr(B, "_torch", lambda: None)
    assert B.build() == B.LIB and os.path.exists(B.LIB)
    assert made == ["libmoe_tsg.so"]
    B.build()
    assert made == ["libmoe_tsg.so"]
    assert "PyTorch" in B.binding_lacks()


def test_library_is_built_without_headers_or_compiler_of_the_binding(made, monkeypatch, tmp_path):
    monkeypatch.setattr(B, "_torch", lambda: str(tmp_path))
    assert "extension.h" in B.binding_lacks()
    assert B.build() == B.LIB
    assert made == ["libmoe_tsg.so"]
    monkeypatch.undo()
    monkeypatch.setenv("CXX", "no-such-compiler")
    assert "no-such-compiler" in B.binding_lacks()


def test_binding_of_another_torch_is_built_anew(made, monkeypatch, tmp_path):
    include = tmp_path / "torch" / "include" / "torch"
    include.mkdir(parents=True)
    (include / "extension.h").touch()
    monkeypatch.setattr(B, "_torch", lambda: str(tmp_path / "torch"))
    for version in ("1.0+a", "1.0+b"):
        (tmp_path / "torch" / "version.py").write_text(f"__version__ = '{version}'")
        B.build()
    assert made == ["libmoe_tsg.so", "_torch_ops.so"] * 2
    B.build()
    assert len(made) == 4
    monkeypatch.setattr(B.sysconfig, "get_config_var", lambda name: "cpython-300")
    B.build()
    assert len(made) == 6
