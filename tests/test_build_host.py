"""The order and the conditions in which build.py compiles; nothing is compiled here."""
import os
import subprocess

import pytest

from block_sparse_attention_38_b200 import build as b


@pytest.fixture
def compilers(monkeypatch, tmp_path):
    """Names of the outputs in the order they are compiled; g++ may be told to fail."""
    made = []

    class Compilers:
        fail, tag = False, b""

    def run(cmd, check):
        out = cmd[cmd.index("-o") + 1]
        name = os.path.basename(out).split(".so")[0]
        if name == "_bsa_torch" and Compilers.fail:
            raise subprocess.CalledProcessError(1, cmd)
        made.append(name)
        with open(out, "wb") as f:
            f.write(Compilers.tag)

    Compilers.made = made
    monkeypatch.setattr(b, "LIB", str(tmp_path / "libbsa.so"))
    monkeypatch.setattr(b, "MARSHAL", str(tmp_path / "_bsa_torch.so"))
    monkeypatch.setattr(b.subprocess, "run", run)
    return Compilers


def test_the_library_comes_first_and_stays(compilers):
    compilers.fail = True
    with pytest.raises(subprocess.CalledProcessError):
        b.build(force=True)
    assert compilers.made == ["libbsa"] and os.path.exists(b.LIB)


def test_without_torch_the_library_is_built(compilers, monkeypatch):
    monkeypatch.setattr(b, "torch_home", lambda: (None, None))
    assert b.build(force=True) == b.LIB and compilers.made == ["libbsa"]


def test_the_module_is_built_again_for_another_torch(compilers, monkeypatch):
    compilers.tag = b.marshal_tag("2.0").encode()
    monkeypatch.setattr(b, "torch_home", lambda: ("/torch", "2.0"))
    b.build_marshal(force=True)
    b.build_marshal()
    assert compilers.made == ["_bsa_torch"]
    monkeypatch.setattr(b, "torch_home", lambda: ("/torch", "2.1"))
    b.build_marshal()
    assert compilers.made == ["_bsa_torch"] * 2


def test_the_version_is_that_of_the_torch_which_is_imported():
    import torch

    assert b.torch_home() == (os.path.dirname(torch.__file__), torch.__version__)


def test_a_module_for_another_torch_is_not_used(monkeypatch):
    from block_sparse_attention_38_b200 import long_stream

    monkeypatch.setattr(long_stream, "_marshal", None)
    long_stream._load()
    monkeypatch.setattr("torch.__version__", "0.1")
    with pytest.raises(ImportError, match="built for"):
        long_stream._load()
