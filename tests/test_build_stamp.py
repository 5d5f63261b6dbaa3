"""The compiled argument marshalling is built again for another torch or Python,
whatever the files' times say."""
import importlib.metadata
import os

import pytest

from loss_scaling_master_gb300 import build as B


@pytest.fixture(scope="module", autouse=True)
def built():
    B.build()


def deps():
    return [B.BIND_SRC]


def test_fresh_after_a_build():
    assert not B._bind_stale(deps())
    assert open(B.BIND_STAMP).read().startswith(importlib.metadata.version("torch") + "\n")


def test_another_torch(monkeypatch):
    real = importlib.metadata.version
    monkeypatch.setattr(importlib.metadata, "version", lambda n: "9.9.9" if n == "torch" else real(n))
    assert B._bind_stale(deps())


def test_another_python(monkeypatch):
    real = B.sysconfig.get_config_var
    monkeypatch.setattr(B.sysconfig, "get_config_var", lambda n: "cpython-399" if n == "SOABI" else real(n))
    assert B._bind_stale(deps())


def test_another_command(monkeypatch):
    real = B._bind_command
    monkeypatch.setattr(B, "_bind_command", lambda target: real(target) + ["-DOTHER"])
    assert B._bind_stale(deps())


def test_a_module_without_a_stamp(monkeypatch, tmp_path):
    monkeypatch.setattr(B, "BIND_STAMP", str(tmp_path / "none"))
    assert B._bind_stale(deps())


def test_build_replaces_what_is_stale(monkeypatch):
    """A module with another build's stamp is compiled again and its stamp renewed."""
    before = os.stat(B.BIND)
    with open(B.BIND_STAMP, "w") as f:
        f.write("another torch")
    B.build()
    assert os.stat(B.BIND).st_ino != before.st_ino and not B._bind_stale(deps())
