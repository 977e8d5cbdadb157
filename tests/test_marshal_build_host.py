"""_vx_marshal.so is rebuilt when torch changes, and refused by the binding when it was built for another."""
import subprocess

import pytest
import torch

from paged_block_sparse_kv_b200 import build, vx


def test_marshal_is_built_again_for_another_torch(monkeypatch):
    build.build_marshal()
    ran = []
    monkeypatch.setattr(subprocess, "run", lambda *a, **k: ran.append(a))
    monkeypatch.setattr(build.os, "replace", lambda *a: None)
    build.build_marshal()
    assert not ran  # up to date
    monkeypatch.setattr(torch, "__version__", torch.__version__ + ".1")
    build.build_marshal()
    assert len(ran) == 1


def test_binding_refuses_a_marshal_for_another_torch(monkeypatch):
    build.build_marshal()
    monkeypatch.setattr(vx, "_native", None)
    vx._marshal()
    monkeypatch.setattr(vx, "_native", None)
    monkeypatch.setattr(torch, "__version__", "1.0")
    with pytest.raises(ImportError, match="run __graft_entry__"):
        vx._marshal()
