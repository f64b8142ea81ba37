"""The build: a binding for one torch and Python is never taken for another's, and the C library does not depend on it."""
import importlib.util
import os
import sysconfig

import pytest
import torch

import kimi_delta_attention_24_b200 as kda
from kimi_delta_attention_24_b200 import attention, build as kbuild


def test_binding_goes_by_the_versions_it_is_built_for():
    kbuild.build()
    name = os.path.basename(kbuild.binding_path())
    assert torch.__version__ in name and name.endswith(sysconfig.get_config_var("EXT_SUFFIX"))
    attention._load()
    assert os.path.samefile(attention._binding.__file__, kbuild.binding_path())


def test_binding_of_another_torch_is_not_loaded(monkeypatch):
    kbuild.build()
    folder, version = kbuild._torch()
    monkeypatch.setattr(kbuild, "_torch", lambda: (folder, version + ".other"))
    with pytest.raises(RuntimeError, match="is not built"):
        attention._load()


def test_c_library_is_linked_although_the_binding_fails(monkeypatch, tmp_path):
    kbuild.build()  # (the objects)
    monkeypatch.setattr(kbuild, "LIB_DIR", str(tmp_path))
    monkeypatch.setattr(kbuild, "LIB_PATH", str(tmp_path / "libkda_b200.so"))
    monkeypatch.setattr(kbuild, "_binding_command", lambda out: ["false"])
    with pytest.raises(RuntimeError, match="compiler failed"):
        kbuild.build()
    assert os.listdir(tmp_path) == ["libkda_b200.so"]


def test_c_library_is_linked_without_torch(monkeypatch, tmp_path):
    kbuild.build()
    monkeypatch.setattr(kbuild, "LIB_DIR", str(tmp_path))
    monkeypatch.setattr(kbuild, "LIB_PATH", str(tmp_path / "libkda_b200.so"))
    find = importlib.util.find_spec
    monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: None if name == "torch" else find(name, *a))
    with pytest.raises(RuntimeError, match="torch, which is not installed"):
        kbuild.build()
    assert os.listdir(tmp_path) == ["libkda_b200.so"]
    assert kda.load()
