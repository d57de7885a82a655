"""The serving operators' binding is built for one Python and one torch, and no other is loaded."""
import os
import sysconfig

import pytest
import torch

from gqa_flash_attention_gb300 import build, serving


def test_its_name_says_what_it_was_built_for():
    name = os.path.basename(serving.BINDING_PATH)
    assert torch.__version__ in name and sysconfig.get_config_var("SOABI") in name
    assert serving._binding_path("9.9.9") != serving.BINDING_PATH
    assert "/" not in os.path.basename(serving._binding_path("9.9/x y"))


def test_one_built_for_another_torch_is_not_loaded(monkeypatch):
    build.build()
    assert os.path.exists(serving.BINDING_PATH)
    assert callable(serving._Binding().fwd_window)
    monkeypatch.setattr(serving, "BINDING_PATH", serving._binding_path("9.9.9"))  # after an upgrade
    with pytest.raises(RuntimeError, match="not built"):
        serving._Binding().fwd_window


def test_a_build_makes_the_missing_one_alone(monkeypatch):
    build.build()
    made = []
    monkeypatch.setattr(build, "BINDING_PATH", serving._binding_path("9.9.9"))
    monkeypatch.setattr(build, "_compile_binding", lambda: "object")
    monkeypatch.setattr(build, "_link_binding", made.append)
    monkeypatch.setattr(build, "_compile", lambda src: pytest.fail("the library is there"))
    build.build()
    assert made == ["object"]
    monkeypatch.setattr(build, "BINDING_PATH", serving.BINDING_PATH)
    build.build()
    assert made == ["object"]
