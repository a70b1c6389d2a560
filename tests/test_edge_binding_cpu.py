"""The binding module of the operators at the block's edge: built for one torch and one Python, and
loaded under no other (no GPU)."""

import os
import sysconfig

import pytest
import torch


@pytest.fixture(scope="module")
def build():
    from mxfp4_quantized_moe_b200 import build as b
    b.build()
    return b


def test_the_name_says_what_it_was_built_for(build):
    name = os.path.basename(build.BINDING)
    assert torch.__version__ in name and sysconfig.get_config_var("SOABI") in name
    assert not build.needs_binding()


def test_under_another_torch_it_is_built_anew_and_not_loaded(build, monkeypatch):
    from mxfp4_quantized_moe_b200 import moe
    other = build.BINDING.replace(torch.__version__, "0.0.0")
    assert other != build.BINDING
    monkeypatch.setattr(build, "BINDING", other)
    assert build.needs_binding()
    with pytest.raises(ImportError, match="mxfp4_quantized_moe_b200.build"):
        moe._load_edge()


def test_the_loaded_module_has_every_call(build):
    from mxfp4_quantized_moe_b200 import moe
    assert moe._edge.__file__ == build.BINDING
    for name in ("route", "route_backward", "norm_forward", "norm_backward", "checkpoint_pack",
                 "checkpoint_unpack"):
        assert callable(getattr(moe._edge, name))
