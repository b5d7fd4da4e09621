"""The marshalling module of the attention calls is built, and looked for, under
the interpreter's own tag: one that was built for another is neither loaded nor
taken for up to date."""
import os
import shutil
import sysconfig

import pytest

import gated_deltanet_linear_07_gb300 as gdn
from gated_deltanet_linear_07_gb300 import _binding, _build


def test_the_module_carries_the_interpreters_tag():
    gdn.build()
    assert _build.CALLS.endswith(sysconfig.get_config_var("EXT_SUFFIX"))
    assert os.path.exists(_build.CALLS)


def test_another_interpreters_module_is_not_taken(monkeypatch, tmp_path):
    gdn.build()
    calls = str(tmp_path / ("_attn_calls" + sysconfig.get_config_var("EXT_SUFFIX")))
    shutil.copy2(_build.CALLS, tmp_path / "_attn_calls.cpython-30-none.so")
    shutil.copy2(_build.CALLS, tmp_path / "_attn_calls.so")
    monkeypatch.setattr(_build, "CALLS", calls)
    monkeypatch.setattr(_binding, "PKG", str(tmp_path))
    monkeypatch.setattr(_binding, "_calls", None)
    assert not _build.up_to_date()
    with pytest.raises(ImportError, match="build it first"):
        _binding._attn_calls()
