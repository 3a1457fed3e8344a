"""The extension module of the calls is built for one torch: its C++ interface is torch's own (no GPU needed)."""
import os

import pytest
import torch


def test_the_module_of_another_torch_is_not_loaded_and_is_built_again(monkeypatch):
    from mxfp8_microscaled_precision_gb300 import build, mxq
    build.build()
    assert os.path.exists(build.calls_path()) and not build._stale()
    assert torch.__version__ in os.path.basename(build.calls_path())
    monkeypatch.setattr(build, "_torch_version", lambda: "0.0.1+another")
    assert build._stale()
    monkeypatch.setattr(mxq, "_calls_module", None)
    with pytest.raises(RuntimeError, match="not built"):
        mxq._calls()
    monkeypatch.undo()
    assert not build._stale() and mxq._calls().__file__ == build.calls_path()
