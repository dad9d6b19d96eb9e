"""The torch binding belongs to the torch it was compiled against, and the C
library is built without one where there is none."""
import os
import sys

import pytest
import torch

from exact_attention_113_b200 import binding
from exact_attention_113_b200 import build as fa_build


def test_another_torch_does_not_load_this_ones_binding(monkeypatch):
    fa_build.build()
    mine = fa_build.binding_path()
    assert os.path.exists(mine)
    monkeypatch.setattr(torch, "__version__", "0.0.1")
    monkeypatch.setattr(binding, "_ext", None)
    assert fa_build.binding_path() != mine
    with pytest.raises(RuntimeError, match="build it with"):
        binding._serving()
    monkeypatch.undo()
    assert fa_build.binding_path() == mine and binding._serving() is not None


def test_c_library_without_torch(monkeypatch, capsys):
    path = fa_build.build()
    monkeypatch.setitem(sys.modules, "torch", None)      # import torch raises ImportError
    assert fa_build.build_binding() is None
    assert fa_build.build() == path
    assert "without its torch binding" in capsys.readouterr().err
