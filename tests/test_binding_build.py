"""The compiled binding belongs to one Python and one torch."""
import os

import pytest
import torch

import block_sparse_long_tiled_b200 as sk
from block_sparse_long_tiled_b200 import build as sk_build


def test_a_binding_of_another_torch_is_neither_loaded_nor_taken_for_built(monkeypatch):
    sk_build.build()
    here = sk.binding_path()
    assert os.path.exists(here) and not sk_build._stale(here, sk_build.BINDING_SOURCES)
    module = sk._marshal()
    assert os.path.samefile(module.__file__, here)
    monkeypatch.setattr(torch, "__version__", torch.__version__ + ".another")
    assert sk.binding_path() != here
    assert sk_build._stale(sk.binding_path(), sk_build.BINDING_SOURCES)
    monkeypatch.setattr(sk, "_binding_module", None)
    with pytest.raises(RuntimeError, match="is missing: build it"):
        sk._marshal()


def test_a_binding_of_another_python_is_another_file(monkeypatch):
    import sys
    import types
    here = sk.binding_path()
    other = types.SimpleNamespace(**{**vars(sys.implementation), "cache_tag": "cpython-999"})
    monkeypatch.setattr(sys, "implementation", other)
    assert sk.binding_path() != here
