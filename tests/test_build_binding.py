"""What the build makes where torch is missing, and the Python module's tie to the torch that it was compiled with."""
import importlib.util

import pytest

import int4_expert_streaming_gb300 as moe
from int4_expert_streaming_gb300 import _build


@pytest.fixture(scope="module", autouse=True)
def _built():
    moe.build()


def test_without_torch_the_library_is_built(monkeypatch):
    """The library needs no torch; only the Python module of the calls on tensors does."""
    find = importlib.util.find_spec
    monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: None if name == "torch" else find(name, *a))
    assert _build.up_to_date()
    assert moe.build() == _build.LIB
    assert moe.load_library().moe_blob_bytes(2048, 512, 4) > 0
