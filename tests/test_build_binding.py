"""What the build makes where torch is missing, and the Python module's tie to the torch that it was compiled with."""
import importlib.util
import os

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


def other_torch(tmp_path, monkeypatch, version):
    """A torch of that version, older than everything built here."""
    folder = tmp_path / "torch"
    folder.mkdir()
    for name, text in (("__init__.py", ""), ("version.py", f"__version__ = '{version}'\n")):
        (folder / name).write_text(text)
        os.utime(folder / name, (0, 0))
    find, spec = importlib.util.find_spec, importlib.util.spec_from_file_location("torch", folder / "__init__.py")
    monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: spec if name == "torch" else find(name, *a))


def test_the_module_of_another_torch_is_out_of_date(tmp_path, monkeypatch):
    """However old that torch's files are, and also where the version is the same but in another place."""
    torch = pytest.importorskip("torch")
    assert _build.up_to_date()
    other_torch(tmp_path, monkeypatch, "1.0.0")
    assert not _build.up_to_date()
    (tmp_path / "torch" / "version.py").write_text(f"__version__ = '{torch.__version__}'\n")
    os.utime(tmp_path / "torch" / "version.py", (0, 0))
    assert not _build.up_to_date()


def test_the_module_of_another_torch_makes_no_call(monkeypatch):
    """A module left from another torch would read tensors at the wrong places, without an error."""
    torch = pytest.importorskip("torch")
    monkeypatch.setattr(moe, "_ops", None)
    monkeypatch.setattr(torch, "__version__", "1.0.0")
    with pytest.raises(RuntimeError, match="built for torch .*not for torch 1.0.0"):
        moe.moe_combine(None, None, None, None)
    monkeypatch.delitem(vars(moe), "moe_conv", raising=False)
    with pytest.raises(RuntimeError, match="built for torch"):
        moe.moe_conv
    monkeypatch.undo()
    with pytest.raises(ValueError):
        moe.moe_conv(None, None, None)
