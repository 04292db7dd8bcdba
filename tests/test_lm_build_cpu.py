"""The library is built without torch, as before it had a compiled binding."""
import importlib.util

from recurrent_nn_amd import build


def test_without_torch_there_is_no_binding_and_no_error(monkeypatch, tmp_path):
    target = tmp_path / "_binding.so"
    find = importlib.util.find_spec
    monkeypatch.setattr(build, "BINDING", str(target))
    monkeypatch.setattr(importlib.util, "find_spec", lambda name: None if name == "torch" else find(name))
    assert build.build_binding() is None
    assert not target.exists()
