"""The native binding of the mixer operators: when it is built again, and what is
said where it cannot be used."""
import sys

import pytest


@pytest.fixture
def fresh(monkeypatch):
    """The package as at its first call, with the binding built."""
    from kalman_linear_attention_b200 import _build, api
    _build.build()
    monkeypatch.setattr(api, "_mixer", None)
    return _build, api


def test_built_again_for_another_torch_or_python(fresh, monkeypatch):
    _build, _ = fresh
    assert _build.binding_up_to_date()
    now = _build.built_for()
    assert f"Python {sys.version_info.major}.{sys.version_info.minor}" in now
    for other in ("torch 1.0, Python 3.8", now[:-1], now + "1"):
        monkeypatch.setattr(_build, "built_for", lambda: other)
        assert not _build.binding_up_to_date(), other


def test_refused_for_another_torch_or_python(fresh, monkeypatch):
    _build, api = fresh
    now = _build.built_for()
    assert api._native().built_for == now
    monkeypatch.setattr(api, "_mixer", None)
    monkeypatch.setattr(_build, "built_for", lambda: "torch 1.0, Python 3.8")
    with pytest.raises(RuntimeError) as e:
        api._native()
    assert now in str(e.value) and "torch 1.0, Python 3.8" in str(e.value)


def test_missing_and_unloadable_are_told_apart(fresh, monkeypatch, tmp_path):
    _build, api = fresh
    monkeypatch.setitem(sys.modules, "kalman_linear_attention_b200._mixer", None)  # an ImportError
    monkeypatch.delattr(sys.modules["kalman_linear_attention_b200"], "_mixer", raising=False)
    with pytest.raises(RuntimeError, match="could not be loaded"):
        api._native()
    monkeypatch.setattr(_build, "BINDING", str(tmp_path / "_mixer.so"))
    with pytest.raises(RuntimeError, match="is not built"):
        api._native()
