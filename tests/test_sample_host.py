"""What BatchModel.sample reports of a call that fails before it has drawn anything:
the library stood in for by one that returns its codes."""
import ctypes
import types

import pytest

pytest.importorskip("torch")

from transformer_decode_token_gb300 import binding


def model(monkeypatch, status, write=()):
    def sample_batch(handle, n, temperature, top_k, top_p, min_p, u, ids):
        for i, t in enumerate(write):
            ids[i] = t
        return status
    monkeypatch.setattr(binding, "lib", lambda *a, **k: types.SimpleNamespace(
        gpt2_sample_batch=sample_batch, gpt2_strerror=lambda s: b"?", gpt2_destroy_batch=lambda h: None))
    m = object.__new__(binding.BatchModel)
    m._h, m.cfg = ctypes.c_void_p(None), types.SimpleNamespace(vocab_size=50)
    return m


def test_a_failed_step_leaves_no_tokens(monkeypatch):
    m = model(monkeypatch, -8)
    with pytest.raises(binding.GPT2Error) as e:
        m.sample(3)
    assert e.value.name == "DEVICE_STATE" and e.value.tokens == [-1, -1, -1]


def test_rows_without_a_choice(monkeypatch):
    m = model(monkeypatch, -8, (7, -1, 9))
    with pytest.raises(binding.GPT2Error) as e:
        m.sample(3)
    assert e.value.name == "DEVICE_STATE" and e.value.tokens == [7, -1, 9]


@pytest.mark.parametrize("status,name", [(-7, "TIMEOUT"), (-5, "NOT_READY"), (-1, "INVALID_ARG")])
def test_other_failures(monkeypatch, status, name):
    m = model(monkeypatch, status)
    with pytest.raises(binding.GPT2Error) as e:
        m.sample(2)
    assert e.value.name == name
