"""Misaligned arrays of the speculative-decoding operations are refused on the
host: on the GPU they would be an address error."""
import pytest

from transformer_decode_token_gb300 import binding

from test_spec_host import P, attend, commit, kv, load, store, verify

CALLS = [(store, ("slot", "pos")), (load, ("slot", "pos")), (commit, ("slot", "cached", "path", "n_path")),
         (attend, ("slot", "cached", "first"))]


@pytest.mark.parametrize("call,names", CALLS)
def test_misaligned_index_arrays_are_refused(call, names):
    for name in names:
        for off in (1, 2, 3):
            assert call(kv(), **{name: P + off}) == -1, (name, off)


@pytest.mark.parametrize("call", [c for c, _ in CALLS])
def test_misaligned_scales_are_refused(call):
    for bad in (dict(k_scale=P + 2, v_scale=P), dict(k_scale=P, v_scale=P + 1)):
        assert call(kv(dtype=binding.GPT2_INT8, **bad)) == -1, bad


def test_misaligned_verification_arrays_are_refused():
    for name in ("tokens", "parents", "first", "draft", "ua", "ud", "path", "n_path", "token"):
        for off in (1, 2):
            assert verify(**{name: P + off}) == -1, (name, off)
