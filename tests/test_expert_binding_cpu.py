"""The backward passes' Python functions without a weight and without its
gradient, which the C entry points take: the sizes come from what there is.  CPU
tensors stand in for device ones, and a recorder for the library.  Also the test
hook of the expert operators, and the current stream's handle.
"""
import ctypes

import pytest
import torch

import moe_token_permute_gb300 as mp
from moe_token_permute_gb300 import _binding as b

BF = torch.bfloat16


@pytest.fixture
def passed(monkeypatch):
    """The sizes and pointers that a call passes on."""
    seen = {}

    class Library:
        def __getattr__(self, name):
            return lambda *args: seen.update({name: args}) or b.MOE_OK

    monkeypatch.setattr(mp._b, "lib", lambda: Library())
    monkeypatch.setattr(mp, "_ptr", lambda t: None if t is None else t.data_ptr())
    return seen


def tensors(R=5, K=16, N=24, E=3):
    z = lambda *s: torch.zeros(*s, dtype=BF)  # noqa: E731
    return z(R, N), z(R, K), z(R, N), z(E, N), torch.zeros(E + 1, dtype=torch.int64)


def test_bias_gradient_alone(passed):
    d, x, z, db, off = tensors()
    mp.moe_expert_linear_backward(d, None, None, off, d_bias=db, stream=0)
    args = passed["moe_expert_linear_backward"]
    R, K, N, E = args[5:9]
    assert (R, N, E) == (5, 24, 3) and K % 8 == 0 and K >= 8
    assert args[14] == db.data_ptr() and args[12] is None and args[13] is None
    mp.moe_expert_linear_backward(d, x, None, off, d_bias=db, activation="relu", preact=z,
                                  d_preact=d, stream=0)
    assert passed["moe_expert_linear_backward"][5:9] == (5, 16, 24, 3)


def test_dz_alone(passed):
    d, x, z, _, off = tensors()
    mp.moe_expert_linear_backward(d, None, None, off, activation="gelu", preact=z, d_preact=z,
                                  stream=0)
    assert passed["moe_expert_linear_backward"][5::2][:2] == (5, 24)
    assert passed["moe_expert_linear_backward"][8] == 3
    mp.moe_expert_gated_backward(d[:, :12].contiguous(), x, None, off, z, z, stream=0)
    assert passed["moe_expert_gated_backward"][5:9] == (5, 16, 12, 3)


def test_what_needs_a_weight_is_still_refused(passed):
    d, x, z, db, off = tensors()
    for kw, match in ((dict(d_rows=x), "d_rows needs weight"),
                      (dict(d_bias=db[:, :8]), "d_bias must hold"),
                      (dict(d_bias=torch.zeros(4, 24, dtype=BF)), "holds 4 elements")):
        with pytest.raises(ValueError, match=match):
            mp.moe_expert_linear_backward(d, None, None, off, stream=0, **kw)
    with pytest.raises(ValueError, match="d_rows needs weight"):
        mp.moe_expert_gated_backward(d[:, :12].contiguous(), x, None, off, z, z, d_rows=x, stream=0)
    with pytest.raises(ValueError, match=r"\[experts, out, in\]"):
        mp.moe_expert_linear_backward(d, x, None, off, d_weight=z, stream=0)
    assert not passed


def test_wait_hook_is_in_the_debug_build_only():
    from moe_token_permute_gb300 import build as cuda_build
    cuda_build.build()
    assert not hasattr(b.lib(), "moe_debug_set_expert_wait")
    hook = b.debug_lib().moe_debug_set_expert_wait
    hook.argtypes = [ctypes.c_int, ctypes.c_ulonglong]
    assert hook(-1, 1000) == b.MOE_ERR_INVALID_ARG
    assert hook(0, 0) == b.MOE_ERR_INVALID_ARG


@pytest.mark.parametrize("name", ["_raw_stream", "_raw_device"])
def test_current_stream_without_torchs_private_names(monkeypatch, name):
    class Current:
        cuda_stream = 0x1234

    monkeypatch.setattr(mp, name, None)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: Current)
    assert mp._stream(None) == 0x1234
    assert mp._stream(77) == 77
