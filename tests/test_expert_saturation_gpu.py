"""Pre-activations that are finite in fp32 and overflow in the 16 bits they are
kept in: the forward pass has used the finite value, and the backward pass takes
the limits of the activation and its derivative, not infinity times zero.
"""
import pytest
import torch

import moe_token_permute_gb300 as mp

pytestmark = pytest.mark.gpu
DEV = "cuda"
HF = torch.float16

# x * w in fp32, one per output: 65504 is fp16's largest, 65520 rounds to infinity
X = 256.0
GATES = [-76800.0, -65536.0, -65504.0, -1024.0, 1024.0, 65504.0, 65536.0, 76800.0]


def column(values):
    """A weight [1, len, 8] whose rows give `values` for x = [X, 16, 0, ...]."""
    w = torch.zeros(1, len(values), 8, dtype=torch.float64, device=DEV)
    v = torch.tensor(values, dtype=torch.float64, device=DEV)
    w[0, :, 0] = (v / X).to(HF).double()
    w[0, :, 1] = (v - w[0, :, 0] * X) / 16.0
    w = w.to(HF)
    assert torch.equal(w[0, :, 0].double() * X + w[0, :, 1].double() * 16.0, v)
    return w


def setup():
    x = torch.zeros(1, 8, dtype=HF, device=DEV)
    x[0, 0], x[0, 1] = X, 16.0
    return x, torch.tensor([0, 1], device=DEV)


@pytest.mark.parametrize("act", ["silu", "gelu", "relu"])
def test_gated(act):
    x, offset = setup()
    w = torch.cat([column(GATES), column([0.5] * 8)], 1).contiguous()
    out, pre, dz = (torch.empty(1, c, dtype=HF, device=DEV) for c in (8, 16, 16))
    mp.moe_expert_gated(x, w, offset, out, activation=act, preact=pre)
    z = torch.tensor(GATES, device=DEV)
    assert torch.isinf(pre[0, :2]).all() and torch.isinf(pre[0, 6:8]).all()
    assert torch.isfinite(pre[0, 2:6]).all()
    want = torch.where(z > 0, z * 0.5, torch.zeros_like(z)).to(HF)
    assert torch.equal(out[0].float().abs(), want.float())  # finite: act(z) * up in fp32
    d = torch.full((1, 8), 2.0, dtype=HF, device=DEV)
    mp.moe_expert_gated_backward(d, None, w, offset, pre, dz, activation=act)
    # d_gate = 2 * 0.5 * act'(z); d_up = 2 * act(z) of the kept z
    assert torch.equal(dz[0, :8].float(), (z > 0).float())
    up = torch.where(z > 0, 2.0 * pre[0, :8].float(), torch.zeros_like(z)).to(HF)
    assert torch.equal(dz[0, 8:].float().abs(), up.float())


@pytest.mark.parametrize("act", ["silu", "gelu", "relu"])
def test_linear(act):
    x, offset = setup()
    w = column(GATES)
    out, pre, dz = (torch.empty(1, 8, dtype=HF, device=DEV) for _ in range(3))
    mp.moe_expert_linear(x, w, offset, out, activation=act, preact=pre)
    d = torch.full((1, 8), 3.0, dtype=HF, device=DEV)
    mp.moe_expert_linear_backward(d, None, w, offset, activation=act, preact=pre, d_preact=dz)
    z = torch.tensor(GATES, device=DEV)
    assert torch.equal(dz[0].float(), 3.0 * (z > 0).float())


@pytest.mark.parametrize("act", ["silu", "gelu", "relu"])
def test_nan_stays(act):
    pre = torch.full((2, 8), float("nan"), dtype=HF, device=DEV)
    d, dz = torch.ones(2, 8, dtype=HF, device=DEV), torch.zeros(2, 8, dtype=HF, device=DEV)
    mp.moe_expert_linear_backward(d, None, None, torch.tensor([0, 2], device=DEV), activation=act,
                                  preact=pre, d_preact=dz)
    assert torch.isnan(dz.float()).all()
