"""The activations and their derivatives over all of their range, against bounds
that grow with the argument as the fast exponential's error does.

With x a unit vector and the arguments as the weight, the kept z is exact, and
one value goes through the activation alone.  u = 2^-23.
  exponent: x = -z for silu; for gelu 2 sqrt(2/pi) z (1 + 0.044715 z^2), computed in
    six roundings, so off by 3 |x| u
  p = sigmoid: relative error (4.5 + 1.173 |x|) u from the exponential (2 + 1.173 |x|
    ulp), the sum and the division (2 ulp), and 3 |x| u from gelu's exponent; 0 where
    1 + exp(-x) passes 2^126, so 2^-126 more
  act = z p; act' = p + z p (1 - p) q, q = 1 for silu and 2 sqrt(2/pi) (1 + 3 0.044715
    z^2) for gelu: each term carries its factors' errors and a rounding each
and the result is rounded to the type.
"""
import math

import pytest
import torch

import expert_ref as ref
import moe_token_permute_gb300 as mp

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, HF = torch.bfloat16, torch.float16
U = 2.0 ** -23
A, B = math.sqrt(2 / math.pi), 0.044715


def arguments(dtype):
    v = torch.cat([torch.linspace(-130, 130, 4097), torch.linspace(-20, 20, 4095),
                   torch.logspace(-6, 1, 1024), -torch.logspace(-6, 1, 1024)]).to(dtype)
    return v[:v.numel() // 8 * 8].to(DEV)


def expected(act, z):
    """act(z) and act'(z) in 64 bits with their bounds."""
    z = z.double()
    if act == "silu":
        x, q, steps = z, torch.ones_like(z), 0.0
    else:
        x, q, steps = 2 * A * z * (1 + B * z * z), 2 * A * (1 + 3 * B * z * z), 3.0
    p = torch.where(x < 0, torch.exp(x) / (1 + torch.exp(x)), 1 / (1 + torch.exp(-x)))
    other = torch.where(x < 0, 1 / (1 + torch.exp(x)), torch.exp(-x) / (1 + torch.exp(-x)))
    e_p = (4.5 + (1.173 + steps) * x.abs()) * U * p + 2.0 ** -126
    a = z * p
    e_a = z.abs() * e_p + U * a.abs() + 2.0 ** -126
    # 1 - p: p's error and a rounding of a value up to 1; from exp(-x) < 2^-25 on the
    # sum is 1, p is 1 and 1 - p is 0
    e_other = torch.where(x > 25 * math.log(2), other, e_p + U / 2)
    slope = a * other * q
    e_slope = (e_a * (other + e_other) + a.abs() * e_other) * q + 8 * U * (
        (a.abs() + e_a) * (other + e_other) * q)
    d = p + slope
    return ref.Val(a, e_a), ref.Val(d, e_p + e_slope + U * (p + slope.abs()) + 2.0 ** -126)


@pytest.mark.parametrize("dtype", [BF, HF], ids=str)
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_linear(act, dtype):
    z = arguments(dtype)
    N = z.numel()
    w = torch.zeros(1, N, 8, dtype=dtype, device=DEV)
    w[0, :, 0] = z
    x = torch.zeros(1, 8, dtype=dtype, device=DEV)
    x[0, 0] = 1
    offset = torch.tensor([0, 1], device=DEV)
    out, pre, dz = (torch.empty(1, N, dtype=dtype, device=DEV) for _ in range(3))
    mp.moe_expert_linear(x, w, offset, out, activation=act, preact=pre)
    assert torch.equal(pre[0], z)
    a, d = expected(act, z)
    ref.check(out[0], a, dtype, "act")
    mp.moe_expert_linear_backward(torch.ones_like(out), None, w, offset, activation=act,
                                  preact=pre, d_preact=dz)
    ref.check(dz[0], d, dtype, "act'")


@pytest.mark.parametrize("dtype", [BF, HF], ids=str)
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_gated(act, dtype):
    z = arguments(dtype)
    F = z.numel()
    w = torch.zeros(1, 2 * F, 8, dtype=dtype, device=DEV)
    w[0, :F, 0], w[0, F:, 0] = z, 1
    x = torch.zeros(1, 8, dtype=dtype, device=DEV)
    x[0, 0] = 1
    offset = torch.tensor([0, 1], device=DEV)
    out = torch.empty(1, F, dtype=dtype, device=DEV)
    pre, dz = (torch.empty(1, 2 * F, dtype=dtype, device=DEV) for _ in range(2))
    mp.moe_expert_gated(x, w, offset, out, activation=act, preact=pre)
    a, d = expected(act, z)
    ref.check(out[0], a, dtype, "act * 1")
    mp.moe_expert_gated_backward(torch.ones_like(out), None, w, offset, pre, dz, activation=act)
    ref.check(dz[0, :F], d, dtype, "d_gate")
    ref.check(dz[0, F:], a, dtype, "d_up")
