"""The whole layer of examples/moe_layer.py (permute, gated and down projection,
unpermute, and their gradients) against autograd through the plain layer in 64
bits.

Tolerance: every tensor between two kernels is rounded to bf16 (relative error
at most u = 2^-8 an element), and so is the result.  A result is a sum of
products of such tensors, so in the 2-norm its relative error is at most about
u times the number of roundings on its longest path, and independent roundings
do far better: 6 for the output (gate and up, h, y, out: the first counts twice,
through silu' and up), 10 for a gradient (those before y, dy, dh, dz, dx).
"""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                                "examples"))
from moe_layer import BF16, MoELayer, plain_layer  # noqa: E402

pytestmark = pytest.mark.gpu
U = 2.0 ** -8


def close(got, want, roundings, what):
    err = (got.double() - want).norm() / want.norm()
    assert err <= roundings * U, (what, err.item())


@pytest.mark.parametrize("T,H,F,E,K", [(1, 256, 64, 8, 2), (7, 136, 72, 5, 3), (64, 512, 264, 32, 4),
                                       (300, 256, 128, 4, 2), (515, 264, 136, 16, 6)])
def test_layer_forwards_and_backwards(T, H, F, E, K):
    g = torch.Generator("cuda").manual_seed(T)
    hidden = torch.randn(T, H, generator=g, device="cuda").to(BF16)
    d_out = torch.randn(T, H, generator=g, device="cuda").to(BF16)
    w_gated = (torch.randn(E, 2 * F, H, generator=g, device="cuda") * H ** -0.5).to(BF16)
    w_down = (torch.randn(E, H, F, generator=g, device="cuda") * F ** -0.5).to(BF16)
    ids = torch.rand(T, E, generator=g, device="cuda").argsort(1)[:, :K].int().contiguous()
    weights = torch.softmax(torch.randn(T, K, generator=g, device="cuda"), 1)
    layer = MoELayer(w_gated, w_down, K, T + 3, training=True)  # buffers may be larger
    out = layer.forward(hidden, ids, weights).clone()
    got = layer.backward(d_out, weights)
    leaves = [t.double().requires_grad_() for t in (hidden, weights, w_gated, w_down)]
    want = plain_layer(leaves[0], ids, leaves[1], leaves[2], leaves[3])
    want.backward(d_out.double())
    close(out, want.detach(), 6, "out")
    for a, leaf, what in zip(got, leaves, ("hidden", "weights", "w_gated", "w_down")):
        close(a, leaf.grad, 10, what)
    assert layer.scratch.read_status() == 0
    # a layer without the backward pass's buffers gives the same bits
    assert torch.equal(MoELayer(w_gated, w_down, K, T).forward(hidden, ids, weights), out)
