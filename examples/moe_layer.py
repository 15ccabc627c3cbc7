"""One Mixture-of-Experts layer, forwards and backwards, on the library's calls:

    permute -> gated projection -> down projection -> unpermute

with every buffer allocated once, the offsets never leaving the device, and the
whole step captured into a CUDA graph.

    python examples/moe_layer.py --tokens 4096 --hidden 2048 --ffn 768 --experts 128 --topk 8

prints the time of the forward pass and of a training step, and how far the
layer is from the same layer in fp32 torch (on up to 256 of the tokens).
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))

import moe_token_permute_gb300 as mp  # noqa: E402

BF16 = torch.bfloat16


class MoELayer:
    """out[t] = sum_k w[t,k] * down[e](act(gate[e] x[t]) * up[e] x[t]), e = ids[t,k].

    w_gated [E, 2F, H] (an expert's gate rows, then its up rows) and w_down
    [E, H, F], bf16.  `training` also allocates what the backward pass keeps and
    writes.  The tensors the methods return are the layer's own buffers.
    """

    def __init__(self, w_gated, w_down, topk, max_tokens, activation="silu", training=False):
        self.w_gated, self.w_down, self.activation = w_gated, w_down, activation
        E, F2, H = w_gated.shape
        R, dev = max_tokens * topk, w_gated.device
        self.topk = topk
        self.scratch = mp.MoEPermuteScratch(max_tokens, topk, E, E, dev, H, BF16)

        def rows(cols):
            return torch.empty(R, cols, dtype=BF16, device=dev)

        self.h, self.y = rows(F2 // 2), rows(H)
        self.z = None
        if training:
            self.z, self.dz = rows(F2), rows(F2)
            self.dy, self.dh, self.dx = rows(H), rows(F2 // 2), rows(H)
            self.d_gated, self.d_down = torch.empty_like(w_gated), torch.empty_like(w_down)
            self.d_hidden = torch.empty(max_tokens, H, dtype=BF16, device=dev)
            self.d_weights = torch.empty(max_tokens, topk, device=dev)
            self.ones = torch.ones(max_tokens, topk, device=dev)

    def forward(self, hidden, ids, weights):
        T = hidden.shape[0]
        n = T * self.topk
        p = self.scratch.permute(hidden, ids)
        self.x, self.offset = p["permuted_hidden_states"], p["expert_first_token_offset"]
        self.inv = p["inv_permuted_idx"]
        ws = self.scratch.workspace
        mp.moe_expert_gated(self.x, self.w_gated, self.offset, self.h[:n],
                            activation=self.activation,
                            preact=None if self.z is None else self.z[:n], workspace=ws)
        mp.moe_expert_linear(self.h[:n], self.w_down, self.offset, self.y[:n], workspace=ws)
        return self.scratch.unpermute(self.y[:n], weights)

    def backward(self, d_out, weights):
        """The gradients of the last forward pass: hidden states, routing
        weights, w_gated and w_down."""
        T = d_out.shape[0]
        n = T * self.topk
        ws = self.scratch.workspace
        mp.moe_unpermute_backward(d_out, self.y[:n], weights, self.inv, self.dy[:n],
                                  self.d_weights[:T], workspace=ws)
        mp.moe_expert_linear_backward(self.dy[:n], self.h[:n], self.w_down, self.offset,
                                      d_rows=self.dh[:n], d_weight=self.d_down, workspace=ws)
        mp.moe_expert_gated_backward(self.dh[:n], self.x, self.w_gated, self.offset, self.z[:n],
                                     self.dz[:n], activation=self.activation,
                                     d_rows=self.dx[:n], d_weight=self.d_gated, workspace=ws)
        # a token's gradient is the sum of its rows': unpermute with unit weights
        mp.moe_unpermute(self.dx[:n], self.ones[:T], self.inv, self.d_hidden[:T], workspace=ws)
        return self.d_hidden[:T], self.d_weights[:T], self.d_gated, self.d_down


def plain_layer(hidden, ids, weights, w_gated, w_down):
    """The same layer in elementary torch operations, differentiable."""
    F = w_gated.shape[1] // 2
    out = torch.zeros_like(hidden)
    for e in range(w_gated.shape[0]):
        t, k = (ids == e).nonzero(as_tuple=True)
        z = hidden[t] @ w_gated[e].t()
        y = (torch.nn.functional.silu(z[:, :F]) * z[:, F:]) @ w_down[e].t()
        out = out.index_add(0, t, y * weights[t, k, None])
    return out


def timed(fn, repeats=20):
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        fn()
    torch.cuda.current_stream().wait_stream(side)
    with torch.cuda.graph(graph):
        fn()
    for _ in range(3):
        graph.replay()
    a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    a.record()
    for _ in range(repeats):
        graph.replay()
    b.record()
    torch.cuda.synchronize()
    return a.elapsed_time(b) / repeats * 1e3


def main():
    ap = argparse.ArgumentParser(description=__doc__,
                                 formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, value in (("tokens", 4096), ("hidden", 2048), ("ffn", 768), ("experts", 128),
                        ("topk", 8)):
        ap.add_argument("--" + name, type=int, default=value)
    a = ap.parse_args()
    T, H, F, E, K = a.tokens, a.hidden, a.ffn, a.experts, a.topk
    g = torch.Generator("cuda").manual_seed(0)

    def normal(*shape, scale=1.0):
        return (torch.randn(*shape, generator=g, device="cuda", dtype=BF16) * scale)

    hidden, d_out = normal(T, H), normal(T, H)
    w_gated, w_down = normal(E, 2 * F, H, scale=H ** -0.5), normal(E, H, F, scale=F ** -0.5)
    ids = torch.rand(T, E, generator=g, device="cuda").argsort(1)[:, :K].int().contiguous()
    weights = torch.softmax(torch.randn(T, K, generator=g, device="cuda"), 1)
    layer = MoELayer(w_gated, w_down, K, T, training=True)

    def step():
        layer.forward(hidden, ids, weights)
        layer.backward(d_out, weights)

    serving = MoELayer(w_gated, w_down, K, T)
    us = timed(lambda: serving.forward(hidden, ids, weights))
    flops = 6.0 * T * K * F * H
    print(f"forward        {us:9.1f} us  {flops / us / 1e6:7.1f} TFLOP/s")
    us = timed(step)
    print(f"training step  {us:9.1f} us  {3 * flops / us / 1e6:7.1f} TFLOP/s")
    n = min(T, 256)
    got = layer.forward(hidden[:n], ids[:n], weights[:n]).float()
    want = plain_layer(hidden[:n].float(), ids[:n], weights[:n], w_gated.float(), w_down.float())
    print(f"against fp32 torch: {((got - want).norm() / want.norm()).item():.2e} of the norm")
    assert layer.scratch.read_status() == 0


if __name__ == "__main__":
    main()
