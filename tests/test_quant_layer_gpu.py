"""A serving layer on 8-bit rows and weights, as it is used, in one CUDA graph:

  fp8   moe_permute_quant_fp8 -> gated -> moe_quant_rows -> linear -> unpermute
  int8  moe_quant_rows -> moe_permute -> gated -> moe_quant_rows -> linear -> unpermute

against the same steps in 64 bits from the codes that the layer itself holds
between them, each step within its own bound, and the codes bit for bit.
"""
import pytest
import torch

import expert_ref as ref
import moe_token_permute_gb300 as mp
import quant_ref as qref

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16
E4M3, INT8 = torch.float8_e4m3fn, torch.int8


class QuantLayer:
    """Buffers allocated once; the offsets never leave the device."""

    def __init__(self, code, w_gated, s_gated, w_down, s_down, topk, experts, max_tokens):
        self.code, self.weights = code, (w_gated, s_gated, w_down, s_down)
        L, F2, H = w_gated.shape
        self.F, rows = F2 // 2, max_tokens * topk
        columns = 1 if code == INT8 else H // 128
        self.scratch = mp.MoEPermuteScratch(max_tokens, topk, experts, L, torch.device(DEV), H,
                                            code, scale_cols=columns)

        def empty(*shape, dtype=BF):
            return torch.empty(*shape, dtype=dtype, device=DEV)

        self.tokens = empty(max_tokens, H, dtype=code)
        self.token_scales = empty(max_tokens, 1, dtype=torch.float32)
        self.h, self.y = empty(rows, self.F), empty(rows, H)
        self.h_codes = empty(rows, self.F, dtype=code)
        self.h_scales = empty(rows, 1 if code == INT8 else qref.groups(self.F),
                              dtype=torch.float32)
        self.out = empty(max_tokens, H)

    def forward(self, hidden, ids, weights, expert_map=None):
        T, n = hidden.shape[0], ids.numel()
        w_gated, s_gated, w_down, s_down = self.weights
        s, ws = self.scratch, self.scratch.workspace
        if self.code == INT8:
            mp.moe_quant_rows(hidden, self.tokens[:T], self.token_scales[:T], workspace=ws)
            p = s.permute(self.tokens[:T], ids, hidden_scales=self.token_scales[:T],
                          expert_map=expert_map)
        else:
            p = s.permute_quant_fp8(hidden, ids, expert_map=expert_map)
        self.x, self.xs = p["permuted_hidden_states"], p["permuted_scales"]
        self.offset = p["expert_first_token_offset"]
        mp.moe_expert_gated_quant(self.x, self.xs, w_gated, s_gated, self.offset, self.h[:n],
                                  workspace=ws)
        mp.moe_quant_rows(self.h[:n], self.h_codes[:n], self.h_scales[:n], workspace=ws,
                          expert_first_token_offset=self.offset)
        mp.moe_expert_linear_quant(self.h_codes[:n], self.h_scales[:n], w_down, s_down,
                                   self.offset, self.y[:n], workspace=ws)
        return s.unpermute(self.y[:n], weights, out=self.out[:T])


def weights(g, code, E, N, K, parts):
    w = (torch.randn(E, N, K, generator=g, device=DEV) * 30).clamp(-120, 120).to(code)
    shape = qref.scale_shapes(code, 1, E, N, K, parts)[1]
    return w, (torch.rand(*shape, generator=g, device=DEV) + 0.5) / (30 * K ** 0.5)


@pytest.mark.parametrize("code", [E4M3, INT8], ids=["fp8", "int8"])
@pytest.mark.parametrize("T,H,F,E,K,local", [(1, 2048, 256, 8, 2, 8), (5, 256, 144, 8, 3, 8),
                                             (64, 512, 272, 32, 4, 8), (515, 384, 128, 10, 3, 10),
                                             (300, 1024, 2048, 4, 2, 4), (200, 256, 272, 16, 4, 5)])
def test_layer(T, H, F, E, K, local, code):
    g = torch.Generator(DEV).manual_seed(T + H)
    hidden = torch.randn(T, H, generator=g, device=DEV).to(BF)
    ids = torch.rand(T, E, generator=g, device=DEV).argsort(1)[:, :K].int().contiguous()
    mix = torch.softmax(torch.randn(T, K, generator=g, device=DEV), 1)
    expert_map = None
    if local < E:
        expert_map = torch.full((E,), -1, dtype=torch.int32, device=DEV)
        expert_map[torch.randperm(E, generator=g, device=DEV)[:local]] = \
            torch.arange(local, dtype=torch.int32, device=DEV)
    gated, down = weights(g, code, local, 2 * F, H, 2), weights(g, code, local, H, F, 1)
    layer = QuantLayer(code, *gated, *down, K, E, T + 3)
    out = layer.forward(hidden, ids, mix, expert_map).clone()
    assert layer.scratch.read_status() == 0
    n = int(layer.offset[-1])
    offset = layer.offset
    # the rows' codes are those of their tokens
    tokens = layer.scratch.permuted_idx[:n].long() // K
    want_codes, want_scales = qref.quantised(hidden, code)
    assert torch.equal(layer.x.view(torch.int8)[:n], want_codes.view(torch.int8)[tokens])
    assert torch.equal(layer.xs[:n], want_scales[tokens])
    ref.check(layer.h[:n], qref.gated(layer.x, layer.xs, *gated, offset, "silu"), BF, "h")
    want_codes, want_scales = qref.quantised(layer.h[:n], code)
    assert torch.equal(layer.h_codes.view(torch.int8)[:n], want_codes.view(torch.int8))
    assert torch.equal(layer.h_scales[:n], want_scales)
    want = qref.linear(layer.h_codes, layer.h_scales, *down, offset, "none")
    ref.check(layer.y[:n], want, BF, "y")
    inv = layer.scratch.inv_permuted_idx[:T * K].long()
    rows = layer.y[inv.clamp(min=0)].double() * (inv >= 0).double()[:, None]
    terms = rows.view(T, K, H) * mix.double()[:, :, None]
    bound = ref.Val(terms.sum(1), 2 * K * 2.0 ** -24 * terms.abs().sum(1))
    ref.check(out, bound, BF, "out")
    # captured and replayed on other tokens, beside a second graph on a layer of its own
    side, stream = QuantLayer(code, *gated, *down, K, E, T + 3), torch.cuda.Stream()
    static = torch.zeros_like(hidden)
    graphs = []
    for one in (layer, side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            one.forward(static, ids, mix, expert_map)
        graphs.append(graph)
    layer.out.zero_(), side.out.zero_()
    static.copy_(hidden)
    stream.wait_stream(torch.cuda.current_stream())
    graphs[0].replay()
    with torch.cuda.stream(stream):
        graphs[1].replay()
    torch.cuda.synchronize()
    assert torch.equal(layer.out[:T], out) and torch.equal(side.out[:T], out)
