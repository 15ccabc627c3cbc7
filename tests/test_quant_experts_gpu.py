"""The products of 8-bit rows and weights against their 64-bit forms
(tests/quant_ref.py), at the row counts, sizes and contents where a tiled,
ragged product can go wrong.
"""
import pytest
import torch

import expert_ref as ref
import moe_token_permute_gb300 as mp
import quant_ref as qref
from moe_token_permute_gb300 import _binding as b

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, HF = torch.bfloat16, torch.float16
E4M3, INT8 = torch.float8_e4m3fn, torch.int8
SENTINEL = -77.0
FORMS = pytest.mark.parametrize("code", [E4M3, INT8], ids=["fp8", "int8"])

# rows per expert: empty, single and ragged segments around every tile edge
COUNTS = {
    "one": [1],
    "empty_between": [0, 3, 0, 0, 17, 0],
    "decode": [1, 0, 2, 1, 0, 0, 5, 1],
    "decode_groups": [8, 9, 0, 15],
    "tile_edges": [15, 16, 17, 127, 128, 129],
    "wide_edges": [255, 256, 257, 31, 33],
    "long": [700, 0, 1, 513],
    "no_rows": [0, 0, 0],
}
# (in or hidden, out or ffn)
SIZES = [(16, 8), (64, 128), (80, 40), (144, 264), (208, 136), (512, 384), (1008, 344),
         (272, 648)]


def make_codes(g, code, *shape):
    """Codes of every size, NaN and -128 not among them."""
    if code == INT8:
        return torch.randint(-127, 128, shape, generator=g, device=DEV).to(INT8)
    return (torch.randn(*shape, generator=g, device=DEV) * 100).clamp(-448, 448).to(E4M3)


def setup(counts, K, N, code, parts, seed, tail=0):
    """Rows, weight [E, N, K], their scales and offsets; `tail` rows behind the last
    expert's hold NaN codes, and infinite and NaN scales."""
    g = torch.Generator(DEV).manual_seed(seed)
    n, E = sum(counts), len(counts)
    offset = torch.tensor([0] + counts, dtype=torch.int64).cumsum(0).to(DEV)
    x, w = make_codes(g, code, n + tail, K), make_codes(g, code, E, N, K)
    shapes = qref.scale_shapes(code, n + tail, E, N, K, parts)
    largest = 60.0 if code == INT8 else 100.0
    xs, ws = (torch.rand(*s, generator=g, device=DEV) + 0.2 for s in shapes)
    xs, ws = xs / largest, ws / largest / K ** 0.5
    x.view(torch.int8)[n:] = 0x7f
    xs[n:] = float("nan")
    if tail > 1:
        xs[n] = float("inf")
    return g, n, offset, x, xs, w, ws


def blank(*shape, dtype):
    return torch.full(shape, SENTINEL, dtype=dtype, device=DEV)


def untouched(t, n):
    assert (t[n:].float() == SENTINEL).all(), "rows of no expert were written"


def run_gated(counts, H, F, code, dtype, act, seed, tail=0):
    _, n, offset, x, xs, w, ws = setup(counts, H, 2 * F, code, 2, seed, tail)
    out = blank(n + tail, F, dtype=dtype)
    mp.moe_expert_gated_quant(x, xs, w, ws, offset, out, activation=act)
    ref.check(out[:n], qref.gated(x, xs, w, ws, offset, act), dtype, "out")
    untouched(out, n)


def run_linear(counts, K, N, code, dtype, act, seed, bias, residual, tail=0):
    g, n, offset, x, xs, w, ws = setup(counts, K, N, code, 1, seed, tail)
    bias = torch.randn(len(counts), N, generator=g, device=DEV).to(dtype) if bias else None
    residual = torch.randn(n + tail, N, generator=g, device=DEV).to(dtype) if residual else None
    out = blank(n + tail, N, dtype=dtype)
    mp.moe_expert_linear_quant(x, xs, w, ws, offset, out, bias=bias, activation=act,
                               residual=residual)
    want = qref.linear(x, xs, w, ws, offset, act, bias, residual)
    ref.check(out[:n], want, dtype, "out")
    untouched(out, n)
    if residual is not None:  # into the residual itself
        mp.moe_expert_linear_quant(x, xs, w, ws, offset, residual, bias=bias, activation=act,
                                   residual=residual)
        assert torch.equal(residual[:n], out[:n])


@FORMS
@pytest.mark.parametrize("counts", list(COUNTS))
@pytest.mark.parametrize("size", SIZES, ids=lambda s: f"{s[0]}x{s[1]}")
def test_gated(size, counts, code):
    i = SIZES.index(size) + list(COUNTS).index(counts)
    run_gated(COUNTS[counts], *size, code, (BF, HF)[i % 2], ("silu", "gelu", "relu", "none")[i % 4],
              i, tail=i % 3)


@FORMS
@pytest.mark.parametrize("counts", list(COUNTS))
@pytest.mark.parametrize("size", SIZES, ids=lambda s: f"{s[0]}x{s[1]}")
def test_linear(size, counts, code):
    i = SIZES.index(size) * 3 + list(COUNTS).index(counts)
    run_linear(COUNTS[counts], *size, code, (HF, BF)[i % 2], ("none", "gelu", "relu", "silu")[i % 4],
               i, bias=i % 3 != 0, residual=i % 2 == 0, tail=(i + 1) % 3)


@FORMS
@pytest.mark.parametrize("rows", [1, 2, 8, 16, 32, 33, 64])
@pytest.mark.parametrize("K,N", [(2048, 256), (4096, 136), (8192, 64), (4112, 72), (14336, 48)])
def test_few_rows_over_long_contractions(K, N, rows, code):
    """What decoding sends: rows of a few experts, weights streamed."""
    counts = [rows // 2, 0, rows - rows // 2 - rows // 3, rows // 3]
    run_gated(counts, K, N, code, BF, "silu", rows + K, tail=2)
    run_linear(counts, K, N, code, HF, "none", rows + N, rows % 2 == 0, True, tail=1)


@FORMS
@pytest.mark.parametrize("E,rows", [(16, 127), (16, 128), (16, 129), (130, 129), (130, 255),
                                    (130, 256), (130, 257)])
def test_rows_of_many_experts(E, rows, code):
    """As many groups of rows as a short call can have, and one more."""
    counts = [rows // E + (e < rows % E) for e in range(E)]
    run_gated(counts, 7168, 40, code, BF, "silu", rows, tail=1)
    run_linear(counts, 7296, 72, code, HF, "none", rows, False, True, tail=2)


@FORMS
@pytest.mark.parametrize("rows", [1, 15, 64, 130, 300, 1000])
@pytest.mark.parametrize("K,N", [(4096, 512), (2064, 4096)])
def test_one_expert(K, N, rows, code):
    """A dense layer, few tiles of a long contraction among them."""
    run_linear([rows], K, N, code, BF, "gelu", rows, True, True, tail=3)
    run_gated([rows], K, N, code, HF, "silu", rows)


@FORMS
def test_many_experts(code):
    counts = [(7 * e) % 23 * (e % 3) for e in range(1024)]
    run_gated(counts, 128, 64, code, BF, "silu", 1)
    run_linear(counts, 64, 128, code, BF, "none", 2, True, False)


@FORMS
@pytest.mark.parametrize("extreme", ["codes", "scales"])
def test_the_largest_values(extreme, code):
    """Codes at their limits (-128 too), where sums pass 2^24; scales far from one."""
    K, N = 4096, 256
    for counts in ([5, 3], [200, 70]):
        _, n, offset, x, xs, w, ws = setup(counts, K, N, code, 1, 3)
        if extreme == "codes":
            x.view(torch.int8).copy_(torch.full_like(x.view(torch.int8), -128 if code == INT8
                                                     else 0x7e))
            w.view(torch.int8).copy_(torch.full_like(w.view(torch.int8), -128 if code == INT8
                                                     else -2))  # 0xfe: -448
            xs /= 1e3
        else:
            xs *= 2.0 ** 60
            ws *= 2.0 ** -60
        out = blank(n, N, dtype=BF)
        mp.moe_expert_linear_quant(x, xs, w, ws, offset, out)
        ref.check(out, qref.linear(x, xs, w, ws, offset, "none"), BF, "out")


@FORMS
@pytest.mark.parametrize("counts", [[3, 4], [140, 90]], ids=["few", "many"])
def test_infinities_and_nan_stay_in_their_row(counts, code):
    """A row or a channel that is not finite makes its own outputs not finite and
    leaves all others as they were."""
    K, N = 2048, 264
    _, n, offset, x, xs, w, ws = setup(counts, K, N, code, 1, 4)
    clean, out = blank(n, N, dtype=BF), blank(n, N, dtype=BF)
    mp.moe_expert_linear_quant(x, xs, w, ws, offset, clean)
    xs[1, 0] = float("nan")
    xs[counts[0] + 2, -1] = float("inf")
    if code == E4M3:
        x.view(torch.int8)[2, 700] = 0x7f
    ws[1, 0] = float("nan")  # of the second expert: features 0..127, or channel 0
    mp.moe_expert_linear_quant(x, xs, w, ws, offset, out)
    bad = torch.zeros(n, N, dtype=torch.bool, device=DEV)
    bad[1] = bad[counts[0] + 2] = True
    if code == E4M3:
        bad[2] = True
    bad[counts[0]:, :128 if code == E4M3 else 1] = True
    assert not torch.isfinite(out[bad]).any()
    assert torch.equal(out[~bad], clean[~bad])


@pytest.mark.parametrize("counts", [[3, 4], [140, 90]], ids=["few", "many"])
@pytest.mark.parametrize("K", [2048, 2176, 14336 + 128])
def test_an_infinite_last_scale(K, counts):
    """What a ring's last stage has behind the contraction adds nothing, not even NaN."""
    _, n, offset, x, xs, w, ws = setup(counts, K, 256, E4M3, 1, 6)
    x.copy_(x.float().abs().clamp(min=1).to(E4M3)), w.copy_(w.float().abs().clamp(min=1).to(E4M3))
    xs[:, -1] = float("inf")
    out = blank(n, 256, dtype=BF)
    mp.moe_expert_linear_quant(x, xs, w, ws, offset, out)
    assert (out == float("inf")).all()


@FORMS
def test_other_experts_cannot_be_seen(code):
    """Segments that end inside a tile, the next expert's rows being NaN."""
    K, N = 256, 128
    counts = [5, 20, 131, 40]
    _, n, offset, x, xs, w, ws = setup(counts, K, N, code, 2, 5)
    clean, out = blank(n, N // 2, dtype=BF), blank(n, N // 2, dtype=BF)
    mp.moe_expert_gated_quant(x, xs, w, ws, offset, clean)
    for e in (0, 2):
        lo, hi = offset[e].item(), offset[e + 1].item()
        x2, xs2 = x.clone(), xs.clone()
        x2.view(torch.int8)[:lo] = x2.view(torch.int8)[hi:] = 0x7f
        xs2[:lo] = xs2[hi:] = float("nan")
        w2, ws2 = w.clone(), ws.clone()
        ws2[:e] = ws2[e + 1:] = float("inf")
        mp.moe_expert_gated_quant(x2, xs2, w2, ws2, offset, out)
        assert torch.equal(out[lo:hi], clean[lo:hi])


@FORMS
@pytest.mark.parametrize("K,R,from0,to0,c", [(256, 70, 50, 60, 10), (4096, 12, 7, 9, 4)],
                         ids=["tiles", "streamed"])
def test_malformed_offsets(K, R, from0, to0, c, code):
    N = 136
    _, _, _, x, xs, w, ws = setup([R, 0, 0], K, N, code, 1, 6)
    status = torch.zeros(mp.moe_permute_workspace_size(1, 1, 1), dtype=torch.uint8, device=DEV)
    mp.moe_permute_workspace_init(status)
    for ends, cut in (([from0, to0, 0, c], [(from0, to0), (to0, to0), (0, c)]),
                      ([-3, c + 2, c, 2 ** 40], [(0, c + 2), (c + 2, c + 2), (c, R)]),
                      ([R + 1, R + 9, 2 ** 33, -1], [(R, R)] * 3)):
        offset = torch.tensor(ends, device=DEV)
        out = blank(R, N, dtype=BF)
        mp.moe_clear_status(status)
        mp.moe_expert_linear_quant(x, xs, w, ws, offset, out, workspace=status)
        assert mp.moe_read_status(status) == b.MOE_FLAG_OFFSET_OUT_OF_RANGE
        overlap = any(lo < h2 and l2 < hi for i, (lo, hi) in enumerate(cut)
                      for l2, h2 in cut[i + 1:])
        used = torch.zeros(R, dtype=torch.bool, device=DEV)
        for e, (lo, hi) in enumerate(cut):
            used[lo:hi] = True
            if not overlap:
                want = qref.product(x[lo:hi], xs[lo:hi], w[e], ws[e], 1)
                ref.check(out[lo:hi], want, BF, f"expert {e}")
        assert (out[~used] == SENTINEL).all()


@FORMS
@pytest.mark.parametrize("K,R", [(256, 70), (4096, 12)], ids=["tiles", "streamed"])
def test_segments_that_all_overlap(K, R, code):
    """Far more groups of rows than rows: the outputs are undefined, but only they."""
    E, N = 600, 136
    _, _, _, x, xs, w, ws = setup([R] + [0] * (E - 1), K, N, code, 1, 10)
    status = torch.zeros(mp.moe_permute_workspace_size(1, 1, 1), dtype=torch.uint8, device=DEV)
    mp.moe_permute_workspace_init(status)
    offset = torch.tensor([R * (e % 2) for e in range(E + 1)], device=DEV)
    out = blank(R + 64, N, dtype=BF)
    mp.moe_expert_linear_quant(x, xs, w, ws, offset, out[:R], workspace=status)
    assert mp.moe_read_status(status) == b.MOE_FLAG_OFFSET_OUT_OF_RANGE
    untouched(out, R)


@FORMS
@pytest.mark.parametrize("counts", [[2, 1, 5], [300, 17, 260]], ids=["few", "many"])
def test_graph_streams_and_repeats_give_the_same_bits(counts, code):
    K, F = 4096, 512
    _, n, offset, x, xs, w, ws = setup(counts, K, 2 * F, code, 2, 7)
    first = blank(n, F, dtype=BF)
    mp.moe_expert_gated_quant(x, xs, w, ws, offset, first)
    torch.cuda.synchronize()
    outs = [blank(n, F, dtype=BF) for _ in range(3)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    mp.moe_expert_gated_quant(x, xs, w, ws, offset, outs[0])
    mp.moe_expert_gated_quant(x, xs, w, ws, offset, outs[1], stream=side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mp.moe_expert_gated_quant(x, xs, w, ws, offset, outs[2])
    outs[2].fill_(SENTINEL)
    graph.replay()
    torch.cuda.synchronize()
    for out in outs:
        assert torch.equal(out, first)


@FORMS
def test_elements_beyond_32_bits(code):
    """Codes of rows, weights and outputs at byte offsets beyond 2^32."""
    K, N, E = 16384, 8, 2
    R = 2 ** 32 // K + 40
    g = torch.Generator(DEV).manual_seed(8)
    x = torch.zeros(R, K, dtype=torch.int8, device=DEV)
    x[-40:] = make_codes(g, code, 40, K).view(torch.int8)
    x = x.view(code)
    w = make_codes(g, code, E, N, K)
    shapes = qref.scale_shapes(code, R, E, N, K, 1)
    xs, ws = (torch.rand(*s, generator=g, device=DEV) / 128 for s in shapes)
    offset = torch.tensor([0, R - 30, R], device=DEV)
    out = blank(R, N, dtype=BF)
    mp.moe_expert_linear_quant(x, xs, w, ws, offset, out)
    tail = torch.tensor([0, 10, 40], device=DEV)
    want = qref.linear(x[-40:], xs[-40:], w, ws, tail, "none")
    ref.check(out[-40:], want, BF, "out")
    assert (out[:-40] == 0).all()
    del x, out
    E, N = 260, 1024  # 2^32 bytes of weights
    w = torch.zeros(E, N, K, dtype=torch.int8, device=DEV)
    w[-1] = make_codes(g, code, N, K).view(torch.int8)
    w = w.view(code)
    for rows in (5, 70, 300):
        x = make_codes(g, code, rows, K)
        shapes = qref.scale_shapes(code, rows, E, N, K, 1)
        xs, ws = (torch.rand(*s, generator=g, device=DEV) / 128 for s in shapes)
        offset = torch.zeros(E + 1, dtype=torch.int64, device=DEV)
        offset[-1] = rows
        out = blank(rows, N, dtype=BF)
        mp.moe_expert_linear_quant(x, xs, w, ws, offset, out)
        want = qref.product(x, xs, w[-1], ws[-1], 1)
        ref.check(out, want, BF, "out")


@FORMS
def test_no_rows(code):
    _, _, offset, x, xs, w, ws = setup([0, 0], 64, 32, code, 2, 9)
    mp.moe_expert_gated_quant(x, xs, w, ws, offset, blank(0, 16, dtype=BF))


@pytest.mark.parametrize("counts", [[3, 4], [140, 90]], ids=["few", "many"])
@pytest.mark.parametrize("K", [2048, 2176, 4096 + 384, 14336 + 128])
def test_an_infinite_last_weight_scale(K, counts):
    """The same where the scales of the weights' last blocks are infinite: in the linear
    product, and of the gate rows, the up rows or both."""
    _, n, offset, x, xs, w, ws = setup(counts, K, 256, E4M3, 2, 6)
    x.copy_(x.float().abs().clamp(min=1).to(E4M3)), w.copy_(w.float().abs().clamp(min=1).to(E4M3))
    out, h = blank(n, 256, dtype=BF), blank(n, 128, dtype=BF)
    for blocks in ([0], [1], [0, 1]):  # of 128 features: gate and up rows, if gated
        scales = ws.clone()
        scales[:, blocks, -1] = float("inf")
        mp.moe_expert_linear_quant(x, xs, w, scales, offset, out)
        mp.moe_expert_gated_quant(x, xs, w, scales, offset, h)
        for block in (0, 1):
            part = out[:, 128 * block:128 * block + 128]
            assert (part == float("inf")).all() if block in blocks else part.isfinite().all()
        assert (h == float("inf")).all()
