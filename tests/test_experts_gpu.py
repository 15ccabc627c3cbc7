"""The expert operators against their 64-bit forms (tests/expert_ref.py), at
the row counts, sizes and contents where a tiled, ragged product can go wrong.
"""
import pytest
import torch

import expert_ref as ref
import moe_token_permute_gb300 as mp
from moe_token_permute_gb300 import _binding as b

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, HF = torch.bfloat16, torch.float16
SENTINEL = -77.0

# rows per expert: empty, single and ragged segments around every tile edge
COUNTS = {
    "one": [1],
    "empty_between": [0, 3, 0, 0, 17, 0],
    "decode": [1, 0, 2, 1, 0, 0, 5, 1],
    "tile_edges": [15, 16, 17, 127, 128, 129],
    "wide_edges": [255, 256, 257, 31, 33],
    "long": [700, 0, 1, 513],
    "no_rows": [0, 0, 0],
}
# (in or hidden, out or ffn)
SIZES = [(8, 8), (64, 128), (72, 40), (136, 264), (200, 136), (512, 384), (1000, 344)]


def normal(g, *shape, dtype, scale=1.0):
    return (torch.randn(*shape, generator=g, device=DEV) * scale).to(dtype)


def setup(counts, n_in, n_out, dtype, seed, tail=0):
    """Rows, weight [E, n_out, n_in] and offsets; `tail` rows behind the last
    expert's hold NaN and infinities."""
    g = torch.Generator(DEV).manual_seed(seed)
    n = sum(counts)
    offset = torch.tensor([0] + counts, dtype=torch.int64).cumsum(0).to(DEV)
    x = normal(g, n + tail, n_in, dtype=dtype)
    x[n:] = float("nan")
    if tail > 1:
        x[n] = float("inf")
    w = normal(g, len(counts), n_out, n_in, dtype=dtype, scale=n_in ** -0.5)
    return g, n, offset, x, w


def blank(*shape, dtype):
    return torch.full(shape, SENTINEL, dtype=dtype, device=DEV)


def untouched(t, n):
    assert (t[n:].float() == SENTINEL).all(), "rows of no expert were written"


def run_gated(counts, H, F, dtype, act, seed, tail=0, train=True):
    g, n, offset, x, w = setup(counts, H, 2 * F, dtype, seed, tail)
    R = n + tail
    out, preact = blank(R, F, dtype=dtype), blank(R, 2 * F, dtype=dtype)
    mp.moe_expert_gated(x, w, offset, out, activation=act, preact=preact)
    y, z = ref.gated(x, w, offset, act)
    ref.check(out[:n], y, dtype, "out")
    ref.check(preact[:n], z, dtype, "preact")
    untouched(out, n), untouched(preact, n)
    out2 = blank(R, F, dtype=dtype)
    mp.moe_expert_gated(x, w, offset, out2, activation=act)
    assert torch.equal(out, out2), "the result depends on whether preact is kept"
    if not train:
        return
    d = normal(g, R, F, dtype=dtype)
    d[n:] = float("nan")
    preact[n:] = float("nan")
    dz = blank(R, 2 * F, dtype=dtype)
    dx, dw = blank(R, H, dtype=dtype), blank(len(counts), 2 * F, H, dtype=dtype)
    mp.moe_expert_gated_backward(d, x, w, offset, preact, dz, activation=act, d_rows=dx,
                                 d_weight=dw)
    # stage by stage, each from what the kernels hold: the saved z, then dz
    ref.check(dz[:n], ref.gated_dz(d, ref.exact(preact[:n]), act), dtype, "d_preact")
    want_x, want_w, _ = ref.gradients(ref.exact(dz[:n]), x, w, offset)
    ref.check(dx[:n], want_x, dtype, "d_rows")
    ref.check(dw, want_w, dtype, "d_weight")
    untouched(dz, n), untouched(dx, n)
    # and through the whole chain
    full = ref.rounded(ref.gated_dz(d, ref.rounded(z, dtype), act), dtype)
    want_x, want_w, _ = ref.gradients(full, x, w, offset)
    ref.check(dx[:n], want_x, dtype, "d_rows from the inputs")
    ref.check(dw, want_w, dtype, "d_weight from the inputs")


def run_linear(counts, K, N, dtype, act, seed, bias, residual, tail=0):
    g, n, offset, x, w = setup(counts, K, N, dtype, seed, tail)
    R, E = n + tail, len(counts)
    bias = normal(g, E, N, dtype=dtype) if bias else None
    residual = normal(g, R, N, dtype=dtype) if residual else None
    out, preact = blank(R, N, dtype=dtype), blank(R, N, dtype=dtype)
    mp.moe_expert_linear(x, w, offset, out, bias=bias, activation=act, residual=residual,
                         preact=preact)
    y, z = ref.linear(x, w, offset, act, bias, residual)
    ref.check(out[:n], y, dtype, "out")
    ref.check(preact[:n], z, dtype, "preact")
    untouched(out, n), untouched(preact, n)
    d = normal(g, R, N, dtype=dtype)
    d[n:] = float("inf")
    dx, dw = blank(R, K, dtype=dtype), blank(E, N, K, dtype=dtype)
    db = blank(E, N, dtype=dtype)
    if act == "none":
        mp.moe_expert_linear_backward(d, x, w, offset, d_rows=dx, d_weight=dw, d_bias=db)
        dz = ref.exact(d[:n])
    else:
        dz_t = blank(R, N, dtype=dtype)
        mp.moe_expert_linear_backward(d, x, w, offset, activation=act, preact=preact,
                                      d_preact=dz_t, d_rows=dx, d_weight=dw, d_bias=db)
        saved = ref.exact(preact[:n])
        ref.check(dz_t[:n], ref.exact(d[:n]) * ref.act_grad(act, saved), dtype, "d_preact")
        untouched(dz_t, n)
        dz = ref.exact(dz_t[:n])
    want_x, want_w, want_b = ref.gradients(dz, x, w, offset)
    ref.check(dx[:n], want_x, dtype, "d_rows")
    ref.check(dw, want_w, dtype, "d_weight")
    ref.check(db, want_b, dtype, "d_bias")
    untouched(dx, n)


@pytest.mark.parametrize("sizes", SIZES, ids=str)
@pytest.mark.parametrize("counts", COUNTS, ids=str)
def test_gated(counts, sizes):
    dtype = (BF, HF)[(len(counts) + sizes[0] // 8) % 2]
    run_gated(COUNTS[counts], *sizes, dtype, "silu", seed=1, tail=0)


@pytest.mark.parametrize("sizes", SIZES, ids=str)
@pytest.mark.parametrize("counts", COUNTS, ids=str)
def test_linear(counts, sizes):
    dtype = (BF, HF)[(len(counts) + sizes[1] // 8) % 2]
    run_linear(COUNTS[counts], *sizes, dtype, "none", seed=2, bias=True, residual=False)


@pytest.mark.parametrize("dtype", [BF, HF], ids=str)
@pytest.mark.parametrize("act", ["none", "silu", "gelu", "relu"])
def test_activations(act, dtype):
    run_gated(COUNTS["tile_edges"], 136, 72, dtype, act, seed=3)
    for bias, residual in ((False, False), (True, True)):
        run_linear(COUNTS["tile_edges"], 72, 136, dtype, act, 4, bias, residual)


@pytest.mark.parametrize("dtype", [BF, HF], ids=str)
def test_rows_of_no_expert_are_neither_written_nor_felt(dtype):
    for counts in ("decode", "tile_edges", "no_rows"):
        run_gated(COUNTS[counts], 200, 136, dtype, "silu", seed=5, tail=70)
        run_linear(COUNTS[counts], 200, 136, dtype, "gelu", 6, True, True, tail=70)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("counts", [[5, 9, 3], [40, 130, 70], [300, 17, 290]], ids=str)
def test_an_experts_infinities_stay_with_it(counts, bad):
    """NaN and infinities in the middle expert's rows, weight and gradients
    reach no other expert's rows or weight gradient, whatever tiles they share."""
    H, F = 136, 72
    g, n, offset, x, w = setup(counts, H, 2 * F, BF, 7)
    lo, hi = counts[0], counts[0] + counts[1]
    d = normal(g, n, F, dtype=BF)
    clean = {}
    for name in ("clean", "bad"):
        if name == "bad":
            x[lo:hi], w[1], d[lo:hi] = bad, bad, bad
        out, pre, dz = (blank(n, c, dtype=BF) for c in (F, 2 * F, 2 * F))
        dx, dw = blank(n, H, dtype=BF), blank(3, 2 * F, H, dtype=BF)
        mp.moe_expert_gated(x, w, offset, out, preact=pre)
        mp.moe_expert_gated_backward(d, x, w, offset, pre, dz, d_rows=dx, d_weight=dw)
        y, dxl, dwl = blank(n, H, dtype=BF), blank(n, H, dtype=BF), blank(3, 2 * F, H, dtype=BF)
        db = blank(3, 2 * F, dtype=BF)
        mp.moe_expert_linear(x, w, offset, dz, activation="none")
        mp.moe_expert_linear_backward(pre, x, w, offset, d_rows=dxl, d_weight=dwl, d_bias=db)
        got = [torch.cat([t[:lo], t[hi:]]) for t in (out, pre, dz, dx, dxl)]
        got += [t[::2] for t in (dw, dwl, db)]
        if name == "clean":
            clean = [t.clone() for t in got]
    for a, c in zip(got, clean):
        assert torch.isfinite(a.float()).all()
        assert torch.equal(a, c)


def test_extreme_arguments_of_the_activations():
    """Large arguments give the limits: no NaN from an overflowing exponential."""
    x = torch.tensor([[1.0] + [0.0] * 7], device=DEV, dtype=BF)
    vals = [-1e30, -3e4, -100.0, -88.0, 88.0, 100.0, 3e4, 1e30]
    w = torch.zeros(1, 16, 8, device=DEV, dtype=BF)
    w[0, :8, 0] = torch.tensor(vals, device=DEV).to(BF)
    w[0, 8:, 0] = 1.0
    offset = torch.tensor([0, 1], device=DEV)
    for name in ("silu", "gelu", "relu"):
        out, pre, dz = (blank(1, c, dtype=BF) for c in (8, 16, 16))
        mp.moe_expert_gated(x, w, offset, out, activation=name, preact=pre)
        z = w[0, :8, 0].double()
        want = torch.where(z > 0, z, torch.zeros_like(z))
        assert torch.allclose(out[0].double(), want, rtol=2.0 ** -8, atol=1e-30)
        d = torch.ones(1, 8, device=DEV, dtype=BF)
        mp.moe_expert_gated_backward(d, None, w, offset, pre, dz, activation=name,
                                     d_rows=blank(1, 8, dtype=BF))
        assert torch.allclose(dz[0, :8].double(), (z > 0).double(), atol=1e-30)


@pytest.mark.parametrize("which", ["gated", "linear"])
def test_gradients_against_differences(which):
    """The kernels' gradients along random directions against central
    differences of the 64-bit forward pass.  The differences' own error is of
    order h^2 = 1e-8 and of rounding 1e-16/h; the kernels' is the bound that
    expert_ref builds, summed along the direction."""
    counts, H, F, act = [5, 0, 33, 18], 72, 40, "silu"
    cols = 2 * F if which == "gated" else F
    g, n, offset, x, w = setup(counts, H, cols, BF, 8)
    d = normal(g, n, F, dtype=BF)
    dx, dw = blank(n, H, dtype=BF), blank(4, cols, H, dtype=BF)
    out, pre, dz = blank(n, F, dtype=BF), blank(n, cols, dtype=BF), blank(n, cols, dtype=BF)
    form = (lambda a, c: ref.gated(a, c, offset, act)) if which == "gated" else \
        (lambda a, c: ref.linear(a, c, offset, act))
    _, z = form(x, w)
    zr = ref.rounded(z, BF)
    if which == "gated":
        mp.moe_expert_gated(x, w, offset, out, preact=pre)
        mp.moe_expert_gated_backward(d, x, w, offset, pre, dz, d_rows=dx, d_weight=dw)
        full = ref.rounded(ref.gated_dz(d, zr, act), BF)
    else:
        mp.moe_expert_linear(x, w, offset, out, activation=act, preact=pre)
        mp.moe_expert_linear_backward(d, x, w, offset, activation=act, preact=pre, d_preact=dz,
                                      d_rows=dx, d_weight=dw)
        full = ref.rounded(ref.exact(d) * ref.act_grad(act, zr), BF)
    want_x, want_w, _ = ref.gradients(full, x, w, offset)
    bounds = [ref.rounded(v, BF).e for v in (want_x, want_w)]
    h = 1e-4
    for i in range(4):
        vx = torch.randn(x.shape, generator=g, device=DEV).double() * (i != 1)
        vw = torch.randn(w.shape, generator=g, device=DEV).double() * (i != 0)
        loss = [(form(x.double() + s * h * vx, w.double() + s * h * vw)[0].v * d.double()).sum()
                for s in (1, -1)]
        slope = (loss[0] - loss[1]) / (2 * h)
        got = (dx.double() * vx).sum() + (dw.double() * vw).sum()
        room = (bounds[0] * vx.abs()).sum() + (bounds[1] * vw.abs()).sum()
        assert abs(got - slope) <= room + 1e-4 * (1 + abs(slope)), (i, got, slope, room)


def test_offsets_out_of_range_are_cut_and_flagged():
    H, F = 64, 40
    _, n, _, x, w = setup([10, 20, 30], H, 2 * F, BF, 9)
    ws = torch.zeros(mp.moe_permute_workspace_size(1, 1, 1), dtype=torch.uint8, device=DEV)
    mp.moe_permute_workspace_init(ws)
    for bad in ([0, 10, 30, 2 ** 40], [-5, 10, 30, 60], [0, 30, 10, 60]):
        offset = torch.tensor(bad, device=DEV)
        cut, prev = [], 0
        for e in range(3):
            lo = min(max(bad[e], 0), n)
            hi = min(max(bad[e + 1], lo), n)
            cut.append((lo, hi))
        out = blank(n, F, dtype=BF)
        mp.moe_expert_gated(x, w, offset, out, workspace=ws)
        assert mp.moe_read_status(ws) & mp.MOE_FLAG_OFFSET_OUT_OF_RANGE
        mp.moe_clear_status(ws)
        dw = blank(3, 2 * F, H, dtype=BF)
        mp.moe_expert_linear_backward(blank(n, 2 * F, dtype=BF), x, w, offset, d_weight=dw,
                                      workspace=ws)
        assert mp.moe_read_status(ws) & mp.MOE_FLAG_OFFSET_OUT_OF_RANGE
        mp.moe_clear_status(ws)
        assert torch.isfinite(dw.float()).all()
        lo, hi = cut[0]
        if bad[2] >= bad[1]:  # segments that do not overlap: the first one's rows are its own
            y, _ = ref.gated(x[lo:hi], w[:1], torch.tensor([0, hi - lo]), "silu")
            ref.check(out[lo:hi], y, BF, "out")
    good = torch.tensor([0, 10, 30, 60], device=DEV)
    mp.moe_expert_gated(x, w, good, out, workspace=ws)
    assert mp.moe_read_status(ws) == 0


def test_residual_may_be_the_output():
    g, n, offset, x, w = setup(COUNTS["tile_edges"], 136, 200, BF, 10)
    r = normal(g, n, 200, dtype=BF)
    y, _ = ref.linear(x, w, offset, "gelu", None, r)
    mp.moe_expert_linear(x, w, offset, r, activation="gelu", residual=r)
    ref.check(r, y, BF, "out")


def test_single_gradients():
    """Each gradient alone is what it is beside the others, and its unused
    inputs may be absent."""
    g, n, offset, x, w = setup([40, 3, 130], 136, 80, BF, 11)
    d = normal(g, n, 80, dtype=BF)
    full = [blank(n, 136, dtype=BF), blank(3, 80, 136, dtype=BF), blank(3, 80, dtype=BF)]
    mp.moe_expert_linear_backward(d, x, w, offset, d_rows=full[0], d_weight=full[1],
                                  d_bias=full[2])
    one = [torch.empty_like(t) for t in full]
    mp.moe_expert_linear_backward(d, None, w, offset, d_rows=one[0])
    mp.moe_expert_linear_backward(d, x, None, offset, d_weight=one[1])
    mp.moe_expert_linear_backward(d, None, w, offset, d_bias=one[2])
    for a, c in zip(full, one):
        assert torch.equal(a, c)


def test_repeats_streams_and_graphs_give_the_same_bits():
    counts, H, F = [130, 0, 17, 260, 1, 64], 264, 136
    g, n, offset, x, w = setup(counts, H, 2 * F, BF, 12)
    d = normal(g, n, F, dtype=BF)
    bufs = [blank(n, F, dtype=BF), blank(n, 2 * F, dtype=BF), blank(n, 2 * F, dtype=BF),
            blank(n, H, dtype=BF), blank(len(counts), 2 * F, H, dtype=BF)]

    def step(stream=None):
        mp.moe_expert_gated(x, w, offset, bufs[0], preact=bufs[1], stream=stream)
        mp.moe_expert_gated_backward(d, x, w, offset, bufs[1], bufs[2], d_rows=bufs[3],
                                     d_weight=bufs[4], stream=stream)

    step()
    want = [t.clone() for t in bufs]
    side = torch.cuda.Stream()
    for _ in range(5):
        for t in bufs:
            t.fill_(SENTINEL)
        side.wait_stream(torch.cuda.current_stream())
        step(side)  # another stream than the tensors' own
        torch.cuda.current_stream().wait_stream(side)
        assert all(torch.equal(a, c) for a, c in zip(bufs, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    for t in bufs:
        t.fill_(SENTINEL)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, c) for a, c in zip(bufs, want))


def test_matrices_beyond_32_bit_element_offsets():
    """Rows, outputs and weights whose element offsets pass 2^31 and 2^32 bytes."""
    H, F, R = 4096, 4096, 2 ** 19 + 40
    g = torch.Generator(DEV).manual_seed(13)
    x = torch.randn(R, H, generator=g, device=DEV, dtype=BF)
    w = normal(g, 3, 2 * 40, H, dtype=BF, scale=H ** -0.5)
    offset = torch.tensor([0, 8, R - 24, R], device=DEV)
    out = torch.empty(R, 40, device=DEV, dtype=BF)
    mp.moe_expert_gated(x, w, offset, out)
    y, _ = ref.gated(x[-24:], w[2:], torch.tensor([0, 24]), "silu")
    ref.check(out[-24:], y, BF, "out of the last rows")
    del out
    # wide output: the last expert's rows lie beyond 2^31 elements
    w2 = normal(g, 3, F, 8, dtype=BF, scale=8 ** -0.5)
    x2 = x.view(-1)[:R * 8].view(R, 8)
    y2 = torch.empty(R, F, device=DEV, dtype=BF)
    mp.moe_expert_linear(x2, w2, offset, y2)
    y, _ = ref.linear(x2[-24:], w2[2:], torch.tensor([0, 24]), "none")
    ref.check(y2[-24:], y, BF, "out of the last rows")
    # and as the operand of a weight gradient: d_weight of the last expert
    dw = torch.empty(3, 8, H, device=DEV, dtype=BF)
    mp.moe_expert_linear_backward(x2, x, None, offset, d_weight=dw)
    _, want, _ = ref.gradients(ref.exact(x2[-24:]), x[-24:], w[2:, :8], torch.tensor([0, 24]))
    ref.check(dw[2:], want, BF, "d_weight of the last expert")


# ---- the other ways a product is cut ---------------------------------------
# Few rows and a long contraction stream the weights (k_expert_decode); few tiles
# are shared by two pairs of SMs; few waves of tiles are cut narrower.

STREAMED = {
    "one": [1], "eight": [8], "spread": [1, 0, 2, 1, 0, 8, 5, 1], "crowded": [9, 0, 17, 6],
    "most": [20, 12, 0, 0], "few": [1, 0, 3, 2, 0, 4], "empty": [0, 0],
}


@pytest.mark.parametrize("K", [2048, 2112, 4096, 4160, 8256])
@pytest.mark.parametrize("counts", STREAMED, ids=str)
def test_few_rows(counts, K):
    dtype = (BF, HF)[K // 64 % 2]
    tail = 3 if counts == "spread" else 0
    run_gated(STREAMED[counts], K, 40, dtype, "silu", seed=20, tail=tail, train=False)
    run_linear(STREAMED[counts], K, 72, dtype, "gelu", 21, True, True, tail=tail)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_few_rows_an_experts_infinities_stay_with_it(bad):
    counts, K = [3, 5, 2], 4096
    g, n, offset, x, w = setup(counts, K, 80, BF, 22)
    outs = []
    for name in ("clean", "bad"):
        if name == "bad":
            x[3:8], w[1] = bad, bad
        h, y = blank(n, 40, dtype=BF), blank(n, 80, dtype=BF)
        mp.moe_expert_gated(x, w, offset, h)
        mp.moe_expert_linear(x, w, offset, y)
        outs.append([torch.cat([t[:3], t[8:]]) for t in (h, y)])
    for a, c in zip(*outs):
        assert torch.isfinite(a.float()).all() and torch.equal(a, c)


@pytest.mark.parametrize("rows", [9, 33, 100, 255, 256, 257, 300])
@pytest.mark.parametrize("K", [512, 520, 1096])
def test_few_tiles(rows, K):
    """One expert: half of the contraction in each of two pairs."""
    dtype = (BF, HF)[rows % 2]
    run_gated([rows], K, 520, dtype, "silu", seed=23)
    run_linear([rows], K, 520, dtype, "gelu", 24, True, True, tail=rows % 3)


@pytest.mark.parametrize("counts,N", [([1900], 2048), ([500], 4096), ([700, 0, 90, 1200], 1024),
                                      ([60] * 40, 512)], ids=str)
def test_few_waves(counts, N):
    run_linear(counts, 264, N, BF, "none", 25, False, False)


def test_many_experts():
    """As many as there may be, most of them without rows."""
    E = mp.MOE_MAX_LOCAL_EXPERTS
    counts = [0] * E
    for e, n in ((0, 3), (1, 130), (511, 1), (700, 40), (E - 1, 7)):
        counts[e] = n
    run_gated(counts, 72, 24, BF, "silu", seed=26, tail=5)
    run_linear(counts, 72, 24, HF, "relu", 27, True, False)
    few = [0] * E
    few[3], few[E - 1] = 4, 9
    run_gated(few, 2048, 16, BF, "silu", seed=28, train=False)


@pytest.mark.parametrize("n,K,E", [(30, 4096, 4), (100, 1024, 1)])
def test_bad_offsets_are_flagged_however_the_product_is_cut(n, K, E):
    _, _, _, x, w = setup([n] + [0] * (E - 1), K, 64, BF, 29)
    ws = torch.zeros(mp.moe_permute_workspace_size(1, 1, 1), dtype=torch.uint8, device=DEV)
    mp.moe_permute_workspace_init(ws)
    for bad in ([0, n, 0, n, n], [0, 2 ** 40, 5, 0, -3], [-1, n + 1, 0, n, 0]):
        offset = torch.tensor(bad[:E + 1] if E > 1 else [bad[0], bad[1] + 1], device=DEV)
        y = blank(n, 64, dtype=BF)
        mp.moe_expert_linear(x, w, offset, y, workspace=ws)
        assert mp.moe_read_status(ws) == mp.MOE_FLAG_OFFSET_OUT_OF_RANGE
        mp.moe_clear_status(ws)


# ---- moe_unpermute's gradient ----------------------------------------------

def run_combine(T, K, E, H, seed, local=None, off=0):
    g = torch.Generator(DEV).manual_seed(seed)
    local = E if local is None else local
    ids = torch.rand(T, E, generator=g, device=DEV).argsort(1)[:, :K].flatten()
    order = torch.argsort(ids, stable=True)
    order = order[ids[order] < local]
    n, R = order.numel(), T * K
    inv = torch.full((R,), -1, dtype=torch.int32, device=DEV)
    inv[order] = torch.arange(n, dtype=torch.int32, device=DEV)

    def at_offset(t):  # the same values `off` elements behind a 16-byte base
        buf = torch.empty(t.numel() + off, dtype=t.dtype, device=DEV)
        v = buf[off:].view(t.shape)
        return v.copy_(t)

    rows, d = at_offset(normal(g, R, H, dtype=BF)), at_offset(normal(g, T, H, dtype=BF))
    rows[n:] = float("nan")
    wts = torch.softmax(torch.randn(T, K, generator=g, device=DEV), 1)
    d_rows, dw = at_offset(blank(R, H, dtype=BF)), blank(T, K, dtype=torch.float32)
    mp.moe_unpermute_backward(d, rows, wts, inv, d_rows, dw)
    keep = inv >= 0
    p = inv[keep].long()
    tok = torch.arange(T, device=DEV).repeat_interleave(K)[keep]
    # one fp32 product rounded to bf16: the value is exact
    want = (wts.flatten()[keep][:, None] * d[tok].float()).to(BF)
    assert torch.equal(d_rows[p], want)
    untouched(d_rows, n)
    a, c = d[tok].double(), rows[p].double()
    dots, room = (a * c).sum(1), H * 2.0 ** -23 * (a * c).abs().sum(1)
    got = dw.flatten()
    assert ((got[keep].double() - dots).abs() <= room).all()
    assert (got[~keep] == 0).all()
    # one gradient at a time; d_rows over the rows themselves
    only = blank(T, K, dtype=torch.float32)
    mp.moe_unpermute_backward(d, rows, wts, inv, None, only)
    assert torch.equal(only, dw)
    fresh = at_offset(blank(R, H, dtype=BF))
    mp.moe_unpermute_backward(d, None, wts, inv, fresh, None)
    assert torch.equal(fresh.view(torch.int16), d_rows.view(torch.int16))
    mp.moe_unpermute_backward(d, rows, wts, inv, rows, only)
    assert torch.equal(only, dw) and torch.equal(rows[:n], d_rows[:n])


@pytest.mark.parametrize("T,K,E,H", [(1, 1, 1, 8), (1, 8, 128, 2048), (3, 2, 4, 1), (5, 3, 7, 33),
                                     (64, 6, 64, 2048), (33, 8, 256, 7168), (17, 32, 64, 264),
                                     (9, 2, 8, 9000), (700, 4, 16, 136)])
def test_unpermute_backward(T, K, E, H):
    run_combine(T, K, E, H, seed=T + H)


@pytest.mark.parametrize("off", [1, 2, 4])
def test_unpermute_backward_alignment_and_dropped_rows(off):
    run_combine(21, 6, 24, 200, seed=off, local=7, off=off)
    run_combine(21, 6, 24, 201, seed=off, local=1, off=off)


def test_unpermute_backward_flags_bad_indices():
    T, K, H = 6, 2, 64
    ws = torch.zeros(mp.moe_permute_workspace_size(1, 1, 1), dtype=torch.uint8, device=DEV)
    mp.moe_permute_workspace_init(ws)
    inv = torch.arange(T * K, dtype=torch.int32, device=DEV)
    inv[3], inv[8] = T * K, -2
    d, rows = (torch.randn(n, H, device=DEV).to(BF) for n in (T, T * K))
    dr, dw = blank(T * K, H, dtype=BF), blank(T, K, dtype=torch.float32)
    mp.moe_unpermute_backward(d, rows, torch.rand(T, K, device=DEV), inv, dr, dw, workspace=ws)
    assert mp.moe_read_status(ws) == mp.MOE_FLAG_INV_OUT_OF_RANGE
    assert dw.flatten()[3] == 0 and dw.flatten()[8] == 0
    assert (dr[3].float() == SENTINEL).all() and (dr[8].float() == SENTINEL).all()


def test_nothing_to_do():
    """No rows: nothing is written but the gradients of the parameters, as zeros."""
    w = torch.ones(2, 16, 8, device=DEV, dtype=BF)
    offset = torch.zeros(3, dtype=torch.int64, device=DEV)
    x, y, z = (torch.empty(0, c, device=DEV, dtype=BF) for c in (8, 8, 16))
    mp.moe_expert_gated(x, w, offset, y, preact=z)
    dw, db = blank(2, 16, 8, dtype=BF), blank(2, 16, dtype=BF)
    mp.moe_expert_gated_backward(y, x, w, offset, z, z, d_rows=x, d_weight=dw)
    assert (dw == 0).all()
    dw.fill_(SENTINEL)
    mp.moe_expert_linear(x, w, offset, z)
    mp.moe_expert_linear_backward(z, x, w, offset, d_rows=x, d_weight=dw, d_bias=db)
    assert (dw == 0).all() and (db == 0).all()
    mp.moe_unpermute_backward(torch.empty(0, 8, device=DEV, dtype=BF), x,
                              torch.empty(0, 2, device=DEV), torch.empty(0, dtype=torch.int32,
                                                                         device=DEV), x,
                              torch.empty(0, 2, device=DEV))
    assert b.MOE_OK == 0
