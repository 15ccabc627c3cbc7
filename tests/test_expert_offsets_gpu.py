"""The expert operators' backward passes where the offsets are not the usual
ones: decreasing, so that the cut segments leave gaps, or not starting at 0.

A row belongs to the experts whose cut segment [lo, hi) holds it, lo and hi
being the offsets cut to [0, num_rows] and hi to at least lo.  All segments here
are apart, so every result has one value.
"""
import pytest
import torch

import expert_ref as ref
import moe_token_permute_gb300 as mp

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16
NAN, SENTINEL = float("nan"), -77.0

# offsets, rows
OFFSETS = {
    "ends_lower": ([0, 60, 30], 60),
    "falls_to_nothing": ([0, 70, -5], 70),
    "gap_between": ([50, 60, 0, 10], 70),
    "falls_first": ([10, 5, 40, 20], 64),
    "starts_late": ([5, 20, 40], 40),
    "beyond_the_rows": ([3, 200, 150, 2 ** 40], 150),
}


def cut(offset, n):
    out = []
    for a, z in zip(offset[:-1], offset[1:]):
        lo = min(max(a, 0), n)
        out.append((lo, min(max(z, lo), n)))
    return out


def members(segments, n):
    m = torch.zeros(n, dtype=torch.bool, device=DEV)
    for lo, hi in segments:
        m[lo:hi] = True
    return m


def rows_of(val, index):
    return ref.Val(val.v[index], val.e[index])


def check_products(dz, x, w, segments, dx, dw, db=None):
    """d_rows, d_weight and d_bias from the dz that the call wrote."""
    for e, (lo, hi) in enumerate(segments):
        d = ref.exact(dz[lo:hi])
        ref.check(dx[lo:hi], ref.product(d, ref.exact(w[e].t())), BF, f"d_rows of {e}")
        ref.check(dw[e], ref.product(ref.transpose(d), ref.exact(x[lo:hi].t())), BF,
                  f"d_weight of {e}")
        if db is not None:
            s = ref.Val(d.v.sum(0), max(1, hi - lo) * 2.0 ** -23 * d.v.abs().sum(0))
            ref.check(db[e], s, BF, f"d_bias of {e}")


@pytest.mark.parametrize("name", OFFSETS)
@pytest.mark.parametrize("form", ["gated", "linear"])
def test_dz_covers_the_cut_segments_and_nothing_else(form, name):
    values, n = OFFSETS[name]
    segments = cut(values, n)
    inside = members(segments, n)
    E, K, W = len(segments), 72, 264  # 264: a block of columns that is not full
    cols = 2 * W if form == "gated" else W
    g = torch.Generator(DEV).manual_seed(n)

    def normal(*shape, scale=1.0):
        return (torch.randn(*shape, generator=g, device=DEV) * scale).to(BF)

    x, w, z, d = normal(n, K), normal(E, cols, K, scale=K ** -0.5), normal(n, cols), normal(n, W)
    for t in (x, z, d):  # rows of no expert reach nothing
        t[~inside] = NAN
    offset = torch.tensor(values, device=DEV)
    # a dz that is read without having been written shows as NaN
    dz, dx = (torch.full((n, c), NAN, dtype=BF, device=DEV) for c in (cols, K))
    dz[~inside], dx[~inside] = SENTINEL, SENTINEL
    dw, db = torch.empty_like(w), torch.empty(E, cols, dtype=BF, device=DEV)
    if form == "gated":
        mp.moe_expert_gated_backward(d, x, w, offset, z, dz, d_rows=dx, d_weight=dw)
        db = None
        want = ref.gated_dz(d, ref.exact(z), "silu")
    else:
        mp.moe_expert_linear_backward(d, x, w, offset, activation="gelu", preact=z, d_preact=dz,
                                      d_rows=dx, d_weight=dw, d_bias=db)
        want = ref.exact(d) * ref.act_grad("gelu", ref.exact(z))
    assert (dz[~inside] == SENTINEL).all(), "d_preact of rows of no expert was written"
    assert (dx[~inside] == SENTINEL).all(), "d_rows of rows of no expert was written"
    ref.check(dz[inside], rows_of(want, inside), BF, "d_preact")
    check_products(dz, x, w, segments, dx, dw, db)


@pytest.mark.parametrize("what", ["d_bias", "d_preact of linear", "d_preact of gated"])
@pytest.mark.parametrize("values", [[0, 60, 30], [0, 20, 2 ** 40], [-1, 20, 60]], ids=str)
def test_malformed_offsets_are_flagged_without_a_product(values, what):
    n, K, N = 60, 16, 64
    x, w = (torch.zeros(*s, dtype=BF, device=DEV) for s in ((n, K), (2, N, K)))
    d, dz = (torch.ones(n, N, dtype=BF, device=DEV) for _ in range(2))
    ws = torch.zeros(mp.moe_permute_workspace_size(1, 1, 1), dtype=torch.uint8, device=DEV)
    mp.moe_permute_workspace_init(ws)
    for offset, flags in ((values, mp.MOE_FLAG_OFFSET_OUT_OF_RANGE), ([0, 20, 60], 0)):
        offset = torch.tensor(offset, device=DEV)
        if what == "d_bias":
            db = torch.empty(2, N, dtype=BF, device=DEV)
            mp.moe_expert_linear_backward(d, x, w, offset, d_bias=db, workspace=ws)
            sizes = [hi - lo for lo, hi in cut(offset.tolist(), n)]
            assert db[:, 0].tolist() == sizes  # sums of ones, below 2^8: exact
        elif what == "d_preact of linear":
            mp.moe_expert_linear_backward(d, x, w, offset, activation="relu", preact=d, d_preact=dz,
                                          workspace=ws)
        else:
            mp.moe_expert_gated_backward(d[:, :N // 2].contiguous(), x, w, offset, d, dz,
                                         workspace=ws)
        assert mp.moe_read_status(ws) == flags
        mp.moe_clear_status(ws)


def test_bias_gradient_needs_no_weight():
    g = torch.Generator(DEV).manual_seed(3)
    d = torch.randn(50, 72, generator=g, device=DEV).to(BF)
    offset = torch.tensor([0, 17, 17, 50], device=DEV)
    db, beside = (torch.empty(3, 72, dtype=BF, device=DEV) for _ in range(2))
    mp.moe_expert_linear_backward(d, None, None, offset, d_bias=db)
    w = torch.zeros(3, 72, 8, dtype=BF, device=DEV)
    mp.moe_expert_linear_backward(d, None, w, offset, d_bias=beside)
    assert torch.equal(db, beside)
    for e, (lo, hi) in enumerate(cut(offset.tolist(), 50)):
        v = d[lo:hi].double()
        ref.check(db[e], ref.Val(v.sum(0), max(1, hi - lo) * 2.0 ** -23 * v.abs().sum(0)), BF, e)
