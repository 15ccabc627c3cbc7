"""The expert products on long segments: element offsets that pass 2^31 in the
middle of one expert's rows, and more than a panel of column blocks beside
several row blocks."""
import pytest
import torch

import expert_ref as ref
import moe_token_permute_gb300 as mp

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16

WIDE = 4096
ROWS = 2 ** 19 + 40  # element 2^31 of a [ROWS, WIDE] matrix is row 2^19
OFFSET = [0, 8, ROWS - 24, ROWS]
# rows of the middle expert around 2^30 and 2^31 elements
LOOK = torch.cat([torch.arange(2 ** 18 - 20, 2 ** 18 + 20), torch.arange(2 ** 19 - 40, ROWS - 24)])


def normal(g, *shape, scale=1.0):
    t = torch.randn(*shape, generator=g, device=DEV, dtype=BF)
    return t if scale == 1.0 else t.mul_(scale)


def of_middle(w, rows):
    """product(rows, the middle expert's w), w as [out, in]."""
    return ref.product(ref.exact(rows), ref.exact(w))


def test_forward_across_32_bit_offsets():
    g = torch.Generator(DEV).manual_seed(1)
    at, offset = LOOK.to(DEV), torch.tensor(OFFSET, device=DEV)
    x = normal(g, ROWS, WIDE)
    w = normal(g, 3, 2 * 40, WIDE, scale=WIDE ** -0.5)
    out = torch.empty(ROWS, 40, device=DEV, dtype=BF)
    mp.moe_expert_gated(x, w, offset, out)
    gate, up = ref.split(of_middle(w[1], x[at]), 40)
    ref.check(out[at], ref.act("silu", gate) * up, BF, "gated")
    # wide results, with a residual as wide
    narrow, w = x.view(-1)[:ROWS * 8].view(ROWS, 8), normal(g, 3, WIDE, 8, scale=8 ** -0.5)
    y, pre = (torch.empty(ROWS, WIDE, device=DEV, dtype=BF) for _ in range(2))
    mp.moe_expert_linear(narrow, w, offset, y, activation="relu", residual=x, preact=pre)
    z = of_middle(w[1], narrow[at])
    ref.check(pre[at], z, BF, "preact")
    ref.check(y[at], ref.act("relu", z) + ref.exact(x[at]), BF, "out")


def test_gradients_across_32_bit_offsets():
    g = torch.Generator(DEV).manual_seed(2)
    at, offset = LOOK.to(DEV), torch.tensor(OFFSET, device=DEV)
    wide, narrow = normal(g, ROWS, WIDE), normal(g, ROWS, 8)
    # wide dz, formed from a wide pre-activation
    pre, dz = normal(g, ROWS, WIDE), torch.empty(ROWS, WIDE, device=DEV, dtype=BF)
    w = normal(g, 3, WIDE, 8, scale=WIDE ** -0.5)
    dx = torch.empty(ROWS, 8, device=DEV, dtype=BF)
    mp.moe_expert_linear_backward(wide, None, w, offset, activation="silu", preact=pre, d_preact=dz,
                                  d_rows=dx)
    ref.check(dz[at], ref.exact(wide[at]) * ref.act_grad("silu", ref.exact(pre[at])), BF, "dz")
    ref.check(dx[at], of_middle(w[1].t(), dz[at]), BF, "d_rows")
    # wide d_rows, over dz
    w = normal(g, 3, 8, WIDE, scale=8 ** -0.5)
    mp.moe_expert_linear_backward(narrow, None, w, offset, d_rows=dz)
    ref.check(dz[at], of_middle(w[1].t(), narrow[at]), BF, "wide d_rows")
    # d_weight and d_bias of dz that is zero but for those rows: as many terms
    few = torch.zeros(ROWS, 8, device=DEV, dtype=BF)
    few[at] = narrow[at]
    dw = torch.empty(3, 8, WIDE, device=DEV, dtype=BF)
    mp.moe_expert_linear_backward(few, wide, None, offset, d_weight=dw)
    want = ref.product(ref.exact(few[at].t()), ref.exact(wide[at].t()))
    ref.check(dw[1], want, BF, "d_weight")
    wide.zero_()
    wide[at] = pre[at]
    dw, db = torch.empty(3, WIDE, 8, device=DEV, dtype=BF), torch.empty(3, WIDE, device=DEV, dtype=BF)
    mp.moe_expert_linear_backward(wide, narrow, None, offset, d_weight=dw, d_bias=db)
    ref.check(dw[1], ref.product(ref.exact(wide[at].t()), ref.exact(narrow[at].t())), BF,
              "d_weight of wide dz")
    d = wide[at].double()
    ref.check(db[1], ref.Val(d.sum(0), d.shape[0] * 2.0 ** -23 * d.abs().sum(0)), BF, "d_bias")


# From six waves of tiles on, blocks have 256 columns: 79 and 157 of them, and the
# last is ragged.
@pytest.mark.parametrize("counts", [[20100], [100, 0, 20001, 7]], ids=str)
def test_linear_in_panels(counts):
    g = torch.Generator(DEV).manual_seed(3)
    K, N = 72, 1544  # seven row blocks of 256
    offset = torch.tensor([0] + counts, device=DEV).cumsum(0)
    x, w = normal(g, sum(counts), K), normal(g, len(counts), N, K, scale=K ** -0.5)
    out = torch.empty(sum(counts), N, device=DEV, dtype=BF)
    mp.moe_expert_linear(x, w, offset, out)
    y, _ = ref.linear(x, w, offset, "none")
    ref.check(out, y, BF, "out")
    # d_rows: row blocks of the weight's other side
    w, dx = w.transpose(1, 2).contiguous(), torch.empty_like(out)
    mp.moe_expert_linear_backward(x, None, w, offset, d_rows=dx)
    assert torch.equal(dx, out)  # the same sums, in the same order


def test_gated_in_panels():
    g = torch.Generator(DEV).manual_seed(4)
    counts, H, F = [40100], 72, 392  # four row blocks of 128
    offset = torch.tensor([0] + counts, device=DEV).cumsum(0)
    x, w = normal(g, counts[0], H), normal(g, 1, 2 * F, H, scale=H ** -0.5)
    out = torch.empty(counts[0], F, device=DEV, dtype=BF)
    mp.moe_expert_gated(x, w, offset, out)
    y, _ = ref.gated(x, w, offset, "silu")
    ref.check(out, y, BF, "out")


def test_d_weight_in_panels():
    g = torch.Generator(DEV).manual_seed(5)
    counts, K, N = [130, 0, 70], 2600, 776  # eleven column blocks, four row blocks
    offset = torch.tensor([0] + counts, device=DEV).cumsum(0)
    x, d = normal(g, 200, K), normal(g, 200, N)
    dw = torch.empty(3, N, K, device=DEV, dtype=BF)
    mp.moe_expert_linear_backward(d, x, None, offset, d_weight=dw)
    _, want, _ = ref.gradients(ref.exact(d), x, dw, offset)
    ref.check(dw, want, BF, "d_weight")
