"""int8 products in tiles, against whole numbers: with scales that are powers of two and
sums below 2^24 a result is the exact sum, rounded once.  Row counts, sizes and experts
are such that tiles have one and two halves of features, share a contraction, and have
every number of columns; and the bounded waits of tiles of two halves, through the debug
build.
"""
import ctypes
import time

import pytest
import torch

import expert_ref as ref
import moe_token_permute_gb300 as mp
import quant_ref as qref
from moe_token_permute_gb300 import _binding as b

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, HF = torch.bfloat16, torch.float16


def operands(counts, K, N, seed):
    g = torch.Generator(DEV).manual_seed(seed)

    def codes(*shape):
        return torch.randint(-128, 128, shape, generator=g, device=DEV).to(torch.int8)

    R, E = sum(counts), len(counts)
    xs = torch.exp2(torch.randint(-12, -8, (R, 1), generator=g, device=DEV).float())
    ws = torch.exp2(torch.randint(-6, -2, (E, N), generator=g, device=DEV).float())
    offset = torch.tensor([0] + counts, device=DEV).cumsum(0)
    return codes(R, K), xs, codes(E, N, K), ws, offset


def exact(x, xs, w, ws, offset):
    parts = []
    for e, (lo, hi) in ref.segments(offset):
        sums = x[lo:hi].double() @ w[e].double().t()
        assert sums.numel() == 0 or sums.abs().max() < 2 ** 24
        parts.append(sums * xs[lo:hi].double() * ws[e].double())
    return torch.cat(parts)


SHAPES = [([rows], K, N) for rows in (33, 64, 65, 128, 161, 192, 193, 500, 700)
          for K, N in ((2064, 4096), (144, 264), (16, 8))]
SHAPES += [([rows] * 10, 1456, 1000) for rows in (1, 16, 33, 63, 97, 150, 177, 200)]
SHAPES += [([rows] * 24, 272, 2048) for rows in (1, 40, 66, 80, 96, 112, 129, 144, 161, 192, 230)]
SHAPES += [([rows], 528, 4096) for rows in (1000, 1536, 2047, 4100, 9000)]
SHAPES += [([(7 * e) % 61 for e in range(200)], 1040, 520)]


@pytest.mark.parametrize("counts,K,N", SHAPES,
                         ids=[f"{len(c)}x{max(c)}-{k}-{n}" for c, k, n in SHAPES])
def test_sums_are_exact(counts, K, N):
    for seed in range(3):
        x, xs, w, ws, offset = operands(counts, K, N, seed)
        want = exact(x, xs, w, ws, offset)
        for dtype in (BF, HF):
            for _ in range(2):
                out = torch.empty(x.shape[0], N, dtype=dtype, device=DEV)
                mp.moe_expert_linear_quant(x, xs, w, ws, offset, out)
                assert torch.equal(out, want.to(dtype))


@pytest.mark.parametrize("counts,K,F", [([90] * 24, 1040, 520), ([161] * 24, 272, 1024),
                                        ([4000], 400, 2048), ([200], 2064, 512)])
def test_gated(counts, K, F):
    x, xs, w, ws, offset = operands(counts, K, 2 * F, 1)
    out = torch.empty(x.shape[0], F, dtype=BF, device=DEV)
    mp.moe_expert_gated_quant(x, xs, w, ws, offset, out, activation="none")
    z = exact(x, xs, w, ws, offset)
    # (a product of two 24-bit numbers, rounded to fp32 and then to bf16)
    ref.check(out, ref.Val(z[:, :F] * z[:, F:], 2.0 ** -24 * (z[:, :F] * z[:, F:]).abs()), BF, "out")


@pytest.mark.parametrize("form,K,N", [("linear", 1008, 2048), ("gated", 1008, 2080)])
def test_a_wait_that_runs_out_is_flagged(monkeypatch, form, K, N):
    dlib = b.debug_lib()
    hook = dlib.moe_debug_set_expert_wait
    hook.restype, hook.argtypes = ctypes.c_int, [ctypes.c_int, ctypes.c_ulonglong]
    monkeypatch.setattr(b, "_lib", dlib)
    x, xs, w, ws, offset = operands([9] * 40, K, N, 2)
    status = torch.zeros(mp.moe_permute_workspace_size(1, 1, 1), dtype=torch.uint8, device=DEV)
    mp.moe_permute_workspace_init(status)
    out = torch.empty(x.shape[0], N // (2 if form == "gated" else 1), dtype=BF, device=DEV)
    fn = mp.moe_expert_gated_quant if form == "gated" else mp.moe_expert_linear_quant

    def call():
        fn(x, xs, w, ws, offset, out, workspace=status)
        return out

    want = call().clone()
    assert mp.moe_read_status(status) == 0
    try:
        assert hook(1, 20_000_000) == b.MOE_OK
        t0 = time.perf_counter()
        call()
        torch.cuda.synchronize()
        assert time.perf_counter() - t0 < 10.0
        assert mp.moe_read_status(status) == b.MOE_FLAG_BARRIER_TIMEOUT
    finally:
        torch.cuda.synchronize()
        assert hook(0, 2_000_000_000) == b.MOE_OK
    mp.moe_clear_status(status)
    assert torch.equal(call(), want)
    assert mp.moe_read_status(status) == 0


@pytest.mark.parametrize("rows", [3, 8, 200, 3000], ids=["streamed", "streamed8", "tiles", "tiles2"])
@pytest.mark.parametrize("K,N", [(4096, 512), (14336, 264)])
def test_sums_that_pass_24_bits_and_cancel(rows, K, N):
    """Few rows are added in whole numbers: exact.  More are added in fp32, whose roundings
    beyond 2^24 stay within the bound of the sums' size, whatever is left of them."""
    g = torch.Generator(DEV).manual_seed(K + rows)
    half = torch.randint(100, 128, (rows, K // 2), generator=g, device=DEV)
    x = torch.cat([half, -half.flip(1)], 1)
    x[:, ::97] += torch.randint(-9, 1, (rows, len(range(0, K, 97))), generator=g, device=DEV)
    w = torch.randint(100, 128, (1, N, K // 2), generator=g, device=DEV)
    w = torch.cat([w, w.flip(2)], 2).to(torch.int8)
    x = x.clamp(-128, 127).to(torch.int8)
    assert (x[:, :K // 2].double() @ w[0, :, :K // 2].double().t()).min() > 2 ** 24
    xs, ws = torch.full((rows, 1), 2.0 ** -6, device=DEV), torch.full((1, N), 2.0 ** -6, device=DEV)
    offset = torch.tensor([0, rows], device=DEV)
    out = torch.empty(rows, N, dtype=BF, device=DEV)
    mp.moe_expert_linear_quant(x, xs, w, ws, offset, out)
    sums = x.double() @ w[0].double().t() * 2.0 ** -12
    if rows <= 8:
        assert torch.equal(out, sums.to(BF))
    else:
        ref.check(out, qref.product(x, xs, w[0], ws[0], 1), BF, "out")
