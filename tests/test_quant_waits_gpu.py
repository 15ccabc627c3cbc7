"""The bounded waits inside the products of 8-bit rows, through the debug build,
whose limit can be set: contractions that take many times the limit are computed
all the same, and waits for slices that no block loads run out, raise the flag and
leave the context usable.  Nothing here faults, traps or loops without bound.
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
BF = torch.bfloat16
E4M3, INT8 = torch.float8_e4m3fn, torch.int8
FORMS = pytest.mark.parametrize("code", [E4M3, INT8], ids=["fp8", "int8"])
PRODUCTION_NS = 2_000_000_000
SHORT_NS = 2_000_000


@pytest.fixture
def debug_library(monkeypatch):
    dlib = b.debug_lib()
    hook = dlib.moe_debug_set_expert_wait  # csrc_experts/debug_hooks.h
    hook.restype, hook.argtypes = ctypes.c_int, [ctypes.c_int, ctypes.c_ulonglong]
    monkeypatch.setattr(b, "_lib", dlib)
    yield dlib
    torch.cuda.synchronize()
    assert dlib.moe_debug_set_expert_wait(0, PRODUCTION_NS) == b.MOE_OK


def operands(code, counts, K, N, parts, seed):
    g = torch.Generator(DEV).manual_seed(seed)
    R, E = sum(counts), len(counts)
    offset = torch.tensor([0] + counts, device=DEV).cumsum(0)

    def codes(*shape):
        return (torch.randn(*shape, generator=g, device=DEV) * 30).clamp(-120, 120).to(code)

    shapes = qref.scale_shapes(code, R, E, N, K, parts)
    xs, ws = (torch.rand(*s, generator=g, device=DEV) / K ** 0.5 for s in shapes)
    status = torch.zeros(mp.moe_permute_workspace_size(1, 1, 1), dtype=torch.uint8, device=DEV)
    mp.moe_permute_workspace_init(status)
    return codes(R, K), xs, codes(E, N, K), ws, offset, status


@pytest.mark.parametrize("R,limit", [(40, SHORT_NS), (8, SHORT_NS // 4)], ids=["tiles", "streamed"])
def test_fp8_contraction_longer_than_the_limit(debug_library, R, limit):
    """int8's are at most MOE_INT8_MAX_IN long, which no limit of this size reaches.  The
    rows are zero but for a thousand columns, so that the sums' bound counts few groups."""
    K, N = 1 << 22, 8
    _, _, _, _, _, status = operands(E4M3, [1], 16, 8, 1, 1)
    g = torch.Generator(DEV).manual_seed(2)
    at = torch.randint(0, K, (1000,), generator=g, device=DEV)
    at[0] = K - 1
    at = at.unique()
    x = torch.zeros(R, K, dtype=torch.int8, device=DEV)
    x[:, at] = torch.randn(R, at.numel(), generator=g, device=DEV).to(E4M3).view(torch.int8)
    x = x.view(E4M3)
    w = torch.randint(0, 100, (1, N, K), generator=g, device=DEV, dtype=torch.int8).view(E4M3)
    xs, ws = torch.ones(R, K // 128, device=DEV), torch.ones(1, 1, K // 128, device=DEV)
    offset, out = torch.tensor([0, R], device=DEV), torch.empty(R, N, dtype=BF, device=DEV)
    assert debug_library.moe_debug_set_expert_wait(0, limit) == b.MOE_OK

    def call():
        mp.moe_expert_linear_quant(x, xs, w, ws, offset, out, workspace=status)

    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    call()
    start.record()
    call()
    end.record()
    end.synchronize()
    assert mp.moe_read_status(status) == 0, "a wait gave up although the work went on"
    assert start.elapsed_time(end) > 1.5 * limit / 1e6, "too short to show anything"
    a, c = x.view(torch.int8)[:, at].view(E4M3).double(), w.view(torch.int8)[0][:, at].view(E4M3)
    want, mag = a @ c.double().t(), a.abs() @ c.double().abs().t()
    # at most a thousand groups have terms, and each is added once
    ref.check(out, ref.Val(want, (128 + 3 * at.numel()) * 2.0 ** -23 * mag), BF, "out")


@FORMS
@pytest.mark.parametrize("form,counts,K,N", [
    ("gated", [300, 0, 17], 1008, 272), ("linear", [300, 0, 17], 1008, 264),
    ("linear", [100], 2048, 512),  # a tile's contraction shared
    ("gated", [3, 0, 5], 8192, 64), ("linear", [3, 0, 5], 8192, 64),  # streamed
])
def test_a_wait_that_runs_out_is_flagged(debug_library, form, counts, K, N, code):
    parts = 2 if form == "gated" else 1
    x, xs, w, ws, offset, status = operands(code, counts, K, N, parts, 5)
    out = torch.empty(x.shape[0], N // parts, dtype=BF, device=DEV)
    fn = mp.moe_expert_gated_quant if form == "gated" else mp.moe_expert_linear_quant

    def call():
        fn(x, xs, w, ws, offset, out, workspace=status)
        return out

    want = call().clone()
    assert mp.moe_read_status(status) == 0
    assert debug_library.moe_debug_set_expert_wait(1, 20_000_000) == b.MOE_OK
    t0 = time.perf_counter()
    call()
    torch.cuda.synchronize()
    assert time.perf_counter() - t0 < 10.0  # the limit, and up to 2 s for what is in flight
    assert mp.moe_read_status(status) == b.MOE_FLAG_BARRIER_TIMEOUT
    assert debug_library.moe_debug_set_expert_wait(0, PRODUCTION_NS) == b.MOE_OK
    mp.moe_clear_status(status)
    got = call()
    assert mp.moe_read_status(status) == 0
    assert torch.equal(got, want)
