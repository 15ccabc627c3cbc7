"""The bounded waits inside the expert products, through the debug build, whose
limit can be set: contractions that take many times the limit are computed all
the same, because their waits go by progress; waits for something that never
comes run out, raise the flag and leave the context usable.  Nothing here
faults, traps or loops without bound: a withheld slice is one that no block
loads, and every copy that is issued arrives.

The long contractions are zero but for a thousand places, so that their sums'
bound counts a thousand terms.
"""
import ctypes
import time

import pytest
import torch

import expert_ref as ref
import moe_token_permute_gb300 as mp
from moe_token_permute_gb300 import _binding as b

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16
PRODUCTION_NS = 2_000_000_000
SHORT_NS = 2_000_000
LONG_MS = 3 * SHORT_NS / 1e6  # a wait checks its limit up to 1.3 ms late


@pytest.fixture
def debug_library(monkeypatch):
    dlib = b.debug_lib()
    hook = dlib.moe_debug_set_expert_wait  # csrc_experts/debug_hooks.h
    hook.restype, hook.argtypes = ctypes.c_int, [ctypes.c_int, ctypes.c_ulonglong]
    monkeypatch.setattr(b, "_lib", dlib)
    yield dlib
    torch.cuda.synchronize()
    assert dlib.moe_debug_set_expert_wait(0, PRODUCTION_NS) == b.MOE_OK


def workspace():
    ws = torch.zeros(mp.moe_permute_workspace_size(1, 1, 1), dtype=torch.uint8, device=DEV)
    mp.moe_permute_workspace_init(ws)
    return ws


def sparse(g, rows, cols, places, along):
    """Zeros with random values in `places` rows or columns, the last among them."""
    t = torch.zeros(rows, cols, dtype=BF, device=DEV)
    at = torch.randint(0, (rows, cols)[along], (places,), generator=g, device=DEV)
    at[0] = (rows, cols)[along] - 1
    at = at.unique()
    if along == 0:
        t[at] = torch.randn(at.numel(), cols, generator=g, device=DEV).to(BF)
    else:
        t[:, at] = torch.randn(rows, at.numel(), generator=g, device=DEV).to(BF)
    return t, at


def timed(call, ws, expect_ms=LONG_MS):
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    call()  # warm
    start.record()
    call()
    end.record()
    end.synchronize()
    assert mp.moe_read_status(ws) == 0, "a wait gave up although the work went on"
    assert start.elapsed_time(end) > expect_ms, "too short to show anything"


def test_d_weight_longer_than_the_limit(debug_library):
    g = torch.Generator(DEV).manual_seed(1)
    R = 12_000_037
    dz, at = sparse(g, R, 8, 1000, 0)
    x = torch.randn(R, 8, generator=g, device=DEV, dtype=BF)
    offset = torch.tensor([0, R], device=DEV)
    dw, ws = torch.empty(1, 8, 8, dtype=BF, device=DEV), workspace()
    assert debug_library.moe_debug_set_expert_wait(0, SHORT_NS) == b.MOE_OK
    timed(lambda: mp.moe_expert_linear_backward(dz, x, None, offset, d_weight=dw, workspace=ws), ws)
    want = ref.product(ref.exact(dz[at].t()), ref.exact(x[at].t()))
    ref.check(dw[0], want, BF, "d_weight")


def test_tail_of_a_tile_behind_a_long_one(debug_library):
    """More tiles than pairs of SMs: the warp that clears the second tile's tail
    waits for it all through the first."""
    g = torch.Generator(DEV).manual_seed(2)
    pairs = torch.cuda.get_device_properties(0).multi_processor_count // 2
    counts = [2_000_003] * pairs + [100, 37]
    offset = torch.tensor([0] + counts, device=DEV).cumsum(0)
    R, E = sum(counts), len(counts)
    dz, at = sparse(g, R, 8, 1000, 0)
    dz[-137:] = torch.randn(137, 8, generator=g, device=DEV).to(BF)
    x = torch.randn(R, 8, generator=g, device=DEV, dtype=BF)
    dw, ws = torch.empty(E, 8, 8, dtype=BF, device=DEV), workspace()
    assert debug_library.moe_debug_set_expert_wait(0, SHORT_NS) == b.MOE_OK
    timed(lambda: mp.moe_expert_linear_backward(dz, x, None, offset, d_weight=dw, workspace=ws), ws)
    rows = torch.cat([at[at < R - 137], torch.arange(R - 137, R, device=DEV)])
    for e in (0, E // 2, E - 2, E - 1):
        lo, hi = offset[e].item(), offset[e + 1].item()
        r = rows[(rows >= lo) & (rows < hi)]
        ref.check(dw[e], ref.product(ref.exact(dz[r].t()), ref.exact(x[r].t())), BF, f"expert {e}")


def test_shared_tiles_longer_than_the_limit(debug_library):
    """Forward and d_rows of one expert, each tile shared by two pairs."""
    g = torch.Generator(DEV).manual_seed(3)
    R, K, N = 40, 1 << 22, 8
    x, at = sparse(g, R, K, 1000, 1)
    w = torch.randn(1, N, K, generator=g, device=DEV, dtype=BF)
    offset, ws = torch.tensor([0, R], device=DEV), workspace()
    out = torch.empty(R, N, dtype=BF, device=DEV)
    assert debug_library.moe_debug_set_expert_wait(0, SHORT_NS) == b.MOE_OK
    timed(lambda: mp.moe_expert_linear(x, w, offset, out, workspace=ws), ws)
    want = ref.product(ref.exact(x[:, at]), ref.exact(w[0][:, at]))
    ref.check(out, want, BF, "out")
    w = w.view(1, K, N)
    dx = torch.empty(R, N, dtype=BF, device=DEV)
    timed(lambda: mp.moe_expert_linear_backward(x, None, w, offset, d_rows=dx, workspace=ws), ws)
    ref.check(dx, ref.product(ref.exact(x[:, at]), ref.exact(w[0][at].t())), BF, "d_rows")


def test_streamed_task_longer_than_the_limit(debug_library):
    g = torch.Generator(DEV).manual_seed(4)
    R, K, N = 8, 1 << 25, 8
    x, at = sparse(g, R, K, 1000, 1)
    w = torch.randn(1, N, K, generator=g, device=DEV, dtype=BF)
    offset, ws = torch.tensor([0, R], device=DEV), workspace()
    out = torch.empty(R, N, dtype=BF, device=DEV)
    assert debug_library.moe_debug_set_expert_wait(0, SHORT_NS) == b.MOE_OK
    timed(lambda: mp.moe_expert_linear(x, w, offset, out, workspace=ws), ws)
    ref.check(out, ref.product(ref.exact(x[:, at]), ref.exact(w[0][:, at])), BF, "out")


@pytest.mark.parametrize("form,counts,K,N", [
    ("gated", [300, 0, 17], 1000, 272), ("linear", [300, 0, 17], 1000, 264),
    ("linear", [100], 1024, 512),  # a tile shared by two pairs
    ("gated", [3, 0, 5], 8192, 64), ("linear", [3, 0, 5], 8192, 64),  # streamed
    ("d_rows", [300, 0, 17], 264, 1000), ("d_weight", [640, 0, 384], 264, 264),
    ("d_weight", [700, 0, 321], 264, 264),  # with tails
])
def test_a_wait_that_runs_out_is_flagged(debug_library, form, counts, K, N):
    g = torch.Generator(DEV).manual_seed(5)

    def normal(*shape):
        return (torch.randn(*shape, generator=g, device=DEV) * 0.25).to(BF)

    R, E = sum(counts), len(counts)
    offset, ws = torch.tensor([0] + counts, device=DEV).cumsum(0), workspace()
    x, w = normal(R, K), normal(E, N, K)
    out = torch.empty(R, N // 2 if form == "gated" else N, dtype=BF, device=DEV)
    d, dx, dw = normal(R, N), torch.empty_like(x), torch.empty_like(w)

    def call():
        if form == "gated":
            mp.moe_expert_gated(x, w, offset, out, workspace=ws)
        elif form == "linear":
            mp.moe_expert_linear(x, w, offset, out, workspace=ws)
        elif form == "d_rows":
            mp.moe_expert_linear_backward(d, None, w, offset, d_rows=dx, workspace=ws)
        else:
            mp.moe_expert_linear_backward(d, x, None, offset, d_weight=dw, workspace=ws)
        return {"d_rows": dx, "d_weight": dw}.get(form, out)

    want = call().clone()
    assert mp.moe_read_status(ws) == 0
    assert debug_library.moe_debug_set_expert_wait(2, 20_000_000) == b.MOE_OK
    t0 = time.perf_counter()
    call()
    torch.cuda.synchronize()
    assert time.perf_counter() - t0 < 10.0  # the limit, and up to 2 s for what is in flight
    assert mp.moe_read_status(ws) == b.MOE_FLAG_BARRIER_TIMEOUT
    assert debug_library.moe_debug_set_expert_wait(0, PRODUCTION_NS) == b.MOE_OK
    mp.moe_clear_status(ws)
    got = call()
    assert mp.moe_read_status(ws) == 0
    assert torch.equal(got, want)
