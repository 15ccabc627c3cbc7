"""int8 rows with one scale each through every permute entry point: codes and scales
are the tokens' own, bit for bit, against the oracle's order.  (Named to run behind the
other tests: moe_permute_noalloc keeps its scratch.)
"""
import numpy as np
import pytest
import torch

import moe_token_permute_gb300 as mp
import oracle
from gpu_util import bytes_of
from moe_token_permute_gb300 import _binding as b
from moe_token_permute_gb300.workloads import make_inputs

pytestmark = pytest.mark.gpu
DEV = "cuda"


def inputs(name, T, H):
    """The workload's routing, with int8 rows of H codes."""
    inp = make_inputs(name, T, seed=T, device=DEV, with_rows=False)
    g = torch.Generator(DEV).manual_seed(T + H)
    codes = torch.randint(-128, 128, (T, H), generator=g, device=DEV).to(torch.int8)
    scales = torch.rand(T, 1, generator=g, device=DEV)
    scales[T // 2] = float("nan")
    return inp, codes, scales


def host(t):
    return None if t is None else t.cpu().numpy()


CASES = [("mixtral", 300, 4096), ("qwen3", 33, 272), ("dsv2lite", 700, 1008), ("dsv3", 128, 7168),
         ("tiny", 1, 16)]


@pytest.mark.parametrize("entry", ["moe_permute", "moe_permute_noalloc"])
@pytest.mark.parametrize("name,T,H", CASES)
def test_permute(name, T, H, entry):
    inp, codes, scales = inputs(name, T, H)
    wl = inp["wl"]
    R = T * wl.K
    off = torch.zeros(wl.e_local + 1, dtype=torch.int64, device=DEV)
    pidx, inv = (torch.zeros(R, dtype=torch.int32, device=DEV) for _ in range(2))
    out = torch.zeros(R, H, dtype=torch.int8, device=DEV)
    out_scales = torch.zeros(R, 1, device=DEV)
    if entry == "moe_permute":
        ws = torch.empty(mp.moe_permute_workspace_size(T, wl.K, wl.E), dtype=torch.uint8, device=DEV)
        mp.moe_permute_workspace_init(ws)
        mp.moe_permute(codes, inp["topk_ids"], off, pidx, inv, ws, num_experts=wl.E,
                       num_local_experts=wl.e_local, expert_map=inp["expert_map"],
                       hidden_scales=scales, permuted_hidden_states=out, permuted_scales=out_scales)
    else:
        expert_map = inp["expert_map"]
        rc = b.lib().moe_permute_noalloc(
            codes.data_ptr(), b.MOE_DTYPE_INT8, scales.data_ptr(), 1, inp["topk_ids"].data_ptr(),
            b.MOE_INDEX_INT32, None if expert_map is None else expert_map.data_ptr(), T, H, wl.K,
            wl.E, wl.e_local, out.data_ptr(), out_scales.data_ptr(), off.data_ptr(),
            pidx.data_ptr(), inv.data_ptr(), torch.cuda.current_stream().cuda_stream)
        assert rc == b.MOE_OK
    want = oracle.permute(host(inp["topk_ids"]), wl.E, expert_map=host(inp["expert_map"]),
                          E_local=wl.e_local, hidden=bytes_of(codes), scales=host(scales))
    n = want["n_valid"]
    np.testing.assert_array_equal(host(off), want["offsets"])
    np.testing.assert_array_equal(host(inv), want["inv_permuted_idx"])
    np.testing.assert_array_equal(bytes_of(out)[:n], want["permuted_hidden"][:n])
    np.testing.assert_array_equal(host(out_scales)[:n].view(np.uint32),
                                  want["permuted_scales"][:n].view(np.uint32))


@pytest.mark.parametrize("name,T,H", CASES)
def test_batched(name, T, H):
    inp, codes, scales = inputs(name, T, H)
    wl = inp["wl"]
    M = max(1, T // 4)  # the busiest experts overflow
    counts = torch.zeros(wl.e_local, dtype=torch.int32, device=DEV)
    inv = torch.zeros(T * wl.K, dtype=torch.int32, device=DEV)
    ws = torch.empty(mp.moe_permute_workspace_size(T, wl.K, wl.E), dtype=torch.uint8, device=DEV)
    mp.moe_permute_workspace_init(ws)
    out = torch.zeros(wl.e_local * M, H, dtype=torch.int8, device=DEV)
    out_scales = torch.zeros(wl.e_local * M, 1, device=DEV)
    mp.moe_permute_batched(codes, inp["topk_ids"], counts, inv, ws, num_experts=wl.E,
                           num_local_experts=wl.e_local, max_rows_per_expert=M,
                           expert_map=inp["expert_map"], hidden_scales=scales,
                           batched_hidden_states=out, batched_scales=out_scales)
    want = oracle.permute_batched(host(inp["topk_ids"]), wl.E, M, expert_map=host(inp["expert_map"]),
                                  E_local=wl.e_local, hidden=bytes_of(codes), scales=host(scales))
    np.testing.assert_array_equal(host(counts), want["expert_num_tokens"])
    np.testing.assert_array_equal(host(inv), want["inv_permuted_idx"])
    assert mp.moe_read_status(ws) == want["flags"]
    filled = np.concatenate([e * M + np.arange(c) for e, c in
                             enumerate(want["expert_num_tokens"])]).astype(np.int64)
    np.testing.assert_array_equal(bytes_of(out)[filled], want["batched_hidden"][filled])
    np.testing.assert_array_equal(host(out_scales)[filled].view(np.uint32),
                                  want["batched_scales"][filled].view(np.uint32))
