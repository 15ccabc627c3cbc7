"""moe_quant_rows against its definition, bit for bit: codes and scales of both
forms, at the widths and contents where they can go wrong.
"""
import pytest
import torch

import moe_token_permute_gb300 as mp
import quant_ref as qref
from moe_token_permute_gb300 import _binding as b

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, HF = torch.bfloat16, torch.float16
E4M3, INT8 = torch.float8_e4m3fn, torch.int8
FORMS = pytest.mark.parametrize("code", [E4M3, INT8], ids=["fp8", "int8"])
TYPES = pytest.mark.parametrize("dtype", [BF, HF], ids=["bf16", "fp16"])
WIDTHS = [16, 32, 112, 128, 144, 496, 512, 528, 1008, 2048, 4096, 4112, 7168, 8208, 14336, 16400,
          33008]


def blank(R, H, code):
    codes = torch.full((R, H), 85, dtype=torch.int8, device=DEV).view(code)
    columns = 1 if code == INT8 else qref.groups(H)
    return codes, torch.full((R, columns), -77.0, device=DEV)


def same(codes, scales, want_codes, want_scales):
    assert torch.equal(scales.view(torch.int32), want_scales.view(torch.int32)) or \
        torch.equal(scales.nan_to_num(-5.0), want_scales.nan_to_num(-5.0))
    nan = want_codes.float().isnan()
    assert torch.equal(codes.float().isnan(), nan)
    assert torch.equal(codes.view(torch.int8)[~nan], want_codes.view(torch.int8)[~nan])


@FORMS
@TYPES
@pytest.mark.parametrize("H", WIDTHS)
@pytest.mark.parametrize("R", [1, 5, 67])
def test_codes_and_scales(R, H, dtype, code):
    g = torch.Generator(DEV).manual_seed(R * H)
    x = torch.randn(R, H, generator=g, device=DEV)
    x *= torch.exp2(torch.randint(-12, 12, (R, 1), generator=g, device=DEV).float())
    x = x.clamp(-60000, 60000).to(dtype)
    x[R // 2] = 0
    codes, scales = blank(R, H, code)
    mp.moe_quant_rows(x, codes, scales)
    same(codes, scales, *qref.quantised(x, code))


@FORMS
@TYPES
@pytest.mark.parametrize("H", [272, 2048, 14336])
def test_rows_of_no_expert(H, dtype, code):
    g = torch.Generator(DEV).manual_seed(H)
    x = torch.randn(301, H, generator=g, device=DEV).to(dtype)
    for ends in ([7, 7, 130, 200], [0, 301], [0, 0], [301, 301], [5, 6]):
        offset = torch.tensor(ends, device=DEV)
        lo, hi = ends[0], ends[-1]
        codes, scales = blank(301, H, code)
        before_c, before_s = codes.clone(), scales.clone()
        mp.moe_quant_rows(x, codes, scales, expert_first_token_offset=offset)
        want = qref.quantised(x, code)
        before_c.view(torch.int8)[lo:hi] = want[0].view(torch.int8)[lo:hi]
        before_s[lo:hi] = want[1][lo:hi]
        assert torch.equal(codes.view(torch.int8), before_c.view(torch.int8))
        assert torch.equal(scales, before_s)


@FORMS
def test_malformed_offsets(code):
    """Cut to segments within the rows, whose gaps are not written, and flagged."""
    x = torch.randn(70, 272, device=DEV).to(BF)
    ws = torch.zeros(mp.moe_permute_workspace_size(1, 1, 1), dtype=torch.uint8, device=DEV)
    mp.moe_permute_workspace_init(ws)
    want = qref.quantised(x, code)
    for ends, rows in (([50, 60, 0, 10], [(50, 60), (0, 10)]), ([-3, 20, 2 ** 40], [(0, 70)]),
                       ([60, 30], [])):
        used = torch.zeros(70, dtype=torch.bool, device=DEV)
        for lo, hi in rows:
            used[lo:hi] = True
        codes, scales = blank(70, 272, code)
        before = codes.view(torch.int8).clone()
        mp.moe_clear_status(ws)
        mp.moe_quant_rows(x, codes, scales, workspace=ws,
                          expert_first_token_offset=torch.tensor(ends, device=DEV))
        assert mp.moe_read_status(ws) == b.MOE_FLAG_OFFSET_OUT_OF_RANGE
        got = codes.view(torch.int8)
        assert torch.equal(got[used], want[0].view(torch.int8)[used])
        assert torch.equal(scales[used], want[1][used])
        assert torch.equal(got[~used], before[~used]) and (scales[~used] == -77).all()


@FORMS
@TYPES
@pytest.mark.parametrize("H", [128, 1040, 16400])
def test_infinities_nan_and_the_smallest_values(H, dtype, code):
    tiny = torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps  # the smallest subnormal
    x = torch.randn(9, H, device=DEV).to(dtype)
    x[1, 5], x[2, H - 1] = float("inf"), float("-inf")
    x[3, 0], x[4, H - 1] = float("nan"), float("nan")
    x[4, 3] = float("inf")
    x[5] = 0
    x[5, 7] = tiny
    x[6] = -tiny
    x[7] = torch.finfo(dtype).max
    x[8] = -0.0
    codes, scales = blank(9, H, code)
    mp.moe_quant_rows(x, codes, scales)
    same(codes, scales, *qref.quantised(x, code))


@FORMS
@TYPES
def test_every_quotient(dtype, code):
    """Every pair of a finite positive value x and an amax >= x: the codes are those
    of fp32 divisions (signs: every second column)."""
    top = 0x7f80 if dtype == BF else 0x7c00
    bits = torch.arange(top, dtype=torch.int32, device=DEV).to(torch.int16)
    values = bits.view(dtype)
    if code == E4M3:  # 127 values and the amax make a group
        pad = -values.numel() % 127
        values = torch.cat([values, values.new_zeros(pad)]).view(-1, 127)
    for at in range(0, top, 1024):
        amax = bits[at:at + 1024].view(dtype)
        n = amax.numel()
        if code == E4M3:
            x = torch.cat([values.expand(n, *values.shape),
                           amax[:, None, None].expand(n, values.shape[0], 1)], 2).reshape(n, -1)
            x = torch.where(x.view(n, -1, 128).float() <= amax[:, None, None].float(),
                            x.view(n, -1, 128), torch.zeros_like(x.view(n, -1, 128))).view(n, -1)
        else:
            x = torch.where(values.float() <= amax[:, None].float(), values, amax[:, None])
            x = torch.nn.functional.pad(x, (0, -x.shape[1] % 16))
        x = x.contiguous()
        x[:, 1::2] = -x[:, 1::2]
        codes, scales = blank(*x.shape, code)
        mp.moe_quant_rows(x, codes, scales)
        same(codes, scales, *qref.quantised(x, code))


@FORMS
def test_beyond_32_bits(code):
    """Elements counted beyond 2^31, and beyond 2^32 bytes of rows."""
    R, H = 160_003, 14336
    x = torch.zeros(R, H, dtype=BF, device=DEV)
    x[-5:] = torch.randn(5, H, device=DEV).to(BF)
    codes, scales = blank(R, H, code)
    mp.moe_quant_rows(x, codes, scales)
    want = qref.quantised(x[-6:], code)
    same(codes[-6:].contiguous(), scales[-6:].contiguous(), *want)
    assert (codes[:-5].view(torch.int8) == 0).all() and (scales[:-5] == 1).all()


@FORMS
def test_unaligned_to_32_bytes(code):
    """Bases that are aligned to 16 bytes and no more."""
    H, R = 1008, 33
    x = torch.randn(R * H + 8, device=DEV).to(BF)[8:].view(R, H)
    raw = torch.zeros(R * H + 16, dtype=torch.int8, device=DEV)
    codes = raw[16:].view(R, H).view(code)
    columns = 1 if code == INT8 else qref.groups(H)
    scales = torch.zeros(R * columns + 1, device=DEV)[1:].view(R, columns)
    assert x.data_ptr() % 32 == 16
    mp.moe_quant_rows(x, codes, scales)
    same(codes, scales, *qref.quantised(x, code))


def test_the_permutes_rule():
    """fp8 codes are those of moe_permute_quant_fp8."""
    T, H = 37, 1024
    x = torch.randn(T, H, device=DEV).to(BF)
    ids = torch.zeros(T, 1, dtype=torch.int32, device=DEV)
    s = mp.MoEPermuteScratch(T, 1, 1, 1, torch.device(DEV), H, E4M3, scale_cols=H // 128)
    got = s.permute_quant_fp8(x, ids)
    codes, scales = blank(T, H, E4M3)
    mp.moe_quant_rows(x, codes, scales)
    assert torch.equal(got["permuted_hidden_states"].view(torch.int8), codes.view(torch.int8))
    assert torch.equal(got["permuted_scales"], scales)


def test_no_rows():
    x = torch.zeros(0, 64, dtype=BF, device=DEV)
    mp.moe_quant_rows(x, x.to(INT8), torch.zeros(0, 1, device=DEV))
