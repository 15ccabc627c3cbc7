"""What the 8-bit expert operators refuse, found on the host before any device
work: through the C ABI with pointers that are never dereferenced, and through
the Python functions with CPU tensors."""
import os
import shutil
import subprocess

import pytest
import torch

import moe_token_permute_gb300 as mp
from moe_token_permute_gb300 import _binding as b
from moe_token_permute_gb300 import build as cuda_build

BF = torch.bfloat16
E4M3, INT8 = torch.float8_e4m3fn, torch.int8
INCLUDE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")


@pytest.fixture(scope="module")
def lib():
    cuda_build.build()
    return b.lib()


def call(lib, name, args, over):
    bad = set(over) - set(args)
    assert not bad, bad
    return getattr(lib, name)(*{**args, **over}.values())


ROWS = dict(x=0x1000, dt=b.MOE_DTYPE_BF16, off=0x2000, R=4, H=32, E=2, code=b.MOE_DTYPE_INT8,
            codes=0x3000, s=0x4000, ws=None, stream=None)
GATED = dict(x=0x1000, xs=0x2000, w=0x3000, s=0x4000, code=b.MOE_DTYPE_FP8_E4M3,
             dt=b.MOE_DTYPE_BF16, off=0x5000, R=4, H=32, F=8, E=2, act=b.MOE_ACT_SILU, out=0x6000,
             ws=None, stream=None)
LINEAR = dict(x=0x1000, xs=0x2000, w=0x3000, s=0x4000, code=b.MOE_DTYPE_INT8,
              dt=b.MOE_DTYPE_FP16, off=0x5000, R=4, K=32, N=8, E=2, bias=None,
              act=b.MOE_ACT_NONE, res=None, out=0x6000, ws=None, stream=None)

TYPES = [dict(dt=b.MOE_DTYPE_FP32), dict(dt=b.MOE_DTYPE_INT8), dict(dt=77),
         dict(code=b.MOE_DTYPE_BF16), dict(code=b.MOE_DTYPE_FP8_E5M2), dict(code=6),
         dict(R=-1), dict(R=2 ** 31), dict(R=2 ** 31 - 1023), dict(x=None), dict(x=0x1008),
         dict(s=None), dict(s=0x4002), dict(ws=0x10), dict(off=0x5004), dict(E=0),
         dict(E=b.MOE_MAX_LOCAL_EXPERTS + 1)]
PRODUCTS = TYPES + [dict(act=4), dict(act=-1), dict(off=None), dict(w=None), dict(w=0x3008),
                    dict(xs=None), dict(xs=0x2001), dict(out=None), dict(out=0x6008)]


@pytest.mark.parametrize("over", TYPES + [
    dict(H=0), dict(H=8), dict(H=24), dict(H=-16), dict(H=2 ** 33), dict(codes=None),
    dict(codes=0x3008)], ids=str)
def test_quant_rows_refuses(lib, over):
    assert call(lib, "moe_quant_rows", ROWS, over) == b.MOE_ERR_INVALID_ARG


@pytest.mark.parametrize("over", PRODUCTS + [
    dict(H=0), dict(H=8), dict(H=24), dict(H=2 ** 33), dict(F=0), dict(F=4), dict(F=12),
    dict(F=-8), dict(F=2 ** 40)], ids=str)
def test_gated_refuses(lib, over):
    assert call(lib, "moe_expert_gated_quant", GATED, over) == b.MOE_ERR_INVALID_ARG


@pytest.mark.parametrize("over", PRODUCTS + [
    dict(K=0), dict(K=8), dict(K=40), dict(K=b.MOE_INT8_MAX_IN + 16), dict(N=0), dict(N=4),
    dict(N=2 ** 33), dict(bias=0x7008), dict(res=0x7008)], ids=str)
def test_linear_refuses(lib, over):
    assert call(lib, "moe_expert_linear_quant", LINEAR, over) == b.MOE_ERR_INVALID_ARG


@pytest.mark.parametrize("name,args", [("moe_quant_rows", ROWS), ("moe_expert_gated_quant", GATED),
                                       ("moe_expert_linear_quant", LINEAR)])
def test_valid_calls_get_past_the_checks(lib, name, args):
    if not torch.cuda.is_available():  # elsewhere they would be enqueued
        assert call(lib, name, args, {}) == b.MOE_ERR_UNSUPPORTED_DEVICE
        assert call(lib, name, args, dict(R=2 ** 31 - 1024)) == b.MOE_ERR_UNSUPPORTED_DEVICE
    none = {k: None for k in ("x", "xs", "w", "s", "off", "out", "codes") if k in args}
    assert call(lib, name, args, dict(none, R=0)) == b.MOE_OK


def test_int8_rows_can_be_permuted(lib):
    """MOE_DTYPE_INT8 is a type of moe_permute's rows: not refused by the checks."""
    if not torch.cuda.is_available():
        args = (0x1000, b.MOE_DTYPE_INT8, 0x2000, 1, 0x3000, b.MOE_INDEX_INT32, None, 4, 16, 2, 4,
                4, 0x4000, 0x5000, 0x6000, 0x7000, 0x8000, 0x100000, 1 << 30, None)
        assert lib.moe_permute(*args) == b.MOE_ERR_UNSUPPORTED_DEVICE


def test_constants(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    src, exe = tmp_path / "c.c", tmp_path / "c"
    src.write_text('#include <stdio.h>\n#include "moe_quant.h"\nint main(void) {\n'
                   '    printf("%d %d\\n", MOE_DTYPE_INT8, MOE_INT8_MAX_IN);\n    return 0;\n}\n')
    subprocess.run([cc, "-std=c11", "-Wall", "-Werror", "-I", INCLUDE, "-o", str(exe), str(src)],
                   check=True)
    out = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout
    assert out.split() == [str(b.MOE_DTYPE_INT8), str(b.MOE_INT8_MAX_IN)]
    # any sum of that many products of two codes fits 32 bits
    assert 128 * 128 * b.MOE_INT8_MAX_IN < 2 ** 31


def refused(match, fn, *args, **kw):
    with pytest.raises(ValueError, match=match):
        fn(*args, **kw)


def test_binding_refuses_quant_rows():
    x = torch.zeros(4, 272, dtype=BF)
    c8, ci = torch.zeros(4, 272, dtype=E4M3), torch.zeros(4, 272, dtype=INT8)
    s8, si = torch.zeros(4, 3), torch.zeros(4, 1)
    f = mp.moe_quant_rows
    refused("bfloat16 or float16", f, x.float(), c8, s8)
    refused("bfloat16 or float16", f, x[0], c8, s8)
    refused("float8_e4m3fn or int8", f, x, c8.view(torch.uint8), s8)
    refused("codes must hold", f, x, c8[:3], s8)
    refused("codes must hold", f, x, ci[:, :256], si)
    refused("scales must hold", f, x, c8, si)
    refused("scales must hold", f, x, ci, s8)
    refused("scales is", f, x, ci, si.double())
    off = torch.zeros(3, dtype=torch.int64)
    refused("must be int64", f, x, ci, si, expert_first_token_offset=off.int())
    refused("holds 1 elements", f, x, ci, si, expert_first_token_offset=off[:1])
    refused("CUDA tensor", f, x, ci, si, expert_first_token_offset=off)


@pytest.mark.parametrize("code", [E4M3, INT8], ids=["fp8", "int8"])
def test_binding_refuses_products(code):
    R, K, N, E = 4, 272, 400, 2
    x, w = torch.zeros(R, K, dtype=code), torch.zeros(E, N, K, dtype=code)
    xs = torch.zeros(R, 1 if code == INT8 else 3)
    gs = torch.zeros(E, N) if code == INT8 else torch.zeros(E, 4, 3)
    ls = torch.zeros(E, N) if code == INT8 else torch.zeros(E, 4, 3)
    off, h = torch.zeros(E + 1, dtype=torch.int64), torch.zeros(R, N // 2, dtype=BF)
    y, bias = torch.zeros(R, N, dtype=BF), torch.zeros(E, N, dtype=BF)
    for f, s, out in ((mp.moe_expert_gated_quant, gs, h), (mp.moe_expert_linear_quant, ls, y)):
        refused("float8_e4m3fn or int8", f, x, xs, w.view(torch.uint8), s, off, out)
        refused("the codes is", f, x.view(torch.uint8), xs, w, s, off, out)
        refused("the codes must hold", f, x[:, :256], xs, w, s, off, out)
        refused(r"must be \[R, in\]", f, x[0], xs, w, s, off, out)
        refused("the rows' scales must hold", f, x, xs[:3], w, s, off, out)
        refused("weight_scales must hold", f, x, xs, w, s[:1], off, out)
        refused("weight_scales is", f, x, xs, w, s.half(), off, out)
        refused("holds 2 elements", f, x, xs, w, s, off[:2], out)
        refused("must be int64", f, x, xs, w, s, off.int(), out)
        refused("bfloat16 or float16", f, x, xs, w, s, off, out.float())
        refused("out must hold", f, x, xs, w, s, off, out[:3])
        refused("activation must be", f, x, xs, w, s, off, out, activation="tanh")
        refused(r"\[experts, out, in\]", f, x, xs, w[0], s, off, out)
        refused("CUDA tensor", f, x, xs, w, s, off, out)
    refused("as many up rows", mp.moe_expert_gated_quant, x, xs, w[:, :399], gs, off, h)
    if code == E4M3:  # gate and up rows count their blocks apart: 2 x 2, not 4 of 400
        refused("weight_scales must hold", mp.moe_expert_gated_quant, x, xs, w[:, :272],
                torch.zeros(E, 3, 3), off, h)
    f = mp.moe_expert_linear_quant
    refused("bias must hold", f, x, xs, w, ls, off, y, bias=bias[:1])
    refused("bias is", f, x, xs, w, ls, off, y, bias=bias.half())
    refused("residual must hold", f, x, xs, w, ls, off, y, residual=h)
    refused("residual is", f, x, xs, w, ls, off, y, residual=y.half())


def test_tensors_of_another_device_are_refused(monkeypatch):
    class Elsewhere:
        device = "cuda:1"

        def get_device(self):
            return 1

    monkeypatch.setattr(mp, "_raw_device", lambda: 0)
    with pytest.raises(ValueError, match="current device"):
        mp._pointers(None, Elsewhere())
