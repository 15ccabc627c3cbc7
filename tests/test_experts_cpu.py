"""What the expert operators refuse, found on the host before any device work:
through the C ABI with pointers that are never dereferenced, and through the
Python functions with CPU tensors, whose sizes are checked before their
pointers are taken.  And the 64-bit forms the GPU tests compare with, against
central differences."""
import pytest
import torch

import expert_ref as ref
import moe_token_permute_gb300 as mp
from moe_token_permute_gb300 import _binding as b
from moe_token_permute_gb300 import build as cuda_build

BF, HF = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def lib():
    cuda_build.build()
    return b.lib()


def call(lib, name, args, over):
    bad = set(over) - set(args)
    assert not bad, bad
    return getattr(lib, name)(*{**args, **over}.values())


GATED = dict(x=0x1000, w=0x2000, dt=b.MOE_DTYPE_BF16, off=0x3000, R=4, H=16, F=8, E=2,
             act=b.MOE_ACT_SILU, out=0x4000, pre=0x5000, ws=None, stream=None)
GATED_BW = dict(d=0x1000, x=0x2000, w=0x3000, dt=b.MOE_DTYPE_BF16, off=0x4000, R=4, H=16, F=8,
                E=2, act=b.MOE_ACT_SILU, pre=0x5000, dpre=0x6000, dx=0x7000, dw=0x8000, ws=None,
                stream=None)
LINEAR = dict(x=0x1000, w=0x2000, dt=b.MOE_DTYPE_BF16, off=0x3000, R=4, K=16, N=8, E=2, bias=None,
              act=b.MOE_ACT_NONE, res=None, out=0x4000, pre=None, ws=None, stream=None)
LINEAR_BW = dict(d=0x1000, x=0x2000, w=0x3000, dt=b.MOE_DTYPE_BF16, off=0x4000, R=4, K=16, N=8,
                 E=2, act=b.MOE_ACT_GELU, pre=0x5000, dpre=0x6000, dx=0x7000, dw=0x8000,
                 db=0x9000, ws=None, stream=None)
UNPERMUTE_BW = dict(d=0x1000, rows=0x2000, R=4, wts=0x3000, inv=0x4000, T=2, H=16, K=2,
                    dr=0x5000, dw=0x6000, ws=None, stream=None)

COMMON = [dict(dt=b.MOE_DTYPE_FP32), dict(dt=b.MOE_DTYPE_FP8_E4M3), dict(dt=77), dict(act=4),
          dict(act=-1), dict(R=-1), dict(R=2 ** 31), dict(E=0),
          dict(E=b.MOE_MAX_LOCAL_EXPERTS + 1), dict(off=None), dict(off=0x3004), dict(w=0x2008),
          dict(x=0x1002), dict(ws=0x10)]


@pytest.mark.parametrize("over", COMMON + [
    dict(H=0), dict(H=12), dict(H=-8), dict(F=0), dict(F=4), dict(F=12), dict(F=2 ** 40),
    dict(x=None), dict(w=None), dict(out=None), dict(out=0x4008), dict(pre=0x5008)], ids=str)
def test_gated_refuses(lib, over):
    assert call(lib, "moe_expert_gated", GATED, over) == b.MOE_ERR_INVALID_ARG


@pytest.mark.parametrize("over", COMMON + [
    dict(H=20), dict(F=2), dict(d=None), dict(d=0x1008), dict(pre=None), dict(pre=0x5004),
    dict(dpre=None), dict(dpre=0x6008), dict(dx=0x7008), dict(dw=0x8008), dict(w=None),
    dict(x=None)], ids=str)
def test_gated_backward_refuses(lib, over):
    assert call(lib, "moe_expert_gated_backward", GATED_BW, over) == b.MOE_ERR_INVALID_ARG


@pytest.mark.parametrize("over", COMMON + [
    dict(K=0), dict(K=9), dict(N=0), dict(N=36), dict(N=2 ** 33), dict(x=None), dict(w=None),
    dict(out=None), dict(out=0x4002), dict(bias=0x5008), dict(res=0x5008), dict(pre=0x5008)],
    ids=str)
def test_linear_refuses(lib, over):
    assert call(lib, "moe_expert_linear", LINEAR, over) == b.MOE_ERR_INVALID_ARG


@pytest.mark.parametrize("over", COMMON + [
    dict(K=9), dict(N=36), dict(d=None), dict(d=0x1008), dict(pre=None), dict(dpre=None),
    dict(dx=0x7008), dict(dw=0x8008), dict(db=0x9008), dict(w=None), dict(x=None),
    dict(act=b.MOE_ACT_NONE)], ids=str)  # no activation: preact and d_preact are refused
def test_linear_backward_refuses(lib, over):
    assert call(lib, "moe_expert_linear_backward", LINEAR_BW, over) == b.MOE_ERR_INVALID_ARG


@pytest.mark.parametrize("over", [
    dict(T=-1), dict(H=0), dict(K=0), dict(K=33), dict(R=-1), dict(R=2 ** 31), dict(T=2 ** 31),
    dict(d=None), dict(d=0x1001), dict(wts=None), dict(wts=0x3002), dict(inv=None),
    dict(inv=0x4002), dict(rows=None), dict(dw=None), dict(rows=None, dr=None, dw=None),
    dict(rows=0x2001), dict(dr=0x5001), dict(dw=0x6002), dict(ws=0x10)], ids=str)
def test_unpermute_backward_refuses(lib, over):
    assert call(lib, "moe_unpermute_backward", UNPERMUTE_BW, over) == b.MOE_ERR_INVALID_ARG


@pytest.mark.parametrize("name,args", [
    ("moe_expert_gated", GATED), ("moe_expert_gated_backward", GATED_BW),
    ("moe_expert_linear", LINEAR), ("moe_expert_linear_backward", LINEAR_BW)],
    ids=["gated", "gated_backward", "linear", "linear_backward"])
def test_rows_are_counted_in_32_bits(lib, name, args):
    """The kernels step past the last row by less than 1024.  (The last number that is
    allowed would be enqueued on a device.)"""
    assert call(lib, name, args, dict(R=2 ** 31 - 1023)) == b.MOE_ERR_INVALID_ARG
    if not torch.cuda.is_available():
        assert call(lib, name, args, dict(R=2 ** 31 - 1024)) == b.MOE_ERR_UNSUPPORTED_DEVICE


def test_no_rows_is_valid_and_needs_no_device(lib):
    none = dict(R=0, x=None, off=None, out=None, w=None)
    assert call(lib, "moe_expert_gated", GATED, none) == b.MOE_OK
    assert call(lib, "moe_expert_linear", LINEAR, none) == b.MOE_OK
    assert call(lib, "moe_unpermute_backward", UNPERMUTE_BW, dict(T=0)) == b.MOE_OK


def tensors(R=4, K=16, N=24, E=2, dtype=BF):
    return dict(x=torch.zeros(R, K, dtype=dtype), w=torch.zeros(E, N, K, dtype=dtype),
                off=torch.zeros(E + 1, dtype=torch.int64), y=torch.zeros(R, N, dtype=dtype),
                h=torch.zeros(R, N // 2, dtype=dtype), b=torch.zeros(E, N, dtype=dtype))


def refused(match, fn, *args, **kw):
    with pytest.raises(ValueError, match=match):
        fn(*args, **kw)


def test_binding_refuses_wrong_sizes_and_types():
    t = tensors()
    x, w, off, y, h, bias = (t[k] for k in ("x", "w", "off", "y", "h", "b"))
    refused("out must hold", mp.moe_expert_gated, x, w, off, y)
    refused("preact must hold", mp.moe_expert_gated, x, w, off, h, preact=h)
    refused("the rows must hold", mp.moe_expert_gated, x[:, :8], w, off, h)
    refused("the rows is", mp.moe_expert_gated, x.half(), w, off, h)
    refused("out is", mp.moe_expert_gated, x, w, off, h.float())
    refused("bfloat16 or float16", mp.moe_expert_gated, x.float(), w.float(), off, h)
    refused("holds 2 elements", mp.moe_expert_gated, x, w, off[:2], h)
    refused("must be int64", mp.moe_expert_gated, x, w, off.int(), h)
    refused("activation must be", mp.moe_expert_gated, x, w, off, h, activation="tanh")
    refused("as many up rows", mp.moe_expert_gated, x, w[:, :23], off, h)
    refused(r"\[experts, out, in\]", mp.moe_expert_gated, x, w[0], off, h)
    refused("CUDA tensor", mp.moe_expert_gated, x, w, off, h)
    refused("bias must hold", mp.moe_expert_linear, x, w, off, y, bias=bias[:1])
    refused("residual must hold", mp.moe_expert_linear, x, w, off, y, residual=h)
    refused("out must hold", mp.moe_expert_linear, x, w, off, h)
    refused("CUDA tensor", mp.moe_expert_linear, x, w, off, y)
    refused("go with an activation", mp.moe_expert_linear_backward, y, x, w, off, preact=y)
    refused("go with an activation", mp.moe_expert_linear_backward, y, x, w, off,
            activation="silu")
    refused("d_rows needs weight", mp.moe_expert_linear_backward, y, x, None, off, d_rows=x,
            d_weight=w)
    refused("d_weight needs rows", mp.moe_expert_linear_backward, y, None, w, off, d_weight=w)
    refused("d_weight must hold", mp.moe_expert_linear_backward, y, x, w, off, d_weight=w[:1])
    refused("d_bias must hold", mp.moe_expert_linear_backward, y, x, w, off, d_bias=bias[:, :8])
    refused("d_out must hold", mp.moe_expert_gated_backward, y, x, w, off, y, y)
    refused("d_preact must hold", mp.moe_expert_gated_backward, h, x, w, off, y, h)
    refused("d_rows needs weight", mp.moe_expert_gated_backward, h, x, None, off, y, y, d_rows=x,
            d_weight=w)


def test_binding_refuses_wrong_unpermute_gradients():
    T, K, H = 3, 2, 8
    d, rows = torch.zeros(T, H, dtype=BF), torch.zeros(T * K, H, dtype=BF)
    wts, inv = torch.zeros(T, K), torch.zeros(T * K, dtype=torch.int32)
    f = mp.moe_unpermute_backward
    refused("nothing to compute", f, d, None, wts, inv, None, None)
    refused("goes with", f, d, None, wts, inv, rows, wts)
    refused("goes with", f, d, rows, wts, inv, rows, None)
    refused("float32", f, d, rows, wts.double(), inv, rows, wts)
    refused("int32", f, d, rows, wts, inv.long(), rows, wts)
    refused("takes bf16", f, d.float(), rows, wts, inv, rows, wts)
    refused("d_rows must hold", f, d, rows, wts, inv, rows[:4], wts)
    refused("d_topk_weights must hold", f, d, rows, wts, inv, rows, wts[:, :1])
    refused("inv_permuted_idx holds", f, d, rows, wts, inv[:4], rows, wts)
    refused("at least 3 rows", f, d[:2], rows, wts, inv, rows, wts)


@pytest.mark.parametrize("act", ["none", "silu", "gelu", "relu"])
def test_reference_gradients_are_the_differences(act):
    g = torch.Generator().manual_seed(1)
    x = torch.randn(7, 6, generator=g, dtype=torch.float64)
    w = torch.randn(2, 8, 6, generator=g, dtype=torch.float64)
    d = torch.randn(7, 8, generator=g, dtype=torch.float64)
    offset = torch.tensor([0, 3, 7])
    for form in ("gated", "linear"):
        fn, dd = (ref.gated, d[:, :4]) if form == "gated" else (ref.linear, d)
        _, z = fn(x, w, offset, act)
        dz = ref.gated_dz(dd, z, act) if form == "gated" else ref.exact(dd) * ref.act_grad(act, z)
        dx, dw, db = ref.gradients(dz, x, w, offset)
        h = 1e-6
        for _ in range(3):
            vx, vw = (torch.randn(t.shape, generator=g, dtype=torch.float64) for t in (x, w))
            up, down = ((fn(x + s * h * vx, w + s * h * vw, offset, act)[0].v * dd).sum()
                        for s in (1, -1))
            slope = (up - down) / (2 * h)
            assert abs((dx.v * vx).sum() + (dw.v * vw).sum() - slope) < 1e-6 * (1 + abs(slope))
        assert torch.allclose(db.v[0], dz.v[:3].sum(0))
