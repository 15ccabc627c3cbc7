"""Plain 64-bit forms of the expert operators, each with a bound on how far a
kernel may be from it, element by element.

The bound is built up with the value.  `Val` holds a 64-bit value v and a bound
e on the error of the number the kernel holds in its place:
  - a product of k terms accumulated in fp32 (in any order, truncating or
    rounding): k * 2^-23 * sum |a||b|, plus the operands' own errors;
  - a rounding to a type of p significant bits: 2^-p |v|, plus half the type's
    smallest subnormal;
  - an activation: its Lipschitz constant times the argument's error, plus
    2^-18 of the value for the fast exponential and reciprocal.
Nothing in it is measured.
"""
import math

import torch

BITS = {torch.bfloat16: 8, torch.float16: 11}
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}
FLUSH = 2.0 ** -126  # an fp32 product or sum this small may be flushed to zero
FAST = 2.0 ** -18
C = math.sqrt(2 / math.pi)
# Lipschitz constants of act and act' (and |act'| <= first): silu' peaks at
# 1.0999, silu'' at 0.5; gelu' at 1.13, gelu'' at 0.80 (2 phi(0), tanh form).
LIP = {"none": (1.0, 0.0), "silu": (1.1, 0.5), "gelu": (1.13, 0.85), "relu": (1.0, 0.0)}


class Val:
    def __init__(self, v, e=None):
        self.v, self.e = v, torch.zeros_like(v) if e is None else e

    def __add__(self, o):
        v = self.v + o.v
        return Val(v, self.e + o.e + 2.0 ** -24 * (v.abs() + self.e + o.e))

    def __mul__(self, o):
        v = self.v * o.v
        e = self.e * o.v.abs() + o.e * self.v.abs() + self.e * o.e
        return Val(v, e + 2.0 ** -24 * (v.abs() + e) + FLUSH)


def exact(t):
    return Val(t.double())


def rounded(a, dtype):
    return Val(a.v, a.e + 2.0 ** -BITS[dtype] * (a.v.abs() + a.e) + TINY[dtype])


def product(a, b):
    """a [i, k] times b [j, k] over k."""
    k = max(1, a.v.shape[1])
    v = a.v @ b.v.t()
    mag = (a.v.abs() + a.e) @ (b.v.abs() + b.e).t()
    e = a.e @ b.v.abs().t() + a.v.abs() @ b.e.t() + a.e @ b.e.t()
    return Val(v, e + k * (2.0 ** -23 * mag + FLUSH))


def act(name, z):
    v = {"none": lambda x: x, "relu": torch.relu,
         "silu": lambda x: x * torch.sigmoid(x),
         "gelu": lambda x: 0.5 * x * (1 + torch.tanh(C * (x + 0.044715 * x ** 3)))}[name](z.v)
    smooth = name in ("silu", "gelu")
    return Val(v, LIP[name][0] * z.e + (FAST * (v.abs() + z.e) + FLUSH if smooth else 0))


def act_grad(name, z):
    x = z.v
    if name == "silu":
        p = torch.sigmoid(x)
        v = p * (1 + x * (1 - p))
    elif name == "gelu":
        t = torch.tanh(C * (x + 0.044715 * x ** 3))
        v = 0.5 * (1 + t) + 0.5 * x * (1 - t * t) * C * (1 + 3 * 0.044715 * x * x)
    elif name == "relu":
        v = (x > 0).double()
        return Val(v, (x.abs() <= z.e).double() * (z.e > 0))  # either side of the kink
    else:
        return Val(torch.ones_like(x))
    # the terms of act' are at most 1 + |z| in size
    return Val(v, LIP[name][1] * z.e + FAST * (1 + x.abs()))


def segments(offset):
    o = offset.tolist()
    return list(enumerate(zip(o[:-1], o[1:])))


def cat(parts):
    return Val(torch.cat([p.v for p in parts]), torch.cat([p.e for p in parts]))


def stack(parts):
    return Val(torch.stack([p.v for p in parts]), torch.stack([p.e for p in parts]))


def split(a, n):
    return Val(a.v[:, :n], a.e[:, :n]), Val(a.v[:, n:], a.e[:, n:])


def gated(x, w, offset, name):
    """out and preact (unrounded) of the rows that belong to an expert."""
    z = cat([product(exact(x[lo:hi]), exact(w[e])) for e, (lo, hi) in segments(offset)])
    gate, up = split(z, w.shape[1] // 2)
    return act(name, gate) * up, z


def linear(x, w, offset, name, bias=None, residual=None):
    parts = []
    for e, (lo, hi) in segments(offset):
        z = product(exact(x[lo:hi]), exact(w[e]))
        parts.append(z if bias is None else z + exact(bias[e].expand(hi - lo, -1)))
    z = cat(parts)
    y = act(name, z)
    return (y if residual is None else y + exact(residual[:z.v.shape[0]])), z


def gated_dz(d_out, z, name):
    """d_preact from the saved z."""
    gate, up = split(z, z.v.shape[1] // 2)
    d = exact(d_out[:z.v.shape[0]])
    g, u = d * up * act_grad(name, gate), d * act(name, gate)
    return Val(torch.cat([g.v, u.v], 1), torch.cat([g.e, u.e], 1))


def transpose(a):
    return Val(a.v.t(), a.e.t())


def gradients(dz, x, w, offset):
    """d_rows, d_weight and d_bias from dz."""
    rows, weight, bias = [], [], []
    for e, (lo, hi) in segments(offset):
        d = Val(dz.v[lo:hi], dz.e[lo:hi])
        rows.append(product(d, exact(w[e].t())))
        weight.append(product(transpose(d), exact(x[lo:hi].t())))
        n = max(1, hi - lo)
        bias.append(Val(d.v.sum(0), d.e.sum(0) + n * 2.0 ** -23 * (d.v.abs() + d.e).sum(0)))
    return cat(rows), stack(weight), stack(bias)


def check(got, want, dtype, what):
    """got against the bound, after its rounding to dtype."""
    want = rounded(want, dtype) if dtype in BITS else want
    got = got.double()
    assert got.shape == want.v.shape, (what, got.shape, want.v.shape)
    assert torch.isfinite(got).all(), f"{what}: not finite"
    over = (got - want.v).abs() - want.e
    worst = over.max().item() if over.numel() else -1.0
    assert worst <= 0, f"{what}: {int((over > 0).sum())} of {over.numel()} beyond the bound, " \
                       f"worst by {worst}"
