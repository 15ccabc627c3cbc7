"""Plain 64-bit forms of the 8-bit expert operators, with a bound on how far a
kernel may be from them, element by element (see expert_ref.Val).

A product's sums are held in 32 bits.  With scales for groups of 128 columns a
group's sum is off by at most 128 * 2^-23 of its terms' size, and each of G
groups is scaled (two roundings) and added (one); with whole numbers the sum is
exact while its terms' size is at most 2^24, and otherwise off by 2^-23 of it per
term; then it is scaled (two roundings) and was converted (one).
"""
import torch

import expert_ref as ref
from expert_ref import Val

E4M3, INT8 = torch.float8_e4m3fn, torch.int8
GROUP = 128


def groups(n):
    return -(-n // GROUP)


def scale_shapes(code, R, E, N, K, parts):
    """Shapes of the rows' and the weights' scales."""
    if code == INT8:
        return (R, 1), (E, N)
    return (R, groups(K)), (E, parts * groups(N // parts), groups(K))


def product(x, xs, w, ws, parts):
    """Rows [R, K] with scales times an expert's weight [N, K] with its scales."""
    N, K = w.shape
    if x.dtype == INT8:
        v = x.double() @ w.double().t()
        mag = x.double().abs() @ w.double().abs().t()
        s = xs.double() * ws.double()
        n = torch.where(mag <= 2.0 ** 24, 0.0, float(K)) + 3
        return Val(v * s, n * 2.0 ** -23 * mag * s.abs() + ref.FLUSH)
    column = torch.arange(K, device=w.device) // GROUP
    feature = torch.arange(N, device=w.device)
    block = feature % (N // parts) // GROUP + feature // (N // parts) * groups(N // parts)
    a = x.double() * xs.double()[:, column]
    b = w.double() * ws.double()[block][:, column]
    n = min(K, GROUP) + 3 * groups(K) + 2
    return Val(a @ b.t(), n * 2.0 ** -23 * (a.abs() @ b.abs().t()) + K * ref.FLUSH)


def gated(x, xs, w, ws, offset, act):
    parts = []
    for e, (lo, hi) in ref.segments(offset):
        z = product(x[lo:hi], xs[lo:hi], w[e], ws[e], 2)
        gate, up = ref.split(z, w.shape[1] // 2)
        parts.append(ref.act(act, gate) * up)
    return ref.cat(parts)


def linear(x, xs, w, ws, offset, act, bias=None, residual=None):
    parts = []
    for e, (lo, hi) in ref.segments(offset):
        z = product(x[lo:hi], xs[lo:hi], w[e], ws[e], 1)
        z = z if bias is None else z + ref.exact(bias[e].expand(hi - lo, -1))
        y = ref.act(act, z)
        parts.append(y if residual is None else y + ref.exact(residual[lo:hi]))
    return ref.cat(parts)


def quantised(x, code):
    """Codes and scales of rows [R, H], by the operator's rule: divisions of fp32."""
    x = x.float()
    R, H = x.shape
    largest = 127.0 if code == INT8 else 448.0
    size = H if code == INT8 else GROUP
    padded = torch.nn.functional.pad(x, (0, -(-H // size) * size - H)).view(R, -1, size)
    amax = padded.nan_to_num(0.0, float("inf"), float("-inf")).abs().amax(2, keepdim=True)
    # (divided by a tensor: by a number, torch multiplies with its reciprocal)
    scale = torch.where(amax > 0, amax / torch.full_like(amax, largest), torch.ones_like(amax))
    if code == INT8:
        scale[padded.isnan().any(2)] = float("nan")
    q = padded / scale
    if code == INT8:
        q = torch.where(scale.isfinite(), q.round().clamp(-127, 127), torch.zeros_like(q))
    else:
        q = q.clamp(-448, 448)
    q = q.to(code).view(torch.int8).view(R, -1)[:, :H].contiguous()
    return q.view(code), scale.view(R, -1).contiguous()
