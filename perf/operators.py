"""Measured cases of the expert operators: the grouped gated projection, the
grouped linear product with its epilogue, and the gradient of moe_unpermute,
each as a user calls it, beside a plain form of the same mathematics.

Rows are in the order moe_permute leaves them in: sorted by local expert,
expert e holding rows offset[e] .. offset[e+1).

  gated    h = act(x Wg^T) * (x Wu^T), weight [E_L, 2F, H] = gate rows, then up
           rows; `train` adds the backward pass (d_rows, d_weight).
  linear   y = act(x W^T + b) + residual, weight [E_L, N, K]; `train` adds the
           backward pass (d_rows, d_weight, d_bias).
  combine  backward of out[t] = sum_k w[t,k] * row[inv[t,k]]: d_rows and d_w.

`own` false: elementary torch operations in fp32, rounded once at the end.
`own` true: the calls of moe_token_permute_gb300.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}

# Padded rows up to which the plain form multiplies all experts as one batch;
# above it, one product per expert wastes less (a skewed routing pads 16-fold).
PADDED_ROWS = 8192


def listed():
    gated = dict(op="gated", dtype="bf16", act="silu", zipf=0.0, train=False)
    linear = dict(op="linear", dtype="bf16", act="none", zipf=0.0, train=False, bias=False,
                  residual=False)
    return [
        # one decoded token, 8 of 128 experts: 8 rows, weights streamed, latency counts
        dict(gated, name="gated_qwen3_T1", T=1, K=8, E=128, local=128, H=2048, F=768, zipf=1.2),
        # a decode batch: a few rows for most experts, bound by the weights
        dict(gated, name="gated_qwen3_T64", T=64, K=8, E=128, local=128, H=2048, F=768, zipf=1.2),
        # a prompt through few large experts: bound by the matrix instructions
        dict(gated, name="gated_mixtral_T4096", T=4096, K=2, E=8, local=8, H=4096, F=14336),
        # a quarter of the experts local, the rows behind the last one unused
        dict(gated, name="gated_dsv2lite_map_T8192", T=8192, K=6, E=64, local=16, H=2048, F=1408,
             dtype="fp16", act="gelu"),
        # a training step over many experts with skewed, ragged segments
        dict(gated, name="gated_train_qwen3_T8192", T=8192, K=8, E=128, local=128, H=2048, F=768,
             zipf=1.2, train=True),
        # a small training step with sizes that fill no tile
        dict(gated, name="gated_train_odd_T515", T=515, K=3, E=10, local=10, H=1000, F=344,
             dtype="fp16", train=True),
        # the down projection of one decoded token
        dict(linear, name="linear_mixtral_T1", T=1, K=2, E=8, local=8, N=4096, D=14336),
        # the down projection of a prompt over many experts: 128 rows each on average
        dict(linear, name="linear_dsv3_T4096", T=4096, K=8, E=256, local=256, N=7168, D=2048,
             zipf=1.0),
        # one dense layer (a single expert holding every row) with the whole epilogue
        dict(linear, name="linear_dense_T8191", T=8191, K=1, E=1, local=1, N=4096, D=4096,
             bias=True, act="gelu", residual=True),
        # the down projection of a training step, with bias gradients
        dict(linear, name="linear_train_mixtral_T4096", T=4096, K=2, E=8, local=8, N=4096,
             D=14336, bias=True, train=True),
        # the combine's gradient for a small micro-batch
        dict(name="combine_backward_qwen3_T64", op="combine", dtype="bf16", T=64, K=8, E=128,
             local=128, H=2048),
        # and for a long one with wide rows: pure memory traffic
        dict(name="combine_backward_dsv3_T4096", op="combine", dtype="bf16", T=4096, K=8, E=256,
             local=256, H=7168),
    ]


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    def width(lo, hi):
        n = max(8, spread(lo, hi) // 8 * 8)
        return n + 8 if n == 3072 else n

    op = rng.choice(["gated", "gated", "linear", "linear", "combine"])
    E = rng.choice([1, 4, 8, 10, 32, 64, 128, 200, 256])
    K = min(E, rng.choice([1, 2, 3, 6, 8]))
    local = E if rng.random() < 0.7 else max(1, E // rng.choice([2, 4]))
    while True:
        T = spread(1, 8192)
        case = dict(op=op, T=T, K=K, E=E, local=local if T >= 32 else E)
        if op == "combine":
            return dict(case, dtype="bf16", H=width(128, 7168))
        case.update(dtype=rng.choice(["bf16", "bf16", "fp16"]), train=rng.random() < 0.4,
                    zipf=rng.choice([0.0, 1.0, 1.2]))
        if op == "gated":
            case.update(act=rng.choice(["silu", "silu", "gelu"]), H=width(512, 7168),
                        F=width(256, 14336))
        else:
            case.update(act=rng.choice(["none", "gelu", "relu"]), N=width(512, 7168),
                        D=width(256, 14336), bias=rng.random() < 0.5, residual=rng.random() < 0.3)
        weight = local * 2 * (2 * case["H"] * case["F"] if op == "gated" else case["N"] * case["D"])
        if _flops(case, case["T"] * K * local / E) <= 1.5e12 and weight <= 3e9:
            return case


def _flops(case, n):
    if case["op"] == "combine":
        return 3.0 * n * case["H"]
    mn = 2 * case["F"] * case["H"] if case["op"] == "gated" else case["N"] * case["D"]
    return (3 if case["train"] else 1) * 2.0 * n * mn


def _routing(case, seed):
    """topk ids [T, K] (distinct experts per token), drawn on the host."""
    g = torch.Generator().manual_seed(seed)
    rank = torch.arange(1, case["E"] + 1, dtype=torch.float32)
    popularity = -case.get("zipf", 0.0) * rank.log()
    popularity = popularity[torch.randperm(case["E"], generator=g)]
    u = torch.rand(case["T"], case["E"], generator=g).clamp_(1e-9, 1 - 1e-7)
    return (popularity - (-u.log()).log()).topk(case["K"], dim=1).indices


def _counts(case, seed):
    return torch.bincount(_routing(case, seed).flatten(), minlength=case["E"])[:case["local"]]


def work(case):
    counts = _counts(case, 0)
    n, active = int(counts.sum()), int((counts > 0).sum())
    rows = case["T"] * case["K"]
    if case["op"] == "combine":
        # read d_out, the rows, weights and indices; write d_rows and d_w
        moved = case["T"] * case["H"] * 2 + n * case["H"] * 4 + rows * 12
    elif case["op"] == "gated":
        H, F = case["H"], case["F"]
        moved = n * (H + F) * 2 + active * 2 * F * H * 2
        if case["train"]:
            moved += n * (H + F) * 2 + case["local"] * 2 * F * H * 2
    else:
        D, N = case["D"], case["N"]
        moved = n * (D + N * (2 if case["residual"] else 1)) * 2 + active * N * D * 2
        moved += case["local"] * N * 2 if case["bias"] else 0
        if case["train"]:
            moved += n * (D + N) * 2 + case["local"] * N * D * 2
            moved += case["local"] * N * 2 if case["bias"] else 0
    if case["op"] != "combine":
        moved += (case["local"] + 1) * 8  # the offsets
    return {"bytes": moved, "flops": _flops(case, n)}


def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    dtype = DTYPES[case["dtype"]]

    def normal(*shape, scale=1.0):
        t = torch.randn(*shape, generator=g, device="cuda", dtype=dtype)
        return t if scale == 1.0 else t.mul_(scale)

    def buffer(*shape, dtype=dtype):  # zeros: rows behind the last expert's stay unwritten
        return torch.zeros(*shape, device="cuda", dtype=dtype)

    R, L = case["T"] * case["K"], case["local"]
    s = dict(case)
    if case["op"] == "combine":
        ids = _routing(case, seed).flatten()
        order = torch.argsort(ids, stable=True)
        order = order[ids[order] < L]
        inv = torch.full((R,), -1, dtype=torch.int32)
        inv[order] = torch.arange(order.numel(), dtype=torch.int32)
        s.update(n=order.numel(), R=R, inv=inv.cuda(), rows=normal(R, case["H"]),
                 d_out=normal(case["T"], case["H"]), d_rows=buffer(R, case["H"]),
                 weights=torch.softmax(torch.randn(case["T"], case["K"], generator=g,
                                                   device="cuda"), dim=1),
                 d_weights=buffer(case["T"], case["K"], dtype=torch.float32))
        return s
    counts = _counts(case, seed)
    ends = counts.cumsum(0)
    offset = torch.cat([torch.zeros(1, dtype=torch.int64), ends])
    inner, outer = ((case["H"], 2 * case["F"]) if case["op"] == "gated"
                    else (case["D"], case["N"]))
    width = case["F"] if case["op"] == "gated" else case["N"]
    s.update(n=int(ends[-1]), R=R, offset=offset.cuda(), rows=normal(R, inner),
             weight=normal(L, outer, inner, scale=inner ** -0.5), out=buffer(R, width),
             bias=None, residual=None, preact=None, d_preact=None, d_bias=None)
    active = torch.nonzero(counts).flatten()
    most = int(counts.max())
    s.update(groups=[(int(e), int(offset[e]), int(offset[e + 1])) for e in active],
             active=active.cuda(), most=most, padded=active.numel() * most <= PADDED_ROWS)
    if s["padded"] and s["n"]:  # row r of the k-th expert with rows: slot k * most + r
        within = torch.cat([torch.arange(int(c)) for c in counts[active]])
        s["slot"] = (torch.repeat_interleave(torch.arange(active.numel()), counts[active]) * most
                     + within).cuda()
    if case.get("bias"):
        s["bias"] = normal(L, outer)
    if case.get("residual"):
        s["residual"] = normal(R, outer)
    if case["train"]:
        s.update(d_out=normal(R, width), d_rows=buffer(R, inner), d_weight=buffer(L, outer, inner))
        if case["op"] == "gated" or case["act"] != "none":
            s.update(preact=buffer(R, outer), d_preact=buffer(R, outer))
        if case.get("bias"):
            s["d_bias"] = buffer(L, outer)
    return s


# ---- the plain form --------------------------------------------------------

def _pad(s, x):
    p = x.new_zeros(len(s["groups"]) * s["most"], x.shape[1])
    p[s["slot"]] = x
    return p.view(len(s["groups"]), s["most"], x.shape[1])


def _product(s, x, transposed):
    """fp32 x [n, in] times each row's expert's weight (or its transpose)."""
    w = s["weight"]
    if not s["n"]:
        return x.new_zeros(0, w.shape[2] if transposed else w.shape[1])
    if s["padded"]:
        w = w[s["active"]].float()
        y = torch.bmm(_pad(s, x), w if transposed else w.transpose(1, 2))
        return y.view(-1, y.shape[2])[s["slot"]]
    return torch.cat([x[lo:hi] @ (w[e].float() if transposed else w[e].float().t())
                      for e, lo, hi in s["groups"]])


def _weight_gradient(s, d, x):
    out = torch.zeros_like(s["weight"])
    if s["padded"] and s["n"]:
        out[s["active"]] = torch.bmm(_pad(s, d).transpose(1, 2), _pad(s, x)).to(out.dtype)
        return out
    for e, lo, hi in s["groups"]:
        out[e] = d[lo:hi].t() @ x[lo:hi]
    return out


def _bias_gradient(s, d):
    out = torch.zeros_like(s["bias"], dtype=torch.float32)
    expert = torch.repeat_interleave(torch.arange(s["local"], device="cuda"),
                                     s["offset"].diff(), output_size=s["n"])
    return out.index_add_(0, expert, d).to(s["bias"].dtype)


def _rows_out(s, y):
    """Rounded to the rows' type, zeros for the rows that belong to no expert."""
    y = y.to(s["rows"].dtype)
    return y if s["n"] == s["R"] else torch.nn.functional.pad(y, (0, 0, 0, s["R"] - s["n"]))


GELU_A, GELU_B = math.sqrt(2.0 / math.pi), 0.044715


def _act(name, z):
    if name == "silu":
        return z / (1 + torch.exp(-z))
    if name == "gelu":
        return 0.5 * z * (1 + torch.tanh(GELU_A * (z + GELU_B * z * z * z)))
    return z.clamp(min=0) if name == "relu" else z


def _act_gradient(name, z):
    if name == "silu":
        p = 1 / (1 + torch.exp(-z))
        return p * (1 + z * (1 - p))
    if name == "gelu":
        t = torch.tanh(GELU_A * (z + GELU_B * z * z * z))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * GELU_A * (1 + 3 * GELU_B * z * z)
    return (z > 0).to(z.dtype) if name == "relu" else torch.ones_like(z)


def _plain_gated(s):
    n, F = s["n"], s["F"]
    x = s["rows"][:n].float()
    z = _product(s, x, False)
    gate, up = z[:, :F], z[:, F:]
    a = _act(s["act"], gate)
    out = {"out": _rows_out(s, a * up)}
    if s["train"]:
        d = s["d_out"][:n].float()
        dz = torch.cat([d * up * _act_gradient(s["act"], gate), d * a], dim=1)
        out["d_rows"] = _rows_out(s, _product(s, dz, True))
        out["d_weight"] = _weight_gradient(s, dz, x)
    return out


def _plain_linear(s):
    n = s["n"]
    x = s["rows"][:n].float()
    z = _product(s, x, False)
    if s["bias"] is not None:
        expert = torch.repeat_interleave(torch.arange(s["local"], device="cuda"),
                                         s["offset"].diff(), output_size=n)
        z = z + s["bias"].float()[expert]
    y = _act(s["act"], z)
    if s["residual"] is not None:
        y = y + s["residual"][:n].float()
    out = {"out": _rows_out(s, y)}
    if s["train"]:
        d = s["d_out"][:n].float()
        if s["act"] != "none":
            d = d * _act_gradient(s["act"], z)
        out["d_rows"] = _rows_out(s, _product(s, d, True))
        out["d_weight"] = _weight_gradient(s, d, x)
        if s["bias"] is not None:
            out["d_bias"] = _bias_gradient(s, d)
    return out


def _plain_combine(s):
    T, K, H = s["T"], s["K"], s["H"]
    inv = s["inv"].long()
    keep = inv >= 0
    d = s["d_out"].float()
    rows = s["rows"][inv.clamp(min=0)].float().view(T, K, H)
    dw = (rows * d[:, None]).sum(dim=2) * keep.view(T, K)
    d_rows = torch.zeros_like(s["rows"])
    d_rows[inv[keep]] = (s["weights"][:, :, None] * d[:, None]).to(d_rows.dtype).view(-1, H)[keep]
    return {"d_rows": d_rows, "d_weights": dw}


# ---- the framework's calls -------------------------------------------------

def _own_gated(s):
    import moe_token_permute_gb300 as mp
    mp.moe_expert_gated(s["rows"], s["weight"], s["offset"], s["out"], activation=s["act"],
                        preact=s["preact"])
    out = {"out": s["out"]}
    if s["train"]:
        mp.moe_expert_gated_backward(s["d_out"], s["rows"], s["weight"], s["offset"], s["preact"],
                                     s["d_preact"], activation=s["act"], d_rows=s["d_rows"],
                                     d_weight=s["d_weight"])
        out.update(d_rows=s["d_rows"], d_weight=s["d_weight"])
    return out


def _own_linear(s):
    import moe_token_permute_gb300 as mp
    mp.moe_expert_linear(s["rows"], s["weight"], s["offset"], s["out"], bias=s["bias"],
                         activation=s["act"], residual=s["residual"], preact=s["preact"])
    out = {"out": s["out"]}
    if s["train"]:
        mp.moe_expert_linear_backward(s["d_out"], s["rows"], s["weight"], s["offset"],
                                      activation=s["act"], preact=s["preact"],
                                      d_preact=s["d_preact"], d_rows=s["d_rows"],
                                      d_weight=s["d_weight"], d_bias=s["d_bias"])
        out.update(d_rows=s["d_rows"], d_weight=s["d_weight"])
        if s["bias"] is not None:
            out["d_bias"] = s["d_bias"]
    return out


def _own_combine(s):
    import moe_token_permute_gb300 as mp
    mp.moe_unpermute_backward(s["d_out"], s["rows"], s["weights"], s["inv"], s["d_rows"],
                              s["d_weights"])
    return {"d_rows": s["d_rows"], "d_weights": s["d_weights"]}


def run(state):
    form = {"gated": (_plain_gated, _own_gated), "linear": (_plain_linear, _own_linear),
            "combine": (_plain_combine, _own_combine)}[state["op"]]
    return form[1 if own else 0](state)


# ---- the definition in 64 bits ---------------------------------------------

def _exact_act(name, z):
    """The activation and its derivative, in 64 bits."""
    if name == "silu":
        p = torch.sigmoid(z)
        return z * p, p + z * p * (1 - p)
    if name == "gelu":
        c = math.sqrt(2 / math.pi)
        arg = c * z + c * 0.044715 * z ** 3
        p = torch.sigmoid(2 * arg)
        return z * p, p + z * p * (1 - p) * 2 * (c + 3 * c * 0.044715 * z ** 2)
    if name == "relu":
        return torch.relu(z), torch.heaviside(z, torch.zeros((), dtype=z.dtype, device=z.device))
    return z, torch.ones_like(z)


def exact(case, seed):
    s = prepare(case, seed)
    if _flops(case, s["n"]) > 8e12:  # over about 20 seconds in 64 bits
        return None
    if case["op"] == "combine":
        return _exact_combine(s)
    gated, F = case["op"] == "gated", case.get("F")
    shape = s["weight"].shape
    got = {"out": [], "d_rows": [], "d_weight": [], "d_bias": []}
    begin = 0
    for e, end in enumerate(s["offset"].tolist()[1:]):
        x, w = s["rows"][begin:end].double(), s["weight"][e].double()
        z = torch.einsum("rk,nk->rn", x, w)
        if s["bias"] is not None:
            z += s["bias"][e].double()
        a, da = _exact_act(case["act"], z[:, :F] if gated else z)
        y = a * z[:, F:] if gated else a
        if s["residual"] is not None:
            y = y + s["residual"][begin:end].double()
        got["out"].append(y)
        if case["train"]:
            dy = s["d_out"][begin:end].double()
            dz = torch.cat([dy * z[:, F:] * da, dy * a], dim=1) if gated else dy * da
            got["d_rows"].append(torch.einsum("rn,nk->rk", dz, w))
            got["d_weight"].append(torch.einsum("rn,rk->nk", dz, x).to(torch.float32)
                                   if shape.numel() > 1 << 29 else
                                   torch.einsum("rn,rk->nk", dz, x))
            got["d_bias"].append(dz.sum(dim=0))
        begin = end
    def whole(parts):
        return torch.nn.functional.pad(torch.cat(parts), (0, 0, 0, s["R"] - s["n"]))

    out = {"out": whole(got["out"])}
    if case["train"]:
        out.update(d_rows=whole(got["d_rows"]), d_weight=torch.stack(got["d_weight"]))
        if s["bias"] is not None:
            out["d_bias"] = torch.stack(got["d_bias"])
    return out


def _exact_combine(s):
    T, K, H = s["T"], s["K"], s["H"]
    at = s["inv"].long()
    slots = torch.nonzero(at >= 0).flatten()
    rows = at[slots]
    token = slots // K
    d_rows = torch.zeros(T * K, H, dtype=torch.float64, device="cuda")
    d_weights = torch.zeros(T * K, dtype=torch.float64, device="cuda")
    for part in torch.arange(slots.numel(), device="cuda").split(8192):
        d = s["d_out"][token[part]].double()
        d_rows[rows[part]] = s["weights"].flatten()[slots[part]].double()[:, None] * d
        d_weights[slots[part]] = torch.einsum("rh,rh->r", d, s["rows"][rows[part]].double())
    return {"d_rows": d_rows, "d_weights": d_weights.view(T, K)}
