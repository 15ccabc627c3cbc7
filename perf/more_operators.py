"""Measured cases of the 8-bit expert operators: rows quantised to 8 bits, and the
grouped products of 8-bit rows and weights, each as a user calls it, beside a plain
form of the same mathematics.

Two forms of 8 bits, a value being its code times a scale:
  fp8   e4m3 codes; rows have a scale for each 128 columns ([R, ceil(H / 128)]),
        weights one for each block of 128 x 128.
  int8  whole numbers; rows have one scale each ([R, 1]), weights one for each
        output channel.

  quant   codes and scales of 16-bit rows: scale = amax / 448 (fp8) or / 127 (int8),
          1 where all is zero; code = x / scale to the nearest, ties to even.
  gated   h = act(x Wg^T) * (x Wu^T), weight [E_L, 2F, H] = gate rows, then up rows.
  linear  y = act(x W^T + b) + residual, weight [E_L, N, D].

Rows are in the order moe_permute leaves them in: sorted by local expert, expert e
holding rows offset[e] .. offset[e+1).

`own` false: elementary torch operations in fp32, rounded once at the end.
`own` true: the calls of moe_token_permute_gb300.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
CODES = {"fp8": torch.float8_e4m3fn, "int8": torch.int8}
LARGEST = {"fp8": 448.0, "int8": 127.0}
GROUP = 128

# Padded rows up to which the plain form multiplies all experts as one batch;
# above it, one product per expert wastes less.
PADDED_ROWS = 8192


def listed():
    gated = dict(op="gated", form="fp8", dtype="bf16", act="silu", zipf=0.0)
    linear = dict(op="linear", form="fp8", dtype="bf16", act="none", zipf=0.0, bias=False,
                  residual=False)
    return [
        # the tokens of a decode batch, ahead of the permute: latency counts
        dict(name="quant_int8_qwen3_T64", op="quant", form="int8", dtype="bf16", R=64, H=2048,
             used=64),
        # rows of odd number and width
        dict(name="quant_fp8_odd", op="quant", form="fp8", dtype="fp16", R=1543, H=1008,
             used=1200),
        # what the gated projection of a prompt hands to the down projection: pure
        # memory traffic
        dict(name="quant_fp8_mixtral_T4096", op="quant", form="fp8", dtype="bf16", R=8192,
             H=14336, used=8192),
        # one decoded token, 8 of 128 experts: 8 rows, weights streamed, latency counts
        dict(gated, name="gated_fp8_qwen3_T1", T=1, K=8, E=128, local=128, H=2048, F=768, zipf=1.2),
        # a decode batch: a few rows for most experts, bound by the weights
        dict(gated, name="gated_fp8_qwen3_T64", T=64, K=8, E=128, local=128, H=2048, F=768,
             zipf=1.2),
        # a prompt through few large experts: bound by the matrix instructions
        dict(gated, name="gated_fp8_mixtral_T4096", T=4096, K=2, E=8, local=8, H=4096, F=14336),
        # a quarter of the experts local, the rows behind the last one unused
        dict(gated, name="gated_int8_dsv2lite_map_T8192", form="int8", T=8192, K=6, E=64, local=16,
             H=2048, F=1408, dtype="fp16", act="gelu"),
        # the down projection of one decoded token
        dict(linear, name="linear_int8_mixtral_T1", form="int8", T=1, K=2, E=8, local=8, N=4096,
             D=14336),
        # a small batch with sizes that fill no tile and no group of 128
        dict(linear, name="linear_fp8_odd_T515", T=515, K=3, E=10, local=10, N=1000, D=1456,
             dtype="fp16", bias=True),
        # the down projection of a prompt over many experts: 128 rows each on average
        dict(linear, name="linear_fp8_dsv3_T4096", T=4096, K=8, E=256, local=256, N=7168, D=2048,
             zipf=1.0),
        # one dense layer (a single expert holding every row) with the whole epilogue
        dict(linear, name="linear_int8_dense_T8191", form="int8", T=8191, K=1, E=1, local=1, N=4096,
             D=4096, bias=True, act="gelu", residual=True),
        # the down projection of a prompt through few large experts
        dict(linear, name="linear_int8_mixtral_T4096", form="int8", T=4096, K=2, E=8, local=8,
             N=4096, D=14336),
    ]


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    def width(lo, hi, step):
        return max(step, spread(lo, hi) // step * step)

    op = rng.choice(["quant", "gated", "gated", "linear", "linear"])
    form = rng.choice(["fp8", "int8"])
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    if op == "quant":
        R, H = spread(1, 32768), width(128, 14336, 16)
        R = min(R, max(1, (8192 * 14336) // H))
        return dict(op=op, form=form, dtype=dtype, R=R, H=H,
                    used=R if rng.random() < 0.6 else rng.randint(0, R))
    E = rng.choice([1, 4, 8, 10, 32, 64, 128, 200, 256])
    K = min(E, rng.choice([1, 2, 3, 6, 8]))
    local = E if rng.random() < 0.7 else max(1, E // rng.choice([2, 4]))
    while True:
        T = spread(1, 8192)
        case = dict(op=op, form=form, dtype=dtype, T=T, K=K, E=E, local=local if T >= 32 else E,
                    zipf=rng.choice([0.0, 1.0, 1.2]))
        if op == "gated":
            case.update(act=rng.choice(["silu", "silu", "gelu"]), H=width(512, 7168, 16),
                        F=width(256, 14336, 8))
        else:
            case.update(act=rng.choice(["none", "gelu", "relu"]), N=width(512, 7168, 8),
                        D=width(256, 14336, 16), bias=rng.random() < 0.5,
                        residual=rng.random() < 0.3)
        weight = local * (2 * case["H"] * case["F"] if op == "gated" else case["N"] * case["D"])
        if _flops(case, case["T"] * K * local / E) <= 1.5e12 and weight <= 3.7e9:
            return case


def _flops(case, n):
    if case["op"] == "quant":
        return 3.0 * n * case["H"]
    mn = 2 * case["F"] * case["H"] if case["op"] == "gated" else case["N"] * case["D"]
    return 2.0 * n * mn


def _counts(case, seed):
    """Rows of each local expert, from topk ids (distinct experts per token) drawn on the host."""
    g = torch.Generator().manual_seed(seed)
    rank = torch.arange(1, case["E"] + 1, dtype=torch.float32)
    popularity = -case["zipf"] * rank.log()
    popularity = popularity[torch.randperm(case["E"], generator=g)]
    u = torch.rand(case["T"], case["E"], generator=g).clamp_(1e-9, 1 - 1e-7)
    ids = (popularity - (-u.log()).log()).topk(case["K"], dim=1).indices
    return torch.bincount(ids.flatten(), minlength=case["E"])[:case["local"]]


def _groups(n):
    return -(-n // GROUP)


def work(case):
    fp8 = case["form"] == "fp8"
    if case["op"] == "quant":
        n, H = case["used"], case["H"]
        # read the rows, write a byte each and the scales
        return {"bytes": n * H * 3 + n * (_groups(H) if fp8 else 1) * 4 + 16,
                "flops": _flops(case, n)}
    counts = _counts(case, 0)
    n, active = int(counts.sum()), int((counts > 0).sum())
    if case["op"] == "gated":
        inner, outer, blocks = case["H"], 2 * case["F"], 2 * _groups(case["F"])
        width, extra = case["F"], 0
    else:
        inner, outer, blocks = case["D"], case["N"], _groups(case["N"])
        width = case["N"]
        extra = (n * width * 2 if case["residual"] else 0) + (active * outer * 2 if case["bias"] else 0)
    scales = (n * _groups(inner) + active * blocks * _groups(inner) if fp8 else n + active * outer) * 4
    moved = n * inner + active * outer * inner + scales + n * width * 2 + extra
    return {"bytes": moved + (case["local"] + 1) * 8, "flops": _flops(case, n)}


def _quantised(x, form, dims):
    """Codes of x (fp32) and the scales that the maxima over `dims` give."""
    amax = x.abs().amax(dim=dims, keepdim=True)
    # (divided by a tensor: by a number, torch multiplies with its reciprocal)
    scale = torch.where(amax > 0, amax / torch.full_like(amax, LARGEST[form]),
                        torch.ones_like(amax))
    q = x / scale
    q = q.clamp(-448, 448) if form == "fp8" else q.round().clamp(-127, 127)
    return q.to(CODES[form]), scale


def _quantised_rows(x, form):
    """[R, H] -> codes [R, H], scales [R, groups or 1]."""
    R, H = x.shape
    if form == "int8":
        return _quantised(x.float(), form, 1)
    padded = torch.nn.functional.pad(x.float(), (0, _groups(H) * GROUP - H))
    codes, scale = _quantised(padded.view(R, _groups(H), GROUP), form, 2)
    return codes.view(R, -1)[:, :H].contiguous(), scale.view(R, -1).contiguous()


def _quantised_weight(w, form):
    """[N, K] of one expert -> codes, scales [ceil(N / 128), ceil(K / 128)] or [N]."""
    N, K = w.shape
    if form == "int8":
        codes, scale = _quantised(w, form, 1)
        return codes, scale.view(N)
    n, k = _groups(N), _groups(K)
    padded = torch.nn.functional.pad(w, (0, k * GROUP - K, 0, n * GROUP - N))
    codes, scale = _quantised(padded.view(n, GROUP, k, GROUP), form, (1, 3))
    return codes.view(n * GROUP, k * GROUP)[:N, :K], scale.view(n, k)


def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    dtype, form = DTYPES[case["dtype"]], case["form"]

    def normal(*shape, dtype=dtype):
        return torch.randn(*shape, generator=g, device="cuda", dtype=dtype)

    def activations(R, width):  # some columns are much larger than the rest, as in a model's
        return normal(R, width) * torch.exp(0.8 * normal(width)).clamp(max=16).to(dtype)

    s = dict(case)
    if case["op"] == "quant":
        R, H = case["R"], case["H"]
        columns = _groups(H) if form == "fp8" else 1
        s.update(rows=activations(R, H), codes=torch.zeros(R, H, device="cuda", dtype=CODES[form]),
                 scales=torch.zeros(R, columns, device="cuda"), offset=None)
        if case["used"] < R:  # the rows behind the last expert's belong to none
            s["offset"] = torch.tensor([0, case["used"] // 3, case["used"]], device="cuda")
        return s
    R, L = case["T"] * case["K"], case["local"]
    counts = _counts(case, seed)
    ends = counts.cumsum(0)
    offset = torch.cat([torch.zeros(1, dtype=torch.int64), ends])
    inner, outer = ((case["H"], 2 * case["F"]) if case["op"] == "gated"
                    else (case["D"], case["N"]))
    width = case["F"] if case["op"] == "gated" else case["N"]
    codes, scales = _quantised_rows(activations(R, inner), form)
    weight = torch.empty(L, outer, inner, device="cuda", dtype=CODES[form])
    parts = 2 if case["op"] == "gated" else 1  # gate and up rows have blocks of their own
    blocks = ((parts * _groups(outer // parts), _groups(inner)) if form == "fp8" else (outer,))
    weight_scales = torch.empty(L, *blocks, device="cuda")
    for e in range(L):  # channels of different size
        w = normal(outer, inner, dtype=torch.float32)
        w *= inner ** -0.5 * torch.exp(0.3 * normal(outer, 1, dtype=torch.float32))
        made = [_quantised_weight(p, form) for p in w.chunk(parts)]
        weight[e] = torch.cat([c.view(torch.int8) for c, _ in made]).view(CODES[form])
        weight_scales[e] = torch.cat([p for _, p in made])
    s.update(n=int(ends[-1]), R=R, offset=offset.cuda(), codes=codes, scales=scales, weight=weight,
             weight_scales=weight_scales, bias=None, residual=None,
             out=torch.zeros(R, width, device="cuda", dtype=dtype))
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
        s["residual"] = normal(R, width)
    return s


# ---- the plain form --------------------------------------------------------

def _spread_scale(scale, sizes):
    """Scales of blocks of 128 repeated over the trailing `sizes`."""
    for d, n in zip(range(-len(sizes), 0), sizes):
        scale = scale.repeat_interleave(GROUP, dim=d).narrow(d, 0, n)
    return scale


def _values(s, codes, scales, wide):
    """The fp32 values of rows (scales [.., groups or 1])."""
    if s["form"] == "int8":
        return codes.to(wide) * scales.to(wide)
    return codes.to(wide) * _spread_scale(scales.to(wide), (codes.shape[-1],))


def _weight_values(s, codes, scales, wide):
    """The values of weights [.., out, in]."""
    if s["form"] == "int8":
        return codes.to(wide) * scales.to(wide)[..., None]
    out, inner = codes.shape[-2:]
    if s["op"] == "linear":
        return codes.to(wide) * _spread_scale(scales.to(wide), (out, inner))
    gate, up = scales.to(wide).chunk(2, dim=-2)
    spread = torch.cat([_spread_scale(p, (out // 2, inner)) for p in (gate, up)], dim=-2)
    return codes.to(wide) * spread


def _product(s):
    """fp32 rows times each row's expert's weight."""
    n = s["n"]
    if not n:
        return s["scales"].new_zeros(0, s["weight"].shape[1])
    x = _values(s, s["codes"][:n], s["scales"][:n], torch.float32)
    if s["padded"]:
        at = s["active"]
        w = _weight_values(s, s["weight"].view(torch.int8)[at].view(s["weight"].dtype),
                           s["weight_scales"][at], torch.float32)
        p = x.new_zeros(len(s["groups"]) * s["most"], x.shape[1])
        p[s["slot"]] = x
        y = torch.bmm(p.view(len(s["groups"]), s["most"], -1), w.transpose(1, 2))
        return y.view(-1, y.shape[2])[s["slot"]]
    return torch.cat([x[lo:hi] @ _weight_values(s, s["weight"][e], s["weight_scales"][e],
                                                torch.float32).t()
                      for e, lo, hi in s["groups"]])


def _rows_out(s, y):
    """Rounded to the rows' type, zeros for the rows that belong to no expert."""
    y = y.to(s["out"].dtype)
    return y if s["n"] == s["R"] else torch.nn.functional.pad(y, (0, 0, 0, s["R"] - s["n"]))


GELU_A, GELU_B = math.sqrt(2.0 / math.pi), 0.044715


def _act(name, z):
    if name == "silu":
        return z / (1 + torch.exp(-z))
    if name == "gelu":
        return 0.5 * z * (1 + torch.tanh(GELU_A * (z + GELU_B * z * z * z)))
    return z.clamp(min=0) if name == "relu" else z


def _plain_quant(s):
    n = s["used"]
    codes, scales = torch.zeros_like(s["codes"]), torch.zeros_like(s["scales"])
    if n:
        codes[:n], scales[:n] = _quantised_rows(s["rows"][:n], s["form"])
    return {"codes": codes, "scales": scales}


def _plain_gated(s):
    z = _product(s)
    F = s["F"]
    return {"out": _rows_out(s, _act(s["act"], z[:, :F]) * z[:, F:])}


def _plain_linear(s):
    z = _product(s)
    if s["bias"] is not None:
        expert = torch.repeat_interleave(torch.arange(s["local"], device="cuda"),
                                         s["offset"].diff(), output_size=s["n"])
        z = z + s["bias"].float()[expert]
    y = _act(s["act"], z)
    if s["residual"] is not None:
        y = y + s["residual"][:s["n"]].float()
    return {"out": _rows_out(s, y)}


# ---- the framework's calls -------------------------------------------------

def _own_quant(s):
    import moe_token_permute_gb300 as mp
    mp.moe_quant_rows(s["rows"], s["codes"], s["scales"], expert_first_token_offset=s["offset"])
    return {"codes": s["codes"], "scales": s["scales"]}


def _own_gated(s):
    import moe_token_permute_gb300 as mp
    mp.moe_expert_gated_quant(s["codes"], s["scales"], s["weight"], s["weight_scales"],
                              s["offset"], s["out"], activation=s["act"])
    return {"out": s["out"]}


def _own_linear(s):
    import moe_token_permute_gb300 as mp
    mp.moe_expert_linear_quant(s["codes"], s["scales"], s["weight"], s["weight_scales"],
                               s["offset"], s["out"], bias=s["bias"], activation=s["act"],
                               residual=s["residual"])
    return {"out": s["out"]}


def run(state):
    form = {"quant": (_plain_quant, _own_quant), "gated": (_plain_gated, _own_gated),
            "linear": (_plain_linear, _own_linear)}[state["op"]]
    return form[1 if own else 0](state)


# ---- the definition in 64 bits ---------------------------------------------

def _exact_act(name, z):
    if name == "silu":
        return z * torch.sigmoid(z)
    if name == "gelu":
        return z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
    return torch.relu(z) if name == "relu" else z


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "quant":
        return _exact_quant(s)
    if _flops(case, s["n"]) > 8e12:  # over about 20 seconds in 64 bits
        return None
    F = case.get("F")
    inner, outer = s["weight"].shape[2], s["weight"].shape[1]
    column = torch.arange(inner, device="cuda")
    feature = torch.arange(outer, device="cuda")
    if case["op"] == "gated":  # gate and up rows count their blocks apart
        block = feature % F // GROUP + (feature >= F) * _groups(F)
    else:
        block = feature // GROUP
    got = torch.zeros(s["R"], F or outer, dtype=torch.float64, device="cuda")
    for e, lo, hi in s["groups"]:
        x, w = s["codes"][lo:hi].double(), s["weight"][e].double()
        if case["form"] == "fp8":
            x = x * s["scales"][lo:hi][:, column // GROUP].double()
            w = w * s["weight_scales"][e][block][:, column // GROUP].double()
            z = torch.einsum("rk,nk->rn", x, w)
        else:
            z = torch.einsum("rk,nk->rn", x, w)
            z = z * torch.outer(s["scales"][lo:hi, 0].double(), s["weight_scales"][e].double())
        if s["bias"] is not None:
            z = z + s["bias"][e].double()
        y = _exact_act(case["act"], z[:, :F] if F else z)
        y = y * z[:, F:] if F else y
        got[lo:hi] = y if s["residual"] is None else y + s["residual"][lo:hi].double()
    return {"out": got}


def _exact_quant(s):
    """The codes follow from the scales as 32 bits hold them: no 64-bit value."""
    R, H = s["rows"].shape
    x = s["rows"].double().abs()
    scales = torch.zeros(s["scales"].shape, dtype=torch.float64, device="cuda")
    for c in range(scales.shape[1]):
        part = x[:, c * GROUP:(c + 1) * GROUP] if s["form"] == "fp8" else x
        top = part.max(dim=1).values / LARGEST[s["form"]]
        scales[:, c] = torch.where(top == 0, torch.ones_like(top), top)
    scales[s["used"]:] = 0
    return {"codes": None, "scales": scales}
