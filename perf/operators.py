"""Timed cases of the decoder layer's products around the attention: the linear layers (the
attention's output projection, dense and shared-expert MLP layers), the expert router, the
experts' grouped products, and the weighted sum of the experts' rows.

Each case names an operator ("op") and its sizes.  ``run`` computes the operator in its
plain form, elementary torch operations in 32 bits rounded once at the end, or, where
``own`` is true, by the library's entry point (relative_bias_hybrid_gb300.inkattn).
"""
import math

import torch

own = False

BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32
ACTS = ("none", "relu", "gelu", "silu", "swiglu")


# ---------------------------------------------------------------- cases

def listed():
    return [
        # the attention's output projection (64 heads x 128 to a hidden width of 8192) of one
        # token, added to the residual stream: a single user's decode step
        {"name": "linear 1 token", "op": "linear", "T": 1, "K": 8192, "F": 8192, "act": "none", "bias": False,
         "residual": True, "out": "bf16"},
        # the same layer on the verification batch, 32 sequences x 9 tokens
        {"name": "linear 288 tokens", "op": "linear", "T": 288, "K": 8192, "F": 8192, "act": "none", "bias": False,
         "residual": True, "out": "bf16"},
        # the same layer on a prefill of 8192 tokens
        {"name": "linear 8192 tokens", "op": "linear", "T": 8192, "K": 8192, "F": 8192, "act": "none",
         "bias": False, "residual": False, "out": "bf16"},
        # an odd batch through a small dense layer with bias and GELU, output in fp32
        {"name": "linear odd", "op": "linear", "T": 777, "K": 1000, "F": 1021, "act": "gelu", "bias": True,
         "residual": False, "out": "f32"},
        # gate and up products of 256 routed experts, six a token, on the verification batch:
        # every expert sees a few rows, the weights are read for them
        {"name": "experts up 288 tokens", "op": "grouped", "T": 288, "k": 6, "E": 256, "K": 8192, "F": 1024,
         "act": "swiglu", "bias": False, "gather": True, "out": "bf16", "skew": 0.5},
        # the same products in a prefill, 64 experts, hidden width 4096
        {"name": "experts up 8192 tokens", "op": "grouped", "T": 8192, "k": 6, "E": 64, "K": 4096, "F": 2048,
         "act": "swiglu", "bias": False, "gather": True, "out": "bf16", "skew": 0.5},
        # the experts' down products on rows that are already grouped; unevenly loaded experts,
        # some of them without rows
        {"name": "experts down ragged", "op": "grouped", "T": 1001, "k": 4, "E": 60, "K": 2048, "F": 4096,
         "act": "none", "bias": True, "gather": False, "out": "bf16", "skew": 2.0},
        # the router's choice for the verification batch: 256 routed and two shared experts
        {"name": "route 288 tokens", "op": "route", "T": 288, "E": 256, "shared": 2, "k": 6, "score": "sigmoid",
         "ties": False},
        # and for a long prefill, on logits that a bf16 product gave (equal logits happen)
        {"name": "route 32768 tokens", "op": "route", "T": 32768, "E": 256, "shared": 2, "k": 6,
         "score": "sigmoid", "ties": True},
        # the weighted sum of each token's six routed and two shared rows
        {"name": "combine 288 tokens", "op": "combine", "T": 288, "k": 6, "shared": 2, "F": 8192},
        {"name": "combine 8192 tokens", "op": "combine", "T": 8192, "k": 6, "shared": 2, "F": 8192},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["linear", "linear", "grouped", "grouped", "route", "combine"])
    if op == "linear":
        act = rng.choice(ACTS)
        F = _log_int(rng, 8, 8192)
        if act == "swiglu":
            F = max(16, min(4096, F // 16 * 16))
        return {"op": op, "T": _log_int(rng, 1, 8192), "K": 8 * _log_int(rng, 1, 1024), "F": F, "act": act,
                "bias": rng.random() < 0.5, "residual": rng.random() < 0.5,
                "out": "f32" if rng.random() < 0.25 else "bf16"}
    if op == "grouped":
        act = rng.choice(("swiglu", "swiglu", "none", "silu"))
        E = _log_int(rng, 2, 256)
        K = 8 * _log_int(rng, 16, 500)
        F = _log_int(rng, 64, 2048)
        if act == "swiglu":
            F = F // 16 * 16
        k = rng.randint(1, min(8, E))
        T = _log_int(rng, 1, max(1, 16384 // k))
        return {"op": op, "T": T, "k": k, "E": E, "K": K, "F": F, "act": act, "bias": rng.random() < 0.3,
                "gather": act != "none", "out": "f32" if rng.random() < 0.2 else "bf16",
                "skew": round(rng.uniform(0.0, 0.8), 2)}
    if op == "route":
        E = rng.randint(2, 384)
        return {"op": op, "T": _log_int(rng, 1, 32768), "E": E, "shared": rng.randint(0, 2),
                "k": rng.randint(1, min(8, E)), "score": rng.choice(("sigmoid", "softmax")),
                "ties": rng.random() < 0.5}
    return {"op": op, "T": _log_int(rng, 1, 8192), "k": rng.randint(1, 8), "shared": rng.randint(0, 2),
            "F": 8 * _log_int(rng, 8, 1024)}


def work(case):
    T = case["T"]
    if case["op"] == "linear":
        K, F = case["K"], case["F"]
        rows_w = 2 * F if case["act"] == "swiglu" else F
        size = 4 if case["out"] == "f32" else 2
        return {"bytes": 2 * T * K + 2 * rows_w * K + size * T * F + (4 * rows_w if case["bias"] else 0)
                + (2 * T * F if case["residual"] else 0), "flops": 2 * T * K * rows_w}
    if case["op"] == "grouped":
        K, F, E, M = case["K"], case["F"], case["E"], T * case["k"]
        rows_w = 2 * F if case["act"] == "swiglu" else F
        size = 4 if case["out"] == "f32" else 2
        busy = E * (1.0 - (1.0 - case["k"] / E) ** T)     # experts with rows, were the choice even
        read = T if case["gather"] else M
        return {"bytes": int(2 * read * K + 2 * busy * rows_w * K + size * M * F + 4 * (M + E + 1)),
                "flops": 2 * M * K * rows_w}
    if case["op"] == "route":
        E, S, k = case["E"], case["shared"], case["k"]
        return {"bytes": 4 * T * (E + S) + 4 * T * (4 * k + S) + 4 * (E + 1), "flops": T * (E + 4 * (k + S))}
    k, S, F = case["k"], case["shared"], case["F"]
    return {"bytes": 2 * T * (k + S + 1) * F + 4 * T * (2 * k + S), "flops": 2 * T * (k + S) * F}


# ---------------------------------------------------------------- inputs

def _rand(g, shape, std, dtype):
    return torch.randn(shape, generator=g, device="cuda", dtype=dtype).mul_(std)


def prepare(case, seed):
    """Inputs of the case on the GPU, drawn from the seed alone; with ``own`` also what a
    program keeps beside them: the output buffers and the filled params struct."""
    g = torch.Generator(device="cuda")
    g.manual_seed(1_000_003 * seed + 7919)
    s = {"case": case}
    T = case["T"]
    if case["op"] == "linear":
        K, F = case["K"], case["F"]
        rows_w = 2 * F if case["act"] == "swiglu" else F
        s["x"] = _rand(g, (T, K), 1.0, BF16)
        s["w"] = _rand(g, (rows_w, K), K ** -0.5, BF16)
        s["bias"] = _rand(g, (rows_w,), 0.5, F32) if case["bias"] else None
        s["residual"] = _rand(g, (T, F), 1.0, BF16) if case["residual"] else None
        if own:
            from relative_bias_hybrid_gb300 import inkattn as ia
            s["out"] = torch.empty((T, F), dtype=F32 if case["out"] == "f32" else BF16, device="cuda")
            s["params"] = ia.linear_params(x=s["x"], w=s["w"], bias=s["bias"], residual=s["residual"],
                                           out=s["out"], act=case["act"])
    elif case["op"] == "grouped":
        E, k, K, F = case["E"], case["k"], case["K"], case["F"]
        M = T * k
        rows_w = 2 * F if case["act"] == "swiglu" else F
        # each token takes its k best of a random score; some experts are liked more than others
        score = torch.randn((T, E), generator=g, device="cuda")
        score += case["skew"] * torch.randn((E,), generator=g, device="cuda")
        ids = score.topk(k, dim=1).indices.reshape(-1)
        counts = torch.bincount(ids, minlength=E)
        s["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(I32)
        s["most"] = int(counts.max())
        order = torch.sort(ids, stable=True).indices
        s["row_token"] = (order // k).to(I32) if case["gather"] else None
        s["x"] = _rand(g, (T if case["gather"] else M, K), 1.0, BF16)
        s["w"] = _rand(g, (E, rows_w, K), K ** -0.5, BF16)
        s["bias"] = _rand(g, (E, rows_w), 0.5, F32) if case["bias"] else None
        if own:
            from relative_bias_hybrid_gb300 import inkattn as ia
            s["out"] = torch.empty((M, F), dtype=F32 if case["out"] == "f32" else BF16, device="cuda")
            s["params"] = ia.grouped_linear_params(x=s["x"], w=s["w"], expert_offsets=s["offsets"],
                                                   row_token=s["row_token"], bias=s["bias"], out=s["out"],
                                                   act=case["act"])
    elif case["op"] == "route":
        E, S, k = case["E"], case["shared"], case["k"]
        logits = _rand(g, (T, E + S), 1.5, F32)
        s["logits"] = logits.to(BF16).float() if case["ties"] else logits
        if own:
            from relative_bias_hybrid_gb300 import inkattn as ia
            s["out"] = {"topk_ids": torch.empty((T, k), dtype=I32, device="cuda"),
                        "weights": torch.empty((T, k + S), dtype=F32, device="cuda"),
                        "expert_offsets": torch.empty(E + 1, dtype=I32, device="cuda"),
                        "row_token": torch.empty(T * k, dtype=I32, device="cuda"),
                        "token_rows": torch.empty((T, k), dtype=I32, device="cuda")}
            s["params"] = ia.route_params(logits=s["logits"], n_shared=S, score=case["score"], scale=1.0,
                                          **s["out"])
            s["workspace"] = torch.empty(ia.inkattn_route_workspace_bytes(s["params"]), dtype=torch.uint8,
                                         device="cuda")
    else:
        k, S, F = case["k"], case["shared"], case["F"]
        M = T * k
        s["y"] = _rand(g, (M, F), 1.0, BF16)
        s["shared"] = _rand(g, (S, T, F), 1.0, BF16) if S else None
        weights = torch.rand((T, k + S), generator=g, device="cuda") + 0.05
        s["weights"] = weights / weights.sum(1, keepdim=True)
        s["token_rows"] = torch.randperm(M, generator=g, device="cuda").to(I32).reshape(T, k)
        if own:
            from relative_bias_hybrid_gb300 import inkattn as ia
            s["out"] = torch.empty((T, F), dtype=BF16, device="cuda")
            s["params"] = ia.expert_combine_params(y=s["y"], shared=s["shared"], weights=s["weights"],
                                                   token_rows=s["token_rows"], out=s["out"])
    return s


# ---------------------------------------------------------------- the operators

def run(s):
    case = s["case"]
    if own:
        from relative_bias_hybrid_gb300 import inkattn as ia
        if case["op"] == "linear":
            ia.inkattn_linear(s["params"])
        elif case["op"] == "grouped":
            ia.inkattn_grouped_linear(s["params"])
        elif case["op"] == "route":
            ia.inkattn_route(s["params"], s["workspace"])
        else:
            ia.inkattn_expert_combine(s["params"])
        return s["out"]
    return {"linear": _linear, "grouped": _grouped, "route": _route, "combine": _combine}[case["op"]](s)


def _activate(y, act):
    if act == "relu":
        return torch.where(y > 0, y, torch.zeros_like(y))
    if act == "gelu":
        return 0.5 * y * (1.0 + torch.erf(y * 2.0 ** -0.5))
    if act == "silu":
        return y / (1.0 + torch.exp(-y))
    if act == "swiglu":
        F = y.shape[-1] // 2
        gate, up = y[..., :F], y[..., F:]
        return gate / (1.0 + torch.exp(-gate)) * up
    return y


def _out_dtype(case):
    return F32 if case["out"] == "f32" else BF16


def _linear(s):
    case = s["case"]
    y = s["x"].float() @ s["w"].float().t()
    if s["bias"] is not None:
        y = y + s["bias"]
    y = _activate(y, case["act"])
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return y.to(_out_dtype(case))


def _grouped(s):
    """The rows of each expert side by side in one padded batch of products."""
    case = s["case"]
    M, E, K = case["T"] * case["k"], case["E"], case["K"]
    row = torch.arange(M, device="cuda")
    starts = s["offsets"].long()
    expert = torch.searchsorted(starts[1:], row, right=True)
    place = row - starts[expert]
    x = s["x"] if s["row_token"] is None else s["x"][s["row_token"].long()]
    padded = torch.zeros((E, s["most"], K), device="cuda")
    padded[expert, place] = x.float()
    y = torch.bmm(padded, s["w"].float().transpose(1, 2))[expert, place]
    if s["bias"] is not None:
        y = y + s["bias"][expert]
    return _activate(y, case["act"]).to(_out_dtype(case))


def _scores(logits, score):
    """Positive scores whose ratios are those of the weights."""
    if score == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-logits))
    return torch.exp(logits - logits.amax(1, keepdim=True))


def _route(s):
    case = s["case"]
    T, E, S, k = case["T"], case["E"], case["shared"], case["k"]
    logits = s["logits"]
    best = torch.sort(logits[:, :E], dim=1, descending=True, stable=True)
    ids = best.indices[:, :k]
    chosen = _scores(torch.cat([best.values[:, :k], logits[:, E:]], 1), case["score"])
    counts = torch.bincount(ids.reshape(-1), minlength=E)
    order = torch.sort(ids.reshape(-1), stable=True).indices
    rows = torch.empty_like(order)
    rows[order] = torch.arange(T * k, device="cuda")
    return {"topk_ids": ids.to(I32), "weights": chosen / chosen.sum(1, keepdim=True),
            "expert_offsets": torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(I32),
            "row_token": (order // k).to(I32), "token_rows": rows.reshape(T, k).to(I32)}


def _combine(s):
    k = s["case"]["k"]
    w = s["weights"]
    out = (s["y"][s["token_rows"].long()].float() * w[:, :k, None]).sum(1)
    if s["shared"] is not None:
        out = out + (s["shared"].float() * w[:, k:].t()[:, :, None]).sum(0)
    return out.to(BF16)


# ---------------------------------------------------------------- in 64 bits

def exact(case, seed):
    """What run returns for these inputs, from the definitions in 64 bits."""
    s = prepare(case, seed)

    def curve(z, act):
        if act == "swiglu":
            a, b = torch.chunk(z, 2, dim=-1)
            return a * torch.sigmoid(a) * b
        return {"none": lambda v: v, "relu": lambda v: v.clamp(min=0.0), "silu": lambda v: v * torch.sigmoid(v),
                "gelu": lambda v: v * 0.5 * torch.special.erfc(-v / math.sqrt(2.0))}[act](z)

    if case["op"] == "linear":
        z = torch.einsum("tk,fk->tf", s["x"].double(), s["w"].double())
        z = curve(z if s["bias"] is None else z + s["bias"].double(), case["act"])
        return z if s["residual"] is None else z + s["residual"].double()
    if case["op"] == "grouped":
        ends = s["offsets"].tolist()
        parts = []
        for e in range(case["E"]):
            rows = slice(ends[e], ends[e + 1])
            x = s["x"][rows] if s["row_token"] is None else s["x"][s["row_token"][rows].long()]
            z = x.double() @ s["w"][e].double().t()
            parts.append(curve(z if s["bias"] is None else z + s["bias"][e].double(), case["act"]))
        return torch.cat(parts)
    if case["op"] == "route":
        E, k = case["E"], case["k"]
        logits = s["logits"].double()
        top = torch.sort(logits[:, :E], dim=1, descending=True, stable=True).values[:, :k]
        z = torch.cat([top, logits[:, E:]], 1)
        p = torch.sigmoid(z) if case["score"] == "sigmoid" else torch.softmax(z, 1)
        return {"topk_ids": None, "weights": p / p.sum(1, keepdim=True), "expert_offsets": None,
                "row_token": None, "token_rows": None}
    total = torch.zeros((case["T"], case["F"]), dtype=torch.float64, device="cuda")
    for j in range(case["k"]):
        total += s["weights"][:, j, None].double() * s["y"][s["token_rows"][:, j].long()].double()
    for j in range(case["shared"]):
        total += s["weights"][:, case["k"] + j, None].double() * s["shared"][j].double()
    return total
