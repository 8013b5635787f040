"""Timed cases of a speculative decode step over a 4-bit KV cache: the attention prologue that writes
such a cache, the attention that reads it (decode and prefill), the probabilities of rows of
logits, the verification of drafted tokens, and the conv states' return to the accepted tokens.

Each case names an operator ("op") and its sizes.  ``run`` computes the operator in its plain
form, elementary torch operations, or, where ``own`` is true, by the library's entry points
(relative_bias_hybrid_gb300.inkattn).

The 4-bit cache: a row of 128 values is four groups of 32.  A group's scale s is the smallest
8-bit float (5 exponent and 3 mantissa bits, the upper byte of an fp16 without its sign) with
7 s >= max|x|, at most 896; its values are n s with n = x / s rounded to nearest, ties to even, and at
most 7 in magnitude.  A 32-bit word holds eight values as n + 8: value 2 i in bits 4 i and value
2 i + 1 in bits 16 + 4 i.
"""
import math
import random

import torch

own = False

BF16, F32, F64, I32 = torch.bfloat16, torch.float32, torch.float64, torch.int32
D, BLOCK, D_R, EPS = 128, 64, 32, 1e-6
UNIT = 2.0 ** 43          # steps of the sampled weights in one


# ---------------------------------------------------------------- cases

def listed():
    return [
        # the prologue of one layer on the verification batch, 32 sequences x 9 tokens: norms,
        # convs and 4-bit cache rows of a decode step
        {"name": "append 288 tokens", "op": "append", "B": 32, "q": 9, "Hq": 64, "Hkv": 8, "ragged": False},
        # the same on a prefill of uneven sequences, some of them without new tokens
        {"name": "append ragged", "op": "append", "B": 13, "q": 1021, "Hq": 64, "Hkv": 8, "ragged": True},
        # a single user's decode step, one token over an 8K context on a full layer
        {"name": "decode 1 token", "op": "attend", "mode": "decode", "B": 1, "q": 1, "kv": 8192, "Hq": 64, "Hkv": 8,
         "ext": 1024, "window": 0, "base": 8192.0, "ragged": False},
        # the verification batch on a full layer: 32 sequences x 9 tokens over 32768 keys each
        {"name": "decode 288 tokens", "op": "attend", "mode": "decode", "B": 32, "q": 9, "kv": 32768, "Hq": 64,
         "Hkv": 8, "ext": 1024, "window": 0, "base": 8192.0, "ragged": False},
        # a sliding-window layer, sequences of all lengths, odd head groups, drafts of odd length
        {"name": "decode ragged window", "op": "attend", "mode": "decode", "B": 21, "q": 5, "kv": 9001, "Hq": 24,
         "Hkv": 4, "ext": 500, "window": 2048, "base": 0.0, "ragged": True},
        # the prefill of a prompt behind a cached prefix on a sliding-window layer
        {"name": "prefill 4096 tokens", "op": "attend", "mode": "prefill", "B": 1, "q": 4096, "kv": 5003, "Hq": 64,
         "Hkv": 8, "ext": 512, "window": 4096, "base": 0.0, "ragged": False},
        # the probabilities of one sequence's 9 rows of logits, as a bf16 head gives them
        {"name": "probs 9 rows", "op": "probs", "T": 9, "V": 50001, "in": "bf16", "temp": "one"},
        # and of the verification batch, each request with its own temperature, some greedy
        {"name": "probs 288 rows", "op": "probs", "T": 288, "V": 131072, "in": "f32", "temp": "mixed"},
        # eight drafts of one user, drawn from a drafter's distribution
        {"name": "verify 1 sequence", "op": "verify", "B": 1, "drafts": 8, "V": 131072, "drafter": True,
         "ragged": False},
        # the verification batch, some sequences with fewer drafts, an odd vocabulary
        {"name": "verify 32 sequences", "op": "verify", "B": 32, "drafts": 8, "V": 200019, "drafter": True,
         "ragged": True},
        # the states of a layer's four convs (K, V, attention output, MLP output) of one user ...
        {"name": "rollback 1 sequence", "op": "rollback", "B": 1, "q": 9, "Hkv": 8, "Hq": 64, "ragged": False},
        # ... and of a large batch
        {"name": "rollback 512 sequences", "op": "rollback", "B": 512, "q": 9, "Hkv": 8, "Hq": 64, "ragged": True},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["append", "append", "decode", "decode", "decode", "prefill", "probs", "verify", "rollback"])
    Hkv = rng.choice((1, 2, 4, 8))
    g = rng.choice((1, 2, 3, 4, 6, 8))
    if op == "append":
        B = _log_int(rng, 1, 64)
        return {"op": op, "B": B, "q": _log_int(rng, 1, max(1, 8192 // B)), "Hq": Hkv * g, "Hkv": Hkv,
                "ragged": rng.random() < 0.5}
    if op == "decode":
        q = rng.randint(1, min(9, 128 // g))
        window = rng.choice((0, 0, _log_int(rng, 64, 8192)))
        return {"op": "attend", "mode": op, "B": _log_int(rng, 1, 32), "q": q, "kv": _log_int(rng, q + 1, 32768),
                "Hq": Hkv * g, "Hkv": Hkv, "ext": rng.choice((0, _log_int(rng, 16, 1024), 1024)), "window": window,
                "base": 0.0 if window else rng.choice((0.0, 8192.0)), "ragged": rng.random() < 0.5}
    if op == "prefill":
        q = _log_int(rng, 17, 3000)
        window = rng.choice((0, _log_int(rng, 128, 4096)))
        return {"op": "attend", "mode": op, "B": rng.randint(1, 3), "q": q, "kv": q + rng.randint(0, 1000),
                "Hq": Hkv * g, "Hkv": Hkv, "ext": rng.choice((0, _log_int(rng, 16, 1024), 512)), "window": window,
                "base": 0.0 if window else rng.choice((0.0, 512.0)), "ragged": rng.random() < 0.5}
    if op == "probs":
        return {"op": op, "T": _log_int(rng, 1, 288), "V": _log_int(rng, 100, 131072), "in": rng.choice(("f32", "bf16")),
                "temp": rng.choice(("one", "mixed"))}
    if op == "verify":
        return {"op": op, "B": _log_int(rng, 1, 32), "drafts": rng.randint(0, 8), "V": _log_int(rng, 50, 200019),
                "drafter": rng.random() < 0.7, "ragged": rng.random() < 0.5}
    return {"op": op, "B": _log_int(rng, 1, 512), "q": rng.randint(1, 9), "Hkv": Hkv, "Hq": Hkv * g,
            "ragged": rng.random() < 0.5}


def _lens(case):
    """New tokens and cached tokens of each sequence: fixed by the case."""
    rng = random.Random("%s %s %s" % (case["op"], case["B"], case["q"]))
    B, q = case["B"], case["q"]
    if case["op"] == "append":
        new = [rng.randint(0, q) if case["ragged"] else q for _ in range(B)]
        new[rng.randrange(B)] = q
        return new, [rng.randint(0, 200) for _ in range(B)]
    if case["op"] == "rollback":
        return [rng.randint(0, q) if case["ragged"] else q for _ in range(B)], [0] * B
    total = [_log_int(rng, 1, case["kv"]) if case["ragged"] else case["kv"] for _ in range(B)]
    total[rng.randrange(B)] = case["kv"]
    new = [min(t, rng.randint(1, q) if case["ragged"] else q) for t in total]
    return new, [t - n for t, n in zip(total, new)]


def _spans(case, new, total):
    """Pairs of a query and a key that it sees, and the keys that some query of the sequence sees."""
    w = case["window"]
    pairs = keys = 0
    for n, t in zip(new, total):
        lo = max(0, t - n - w + 1) if w else 0
        keys += t - lo if n else 0
        if w:
            full = max(0, min(n, t - w + 1))          # queries whose window is whole
            rest = n - full
            first = t - n + 1
            pairs += full * w + sum((first, first + rest - 1)) * rest // 2
        else:
            pairs += n * (2 * t - n + 1) // 2
    return pairs, keys


def work(case):
    op = case["op"]
    if op == "probs":
        return {"bytes": case["T"] * case["V"] * ((2 if case["in"] == "bf16" else 4) + 4), "flops": 4 * case["T"] * case["V"]}
    if op == "verify":
        rows = 2 if case["drafter"] and case["drafts"] else 1
        return {"bytes": 4 * case["B"] * case["V"] * rows + 16 * case["B"] * (case["drafts"] + 1),
                "flops": 4 * case["B"] * case["V"]}
    new, cached = _lens(case)
    N, B, Hq, Hkv = sum(new), case["B"], case["Hq"], case["Hkv"]
    C = Hkv * D
    if op == "rollback":
        widths = 2 * C + 2 * Hq * D
        return {"bytes": 2 * 2 * 3 * B * widths + 16 * B, "flops": 0}
    if op == "append":
        return {"bytes": 2 * 2 * N * Hq * D + 2 * (2 * N * C) + 2 * N * Hkv * 68 + 2 * 2 * (2 * 3 * B * C) + 4 * N,
                "flops": 8 * N * 2 * C + 4 * N * (Hq + Hkv) * D}
    total = [n + p for n, p in zip(new, cached)]
    pairs, keys = _spans(case, new, total)
    ext = case["ext"]
    return {"bytes": 2 * keys * Hkv * 68 + 4 * N * Hq * D + (2 * N * Hq * D_R + 4 * Hq * ext * D_R if ext else 0),
            "flops": 4 * pairs * Hq * D}


# ---------------------------------------------------------------- the 4-bit cache in plain torch

def _quantise(x):
    """Groups of 32 along the last axis: whole numbers n as float64 and their scales."""
    g = x.double().unflatten(-1, (-1, 32))
    t = g.abs().amax(-1) / 7.0
    step = torch.exp2((torch.frexp(t).exponent - 1).clamp(min=-14).double() - 3.0)
    s = (torch.ceil(t / step) * step).clamp(max=896.0)
    n = torch.round(g / torch.where(s > 0, s, torch.ones_like(s))[..., None]).clamp(-7, 7)
    return n, s


def _values(n, s):
    """n s, exact in bf16."""
    return (n * s[..., None]).flatten(-2).to(BF16)


def _pack(n):
    """Codes of [..., 4, 32] whole numbers as bytes [..., 64]."""
    u = (n + 8.0).to(torch.int64).reshape(*n.shape[:-2], 16, 4, 2)
    at = 4 * torch.arange(4, device=n.device)[:, None] + 16 * torch.arange(2, device=n.device)
    word = (u << at).sum((-1, -2))
    return torch.where(word >= 2 ** 31, word - 2 ** 32, word).to(I32).view(torch.uint8)


def _unpack(codes, scales):
    """float32 values of code bytes [..., 64] with scale bytes [..., 4]."""
    at = (4 * torch.arange(4, device="cuda", dtype=I32)[:, None] + 16 * torch.arange(2, device="cuda", dtype=I32)).reshape(8)
    n = ((codes.view(I32)[..., None] >> at) & 15) - 8
    s = (scales.to(torch.int16) << 7).view(torch.float16).float()
    return (n.reshape(*codes.shape[:-1], 4, 32).float() * s[..., None]).flatten(-2)


def _scale_bytes(s):
    return ((s.to(torch.float16).view(torch.int16) >> 7) & 255).to(torch.uint8)


# ---------------------------------------------------------------- inputs

def _rand(g, shape, std=1.0, dtype=F32):
    return torch.randn(shape, generator=g, device="cuda", dtype=F32).mul_(std).to(dtype)


def _ints(v, dtype=I32):
    return torch.tensor(v, dtype=dtype, device="cuda")


def _layout(s, case):
    new, cached = _lens(case)
    total = [n + p for n, p in zip(new, cached)]
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    s["new"], s["cached"], s["total"], s["N"] = new, cached, total, cu[-1]
    s["cu"], s["kv_len"] = _ints(cu), _ints(total)
    s["slot"] = torch.arange(case["B"], dtype=I32, device="cuda")


def _pages(s, g):
    """A block table of blocks in random order, -1 behind each sequence's."""
    need = [-(-t // BLOCK) for t in s["total"]]
    s["blocks"] = max(1, sum(need))
    perm = torch.randperm(s["blocks"], generator=g, device="cuda").to(I32)
    j = torch.arange(max(1, max(need)), device="cuda")
    first = torch.cumsum(_ints(need, torch.int64), 0) - _ints(need, torch.int64)
    at = (first[:, None] + j).clamp(max=s["blocks"] - 1)
    s["table"] = torch.where(j < _ints(need, torch.int64)[:, None], perm[at], torch.full_like(perm[at], -1)).contiguous()


def _positions(s):
    """Sequence and place within it of each new token."""
    cu = s["cu"].long()
    row = torch.arange(s["N"], device="cuda")
    seq = torch.searchsorted(cu[1:], row, right=True)
    return seq, row - cu[seq]


def prepare(case, seed):
    """Inputs of the case on the GPU, drawn from the seed alone; with ``own`` also the output buffers,
    the workspace and the filled params struct that a program keeps beside them."""
    g = torch.Generator(device="cuda")
    g.manual_seed(1_000_003 * seed + 7907)
    s = {"case": case}
    {"append": _prepare_append, "attend": _prepare_attend, "probs": _prepare_probs, "verify": _prepare_verify,
     "rollback": _prepare_rollback}[case["op"]](s, case, g)
    return s


def _prepare_append(s, case, g):
    B, Hq, Hkv = case["B"], case["Hq"], case["Hkv"]
    C = Hkv * D
    _layout(s, case)
    _pages(s, g)
    N = s["N"]
    s["q"], s["k"], s["v"] = _rand(g, (N, Hq, D), 1.0, BF16), _rand(g, (N, C), 1.0, BF16), _rand(g, (N, C), 1.0, BF16)
    s["wk"], s["wv"] = _rand(g, (C, 4), 0.5), _rand(g, (C, 4), 0.5)
    s["gq"], s["gk"] = 1.0 + _rand(g, (D,), 0.1), 1.0 + _rand(g, (D,), 0.1)
    s["state_k"], s["state_v"] = _rand(g, (B, 3, C), 1.0, BF16), _rand(g, (B, 3, C), 1.0, BF16)
    seq, place = _positions(s)
    pos = place + _ints(s["cached"], torch.int64)[seq]
    s["slots"] = s["table"][seq, pos // BLOCK] * BLOCK + (pos % BLOCK).to(I32)
    if own:
        from relative_bias_hybrid_gb300 import inkattn as ia
        s["now_k"], s["now_v"], s["q_out"] = torch.empty_like(s["state_k"]), torch.empty_like(s["state_v"]), torch.empty_like(s["q"])
        s["cache"] = torch.zeros((2, s["blocks"], Hkv, BLOCK, D // 2), dtype=torch.uint8, device="cuda")
        s["scale"] = torch.zeros((2, s["blocks"], Hkv, BLOCK, D // 32), dtype=torch.uint8, device="cuda")
        s["params"] = ia.prologue_params(
            q=s["q"], k=s["k"], v=s["v"], conv_w_k=s["wk"], conv_w_v=s["wv"], q_norm_w=s["gq"], k_norm_w=s["gk"],
            cu_seqlens_q=s["cu"], state_slot=s["slot"], slot_mapping=s["slots"], conv_state_k=s["now_k"],
            conv_state_v=s["now_v"], q_out=s["q_out"], k_cache=s["cache"][0], v_cache=s["cache"][1],
            k_scale=s["scale"][0], v_scale=s["scale"][1], max_seqlen_q=max(s["new"]), eps=EPS)


def _prepare_attend(s, case, g):
    Hq, Hkv, ext = case["Hq"], case["Hkv"], case["ext"]
    _layout(s, case)
    _pages(s, g)
    N = s["N"]
    s["q"] = _rand(g, (N, Hq, D), 1.0, BF16)
    s["r"] = _rand(g, (N, Hq, D_R), 1.0, BF16)
    s["P"] = _rand(g, (Hq, max(1, ext), D_R), 0.02)
    for name in ("k", "v"):
        # values of about unit size, as a normalised key has them
        n, sc = _quantise(_rand(g, (s["blocks"], Hkv, BLOCK, D)))
        s[name] = _pack(n)
        s[name + "_scale"] = _scale_bytes(sc)
        del n, sc
    if own:
        from relative_bias_hybrid_gb300 import inkattn as ia
        s["out"] = torch.empty((N, Hq, D), dtype=BF16, device="cuda")
        s["params"] = p = ia.attn_params(
            q=s["q"], k_cache=s["k"], v_cache=s["v"], k_scale=s["k_scale"], v_scale=s["v_scale"], cu_seqlens_q=s["cu"],
            seqlen_k=s["kv_len"], block_table=s["table"], out=s["out"], max_seqlen_q=max(s["new"]),
            max_seqlen_k=max(s["total"]), r=s["r"], P=s["P"], rel_extent=ext, window=case["window"],
            log_scale_base=case["base"])
        if case["mode"] == "decode":
            sms = torch.cuda.get_device_properties(0).multi_processor_count
            s["splits"] = ia.inkattn_decode_num_splits(p, sms)
            size = ia.inkattn_decode_workspace_bytes(p, s["splits"])
        else:
            size = ia.inkattn_prefill_workspace_bytes(p)
        s["workspace"] = torch.empty(size, dtype=torch.uint8, device="cuda") if size else None


def _prepare_probs(s, case, g):
    T, V = case["T"], case["V"]
    s["logits"] = _rand(g, (T, V), 3.0, BF16 if case["in"] == "bf16" else F32)
    s["temperature"] = None
    if case["temp"] == "mixed":
        t = 0.3 + 1.2 * torch.rand((T,), generator=g, device="cuda")
        s["temperature"] = torch.where(torch.rand((T,), generator=g, device="cuda") < 0.2, torch.zeros_like(t), t)
    if own:
        from relative_bias_hybrid_gb300 import inkattn as ia
        s["out"] = torch.empty((T, V), dtype=F32, device="cuda")
        s["params"] = ia.token_probs_params(logits=s["logits"], probs=s["out"], temperature=s["temperature"])


def _prepare_verify(s, case, g):
    B, V = case["B"], case["V"]
    rng = random.Random("verify %s %s" % (B, case["drafts"]))
    n = [1 + (rng.randint(0, case["drafts"]) if case["ragged"] else case["drafts"]) for _ in range(B)]
    cu = [0]
    for x in n:
        cu.append(cu[-1] + x)
    N = s["N"] = cu[-1]
    s["cu"], s["most"] = _ints(cu), max(n)
    logits = _rand(g, (N, V), 3.0)
    s["p"] = torch.softmax(logits, 1)
    q = torch.softmax(logits + _rand(g, (N, V), 0.7), 1)
    drawn = torch.multinomial(q, 1, generator=g)[:, 0]
    del logits
    s["q"] = q if case["drafter"] else None
    # the step's input tokens: a sequence's last token, then its drafts, each drawn from the row before
    s["ids"] = torch.cat([torch.randint(0, V, (1,), generator=g, device="cuda"), drawn[:-1]]).to(I32)
    s["u"] = torch.rand((N,), generator=g, device="cuda")
    s["u_sample"] = torch.rand((B,), generator=g, device="cuda")
    if own:
        from relative_bias_hybrid_gb300 import inkattn as ia
        s["out"] = {"n_new": torch.empty(B, dtype=I32, device="cuda"), "tokens": torch.empty(N, dtype=I32, device="cuda")}
        s["params"] = ia.verify_drafts_params(target_p=s["p"], draft_p=s["q"], token_ids=s["ids"], cu_seqlens_q=s["cu"],
                                              u_accept=s["u"], u_sample=s["u_sample"], n_new=s["out"]["n_new"],
                                              out_tokens=s["out"]["tokens"])


def _prepare_rollback(s, case, g):
    B, C = case["B"], case["Hkv"] * D
    _layout(s, case)
    widths = (C, C, case["Hq"] * D, case["Hq"] * D)
    s["x"] = [_rand(g, (s["N"], w), 1.0, BF16) for w in widths]
    s["before"] = [_rand(g, (B, 3, w), 1.0, BF16) for w in widths]
    most = _ints(s["new"], torch.int64)
    s["keep"] = (torch.rand((B,), generator=g, device="cuda") * (most + 1)).long().clamp(max=most).to(I32)
    if own:
        from relative_bias_hybrid_gb300 import inkattn as ia
        s["after"] = [torch.empty_like(t) for t in s["before"]]
        s["params"] = ia.conv_rollback_params(x=s["x"], state_before=s["before"], state_after=s["after"], n_keep=s["keep"],
                                              cu_seqlens_q=s["cu"], state_slot=s["slot"])


# ---------------------------------------------------------------- the operators

def run(s):
    case = s["case"]
    if own:
        return _own(s, case)
    return {"append": _append, "attend": _attend, "probs": _probs, "verify": _verify, "rollback": _rollback}[case["op"]](s)


def _own(s, case):
    from relative_bias_hybrid_gb300 import inkattn as ia
    op = case["op"]
    if op == "append":
        s["now_k"].copy_(s["state_k"])           # the states before the step are kept for a rollback
        s["now_v"].copy_(s["state_v"])
        ia.inkattn_prologue(s["params"])
        blk, off = s["slots"].long() // BLOCK, s["slots"].long() % BLOCK
        rows = _unpack(s["cache"][:, blk, :, off].contiguous(), s["scale"][:, blk, :, off]).to(BF16)     # [N][2][Hkv][128]
        return {"q_out": s["q_out"], "k": rows[:, 0], "v": rows[:, 1], "state_k": s["now_k"], "state_v": s["now_v"]}
    if op == "attend":
        if case["mode"] == "decode":
            ia.inkattn_decode(s["params"], s["splits"], s["workspace"])
            ia.inkattn_combine(s["params"], s["splits"], s["workspace"])
        else:
            ia.inkattn_prefill_i4(s["params"], s["workspace"])
        return s["out"]
    if op == "probs":
        ia.inkattn_token_probs(s["params"])
        return s["out"]
    if op == "verify":
        ia.inkattn_verify_drafts(s["params"])
        return s["out"]
    ia.inkattn_conv_rollback(s["params"])
    return s["after"]


def _history(s, x, state, seq, at):
    """Rows at places `at` (from -3 on) of sequences `seq`: new rows, or the state's in front of them."""
    both = torch.cat([state.flatten(0, 1), x])
    return both[torch.where(at >= 0, 3 * state.shape[0] + s["cu"].long()[seq] + at, 3 * seq + at + 3)]


def _last_three(s, x, state, count):
    """The state behind the first count[b] new rows of each sequence."""
    B = state.shape[0]
    seq = torch.arange(B, device="cuda")[:, None].expand(B, 3)
    return _history(s, x, state, seq, count.long()[:, None] - 3 + torch.arange(3, device="cuda"))


def _append(s):
    """In 64 bits: a rounding next to a border would move a 4-bit value by a whole step."""
    case = s["case"]
    seq, place = _positions(s)
    at = place[:, None] + torch.arange(-3, 1, device="cuda")
    seq4 = seq[:, None].expand_as(at)
    k = (_history(s, s["k"], s["state_k"], seq4, at).double() * s["wk"].double().t()).sum(1).to(BF16)
    v = (_history(s, s["v"], s["state_v"], seq4, at).double() * s["wv"].double().t()).sum(1).to(BF16)
    k = k.unflatten(1, (case["Hkv"], D)).double()
    k = (k / torch.sqrt((k * k).mean(-1, keepdim=True) + EPS) * s["gk"].double()).to(BF16)
    q = s["q"].float()
    q = (q / torch.sqrt((q * q).mean(-1, keepdim=True) + EPS) * s["gq"]).to(BF16)
    count = s["cu"][1:] - s["cu"][:-1]
    return {"q_out": q, "k": _values(*_quantise(k)), "v": _values(*_quantise(v.unflatten(1, (case["Hkv"], D)))),
            "state_k": _last_three(s, s["k"], s["state_k"], count),
            "state_v": _last_three(s, s["v"], s["state_v"], count)}


def _attend(s):
    """All sequences side by side, padded to the longest."""
    case = s["case"]
    B, Hq, Hkv = case["B"], case["Hq"], case["Hkv"]
    g, nq, nk = Hq // Hkv, max(s["new"]), s["table"].shape[1] * BLOCK
    seq, place = _positions(s)
    table = s["table"].clamp(min=0).long()
    k = _unpack(s["k"][table], s["k_scale"][table]).permute(0, 2, 4, 1, 3).reshape(B, Hkv, D, nk)
    qp = torch.zeros((B, nq, Hq, D), device="cuda")
    qp[seq, place] = s["q"].float()
    logit = torch.matmul(qp.view(B, nq, Hkv, g, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, g * nq, D), k).mul_(D ** -0.5)
    del k
    logit = logit.view(B, Hq, nq, nk)
    total = s["kv_len"].long()
    count = (s["cu"][1:] - s["cu"][:-1]).long()
    pos = (total - count)[:, None] + torch.arange(nq, device="cuda")
    away = pos[:, :, None] - torch.arange(nk, device="cuda")                         # [B][nq][nk]
    if case["ext"]:
        r = torch.zeros((B, nq, Hq, D_R), device="cuda")
        r[seq, place] = s["r"].float()
        bias = torch.matmul(r.transpose(1, 2), s["P"].transpose(1, 2))               # [B][Hq][nq][ext]
        at = away.clamp(0, case["ext"] - 1)[:, None].expand(B, Hq, nq, nk)
        logit += torch.gather(bias, 3, at) * ((away >= 0) & (away < case["ext"]))[:, None]
    if case["base"] > 1:
        lam = (torch.log(total.double()) / math.log(case["base"])).clamp(min=1.0).float()
        logit *= lam[:, None, None, None]
    seen = (away >= 0) & (torch.arange(nq, device="cuda")[:, None] < count[:, None, None])
    if case["window"]:
        seen &= away < case["window"]
    logit.masked_fill_(~seen[:, None], float("-inf"))
    m = logit.amax(-1, keepdim=True)
    w = torch.exp(logit - torch.where(m == float("-inf"), torch.zeros_like(m), m))
    del logit
    w /= w.sum(-1, keepdim=True).clamp(min=1e-30)
    v = _unpack(s["v"][table], s["v_scale"][table]).permute(0, 2, 1, 3, 4).reshape(B, Hkv, nk, D)
    out = torch.matmul(w.view(B, Hkv, g * nq, nk), v).view(B, Hq, nq, D)
    return out.transpose(1, 2)[seq, place].to(BF16)


def _probs(s):
    l = s["logits"].float()
    m = l.amax(1, keepdim=True)
    if s["temperature"] is None:
        e = torch.exp(l - m)
        return e / e.sum(1, keepdim=True)
    t = s["temperature"][:, None]
    e = torch.exp((l - m) / torch.where(t > 0, t, torch.ones_like(t)))
    place = torch.arange(l.shape[1], device="cuda")
    best = torch.where(l == m, place, l.shape[1]).amin(1, keepdim=True)
    return torch.where(t > 0, e / e.sum(1, keepdim=True), (place == best).float())


def _verify(s):
    """Weights as whole steps of 2^-43, so that sums are exact and no border depends on their order."""
    p, cu = s["p"], s["cu"].long()
    N, V = p.shape
    B = cu.numel() - 1
    drafts = cu[1:] - cu[:-1] - 1
    row = torch.arange(N, device="cuda")
    draft = s["ids"].long()[(row + 1).clamp(max=N - 1)]
    pd = p[row, draft]
    ok = s["u"] < pd if s["q"] is None else s["u"] * s["q"][row, draft] < pd
    i = torch.arange(s["most"], device="cuda")
    at = (cu[:-1, None] + i).clamp(max=N - 1)
    good = ok[at] & (i < drafts[:, None])
    accepted = torch.cumprod(good.long(), 1).sum(1)
    last = cu[:-1] + accepted
    rejected = accepted < drafts
    if s["q"] is None:
        w = torch.where(rejected[:, None] & (torch.arange(V, device="cuda") == draft[last][:, None]), 0.0, p[last])
    else:
        w = torch.where(rejected[:, None], p[last] - s["q"][last], p[last])
    n = torch.round(w.clamp(0.0, 1.0).double() * UNIT).long()
    empty = n.sum(1) == 0
    n = torch.where(empty[:, None], torch.round(p[last].clamp(0.0, 1.0).double() * UNIT).long(), n)
    cum = n.cumsum(1)
    total, u = cum[:, -1], torch.floor(s["u_sample"].double() * 2.0 ** 32).long()
    limit = (total >> 32) * u + (((total & 0xFFFFFFFF) * (u >> 16) + (((total & 0xFFFFFFFF) * (u & 0xFFFF)) >> 16)) >> 16)
    token = (cum <= limit[:, None]).sum(1)
    out = torch.where(i < accepted[:, None], draft[at], torch.where(i == accepted[:, None], token[:, None], -1))
    return {"n_new": (accepted + 1).to(I32), "tokens": out[i < (drafts + 1)[:, None]].to(I32)}


def _rollback(s):
    one = lambda x, state: _last_three(s, x, state, s["keep"])     # noqa: E731
    return list(map(one, s["x"], s["before"]))


# ---------------------------------------------------------------- in 64 bits

def _grid():
    """Every scale in order, from the bits of the 8-bit floats."""
    return torch.arange(199, device="cuda").to(torch.int16).mul(128).view(torch.float16).double()


def _four_bit(x):
    """x [..., 128] as the cache holds it: the first scale of the grid that is not below max / 7."""
    grid = _grid()
    parts = x.double().reshape(*x.shape[:-1], 4, 32)
    s = grid[torch.searchsorted(grid, parts.abs().amax(-1) / 7.0).clamp(max=198)][..., None]
    return torch.nan_to_num(parts / s, 0.0).round().clamp(-7.0, 7.0).mul(s).reshape(x.shape)


def exact(case, seed):
    """What run returns for these inputs, from the definitions in 64 bits (None where it is whole numbers)."""
    op = case["op"]
    if op == "verify":
        return None
    s = prepare(case, seed)
    if op == "probs":
        l = s["logits"].double()
        if s["temperature"] is None:
            return torch.softmax(l, 1)
        out = torch.zeros_like(l)
        for t, temp in enumerate(s["temperature"].tolist()):
            if temp > 0:
                out[t] = torch.softmax(l[t] / temp, 0)
            else:
                out[t, int((l[t] == l[t].max()).nonzero()[0])] = 1.0
        return out
    cu = s["cu"].tolist()
    if op == "rollback":
        keep = s["keep"].tolist()
        return [torch.stack([torch.cat([st[b], x[cu[b]:cu[b] + keep[b]]])[-3:] for b in range(case["B"])]).double()
                for x, st in zip(s["x"], s["before"])]
    if op == "append":
        Hkv = case["Hkv"]

        def conv(x, state, w):
            parts, states = [], []
            for b in range(case["B"]):
                xs = torch.cat([state[b], x[cu[b]:cu[b + 1]]]).double()
                states.append(xs[-3:])
                n = cu[b + 1] - cu[b]
                parts.append(sum(w.double()[:, j] * xs[j:j + n] for j in range(4)))
            return torch.cat(parts).to(BF16).double().reshape(-1, Hkv, D), torch.stack(states)

        def norm(x, gain):
            return x.double() * torch.rsqrt(x.double().pow(2).mean(-1, keepdim=True) + EPS) * gain.double()

        k, state_k = conv(s["k"], s["state_k"], s["wk"])
        v, state_v = conv(s["v"], s["state_v"], s["wv"])
        return {"q_out": norm(s["q"], s["gq"]), "k": _four_bit(norm(k, s["gk"]).to(BF16)), "v": _four_bit(v),
                "state_k": state_k, "state_v": state_v}
    # attention: sequence by sequence, a few heads at a time
    lut = torch.arange(-8, 8, device="cuda", dtype=F64)
    grid = torch.arange(256, device="cuda").to(torch.int16).mul(128).view(torch.float16).double()
    where = torch.tensor([4 * (e // 2) + 16 * (e % 2) for e in range(8)], device="cuda")
    g = case["Hq"] // case["Hkv"]
    out = torch.empty((s["N"], case["Hq"], D), dtype=F64, device="cuda")
    for b in range(case["B"]):
        T, n = s["total"][b], s["new"][b]
        rows = slice(cu[b], cu[b + 1])
        blocks = s["table"][b, :-(-T // BLOCK)].long()
        i = torch.arange(T - n, T, device="cuda")[:, None]
        delta = i - torch.arange(T, device="cuda")
        hidden = delta < 0
        if case["window"]:
            hidden = hidden | (delta >= case["window"])
        lam = max(1.0, math.log(T) / math.log(case["base"])) if case["base"] > 1 else 1.0
        for h in range(case["Hkv"]):
            kv = []
            for name in ("k", "v"):
                word = s[name][blocks, h].reshape(-1, 64)[:T].contiguous().view(I32).long()
                x = lut[(word[:, :, None] >> where) & 15].reshape(T, 4, 32)
                kv.append((x * grid[s[name + "_scale"][blocks, h].reshape(-1, 4)[:T].long()][..., None]).reshape(T, D))
            heads = slice(h * g, (h + 1) * g)
            z = torch.einsum("nhd,td->hnt", s["q"][rows, heads].double(), kv[0]) / math.sqrt(D)
            if case["ext"]:
                bias = torch.einsum("nhe,hxe->hnx", s["r"][rows, heads].double(), s["P"][heads].double())
                near = (delta >= 0) & (delta < case["ext"])
                z = z + torch.where(near, torch.gather(bias, 2, delta.clamp(0, case["ext"] - 1).expand(g, n, T)), 0.0)
            z = (lam * z).masked_fill(hidden, float("-inf"))
            out[rows, heads] = torch.einsum("hnt,td->nhd", torch.softmax(z, -1), kv[1])
    return out
