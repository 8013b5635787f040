"""A verification step's end on the GPU: probabilities against float64, drafts and drawn tokens equal to a
plain whole-number implementation, conv states bit for bit, and the whole step together.

Bars of the probabilities: a value's error is at most (32 + V 2^-13 + 2 (m - l) / t) 2^-23 of it, as the
header states.  The exponent (l - m) log2(e) / t is rounded four times, 2^-24 of it each, so the
exponential by 4 2^-24 (m - l) / t; the exponential unit adds 2 2^-23.  The sum of a row: a thread adds
at most max(32, V / 4096) values one after the other, then 9 halvings and 8 CTAs, 2^-24 of the sum each:
(V / 4096 + 49) 2^-24 < (V 2^-13 + 25) 2^-23; and a division and three products, 2 2^-23."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda"
F32, I32, BF16 = torch.float32, torch.int32, torch.bfloat16


@pytest.fixture(scope="module")
def ia():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from relative_bias_hybrid_gb300 import build
    build.build()
    import relative_bias_hybrid_gb300.inkattn as ia
    return ia


def _status():
    return torch.zeros(1, dtype=I32, device=DEV)


# ---------------------------------------------------------------- probabilities

def _probs_ref(logits, temperature):
    l = logits.double().cpu()
    l = torch.where(l.isnan(), -torch.inf, l)
    out, bar = torch.zeros_like(l), torch.zeros_like(l)
    for i in range(l.shape[0]):
        t = 1.0 if temperature is None else float(temperature[i])
        m = l[i].max()
        if m == -torch.inf or not 0 <= t < float("inf"):
            continue
        if t == 0:
            out[i, int((l[i] == m).nonzero()[0])] = 1
            continue
        d = torch.where(l[i] == m, 0.0, l[i] - m) / t
        e = torch.exp(d)
        out[i] = e / e.sum()
        bar[i] = torch.where(e > 0, out[i] * (32 + l.shape[1] * 2.0 ** -13 + 2 * d.abs()) * 2.0 ** -23, 0.0) + 2.0 ** -125
    return out, bar


def _check_probs(ia, logits, temperature=None, probs=None, flagged=False):
    probs = torch.full(logits.shape, float("nan"), device=DEV) if probs is None else probs
    want, bar = _probs_ref(logits, temperature)
    st = _status()
    ia.inkattn_token_probs(ia.token_probs_params(logits=logits, probs=probs, temperature=temperature, dev_status=st))
    torch.cuda.synchronize()
    assert int(st) == (ia.INKATTN_ERR_DEVICE_BOUNDS if flagged else 0)
    got = probs.double().cpu()
    assert ((got - want).abs() <= bar).all(), float(((got - want).abs() - bar).max())
    return probs


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T, V", [(1, 1), (1, 2), (3, 3), (2, 5), (7, 31), (5, 1000), (9, 2053), (1, 16389), (2, 50001),
                                  (400, 2049), (1, 131072), (2, 131075), (2, 200019), (1, 262144), (1, 262147), (1, 1 << 20)])
def test_probs_sizes(ia, dtype, T, V):
    g = torch.Generator(device=DEV).manual_seed(V)
    logits = (3 * torch.randn((T, V), generator=g, device=DEV)).to(dtype)
    t = 0.3 + torch.rand((T,), generator=g, device=DEV)
    t[T // 2] = 0.0
    _check_probs(ia, logits)
    _check_probs(ia, logits, t)


@pytest.mark.parametrize("V", [11, 5000, 40003, 300001])
def test_probs_of_odd_values(ia, V):
    """Infinities, NaN, rows without anything, equal maxima, temperatures from tiny to large."""
    g = torch.Generator(device=DEV).manual_seed(V)
    l = 3 * torch.randn((12, V), generator=g, device=DEV)
    l[0] = -torch.inf
    l[1] = torch.nan
    l[2, ::2] = -torch.inf
    l[3, V // 2] = torch.inf
    l[4, V // 3] = l[4, V - 1] = torch.inf
    l[5, 1::3] = torch.nan
    l[6] = 0.0
    l[7] = -3e38
    l[7, V - 2] = 3e38
    l[8, [V // 2, V - 1]] = 100.0                     # a greedy row with two maxima: the first
    l[9] = 2.0                                        # a greedy row of equal logits
    t = torch.ones(12, device=DEV)
    t[8] = t[9] = 0.0
    t[10], t[11] = 1e-30, 1e30
    _check_probs(ia, l)
    _check_probs(ia, l, t)


def test_probs_of_bad_temperatures_are_zero_and_flagged(ia):
    l = torch.randn((4, 700), device=DEV)
    t = torch.tensor([1.0, -1.0, float("nan"), float("inf")], device=DEV)
    probs = _check_probs(ia, l, t, flagged=True)
    assert not probs[1:].any()


@pytest.mark.parametrize("V, wide, at", [(1000, 1003, 0), (40001, 40010, 3), (300000, 300007, 1)])
def test_probs_of_columns_of_wider_rows(ia, V, wide, at):
    """Logits and probabilities at any element of rows of any width, aligned alike or not; what lies beside is left."""
    l = torch.randn((3, wide), device=DEV)
    for shift, dtype in ((at, F32), (at + 1, F32), (at, BF16)):
        probs = torch.full((3, wide + 5), 7.0, device=DEV)
        _check_probs(ia, l.to(dtype)[:, at:at + V], None, probs[:, shift:shift + V])
        assert (probs[:, :shift] == 7).all() and (probs[:, shift + V:] == 7).all()


@pytest.mark.parametrize("V", [4096, 50001, 400001])
def test_probs_in_place(ia, V):
    l = torch.randn((5, V), device=DEV)
    want = _check_probs(ia, l.clone())
    ia.inkattn_token_probs(ia.token_probs_params(logits=l, probs=l))
    torch.cuda.synchronize()
    assert torch.equal(l, want)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("V, wide", [(8192, 8192), (16411, 16417)])
def test_probs_of_many_rows(ia, dtype, V, wide):
    """Rows enough to be read twice, whole batches of groups and ragged ends, greedy rows and odd values among
    them; aligned like their logits or not, and in place."""
    T = 310
    l = (3 * torch.randn((T, wide), device=DEV)).to(dtype)[:, :V]
    t = 0.3 + torch.rand((T,), device=DEV)
    t[::7] = 0.0
    l[3], l[5, V // 2], l[6, 1::3], l[14, [9, V - 1]] = -torch.inf, torch.inf, torch.nan, 100.0
    _check_probs(ia, l, t)
    _check_probs(ia, l, t, torch.empty((T, wide + 4), device=DEV)[:, 3:V + 3])
    if dtype == F32:
        _check_probs(ia, l, t, l)


def test_probs_of_the_most_rows(ia):
    """2^24 rows of one logit, and of a few logits more rows than a grid's smaller dimensions hold."""
    probs = torch.zeros((1 << 24, 1), device=DEV)
    ia.inkattn_token_probs(ia.token_probs_params(logits=torch.randn((1 << 24, 1), device=DEV), probs=probs))
    assert bool((probs == 1).all())
    l = torch.randn((70001, 5), device=DEV)
    probs = torch.empty_like(l)
    ia.inkattn_token_probs(ia.token_probs_params(logits=l, probs=probs))
    want = torch.softmax(l.double(), 1)
    # the bar of _probs_ref at 5 logits less than 12 apart
    assert float((l.max(1).values - l.min(1).values).max()) < 12
    assert bool(((probs.double() - want).abs() <= want * (33 + 24) * 2.0 ** -23).all())


def test_rows_past_32_bits(ia):
    """Rows whose elements lie past 2^32 of the arrays' start: the same probabilities and tokens as of a copy."""
    V, last = 131072, 2 ** 32 // 131072 + 3
    c = _case(7, [9], V)
    far = {k: torch.empty((last + 9, V), device=DEV) for k in ("logits", "target_p", "draft_p")}
    near = 3 * torch.randn((3, V), device=DEV)
    rows = [i * (last // 2) for i in range(3)]                     # three rows of the array, the last past 2^32
    for i, r in enumerate(rows):
        far["logits"][r] = near[i]
    p = ia.token_probs_params(logits=far["logits"], probs=far["target_p"])
    p.N_tok, p.logits_stride, p.probs_stride = 3, V * rows[1], V * rows[1]
    ia.inkattn_token_probs(p)
    want = torch.empty_like(near)
    ia.inkattn_token_probs(ia.token_probs_params(logits=near, probs=want))
    torch.cuda.synchronize()
    for i, r in enumerate(rows):
        assert torch.equal(far["target_p"][r], want[i])
    far["target_p"][last:], far["draft_p"][last:] = c["target_p"], c["draft_p"]
    ids = torch.zeros(last + 9, dtype=I32, device=DEV)
    ids[last:] = c["token_ids"]
    u = torch.zeros(last + 9, device=DEV)
    u[last:] = c["u_accept"]
    got = _verify(ia, dict(c, target_p=far["target_p"], draft_p=far["draft_p"], token_ids=ids, u_accept=u,
                           cu_seqlens_q=torch.tensor([last, last + 9], dtype=I32, device=DEV)))
    near_got = _verify(ia, c)
    assert got[0] == near_got[0] and got[1][last:] == near_got[1] and got[1][:last] == [-7] * last


def test_verify_of_the_most_sequences(ia):
    """2^20 sequences of one row each."""
    B = 1 << 20
    p = torch.zeros((B, 2), device=DEV)
    odd = torch.arange(B, device=DEV) % 2
    p[torch.arange(B, device=DEV), odd] = 1
    n_new, out = torch.zeros(B, dtype=I32, device=DEV), torch.zeros(B, dtype=I32, device=DEV)
    st = _status()
    ia.inkattn_verify_drafts(ia.verify_drafts_params(
        target_p=p, token_ids=torch.zeros(B, dtype=I32, device=DEV), cu_seqlens_q=torch.arange(B + 1, dtype=I32, device=DEV),
        u_accept=torch.zeros(B, device=DEV), u_sample=torch.rand(B, device=DEV), n_new=n_new, out_tokens=out, dev_status=st))
    assert int(st) == 0 and bool((n_new == 1).all()) and torch.equal(out, odd.to(I32))


# ---------------------------------------------------------------- verification

def _steps(w):
    """Whole multiples of 2^-43 of weights in [0, 1] (numpy rounds ties to even)."""
    return np.rint(np.clip(np.nan_to_num(w.astype(np.float64), nan=0.0), 0, 1) * 2.0 ** 43).astype(object)


def _verify_ref(p, q, ids, cu, ua, us):
    """Row by row, in Python's whole numbers."""
    p, ids, cu, ua, us = (x.cpu().numpy() for x in (p, ids, cu, ua, us))
    q = None if q is None else q.cpu().numpy()
    V = p.shape[1]

    def unit(v):
        return np.float32(np.clip(np.nan_to_num(v, nan=0.0), 0, 1))
    below = np.float32(1 - 2.0 ** -24)
    n_new, out, flagged = [], [None] * p.shape[0], False
    for b in range(len(cu) - 1):
        rows = list(range(cu[b], cu[b + 1]))
        if not rows:
            n_new.append(0)
            continue
        k, lost = 0, None
        while k < len(rows) - 1:
            r, x = rows[k], int(ids[rows[k] + 1])
            u = min(unit(ua[r]), below)
            if not 0 <= x < V or not np.float32(u * (np.float32(1) if q is None else unit(q[r, x]))) < unit(p[r, x]):
                lost = x
                break
            out[r] = x
            k += 1
        r = rows[k]
        pr = np.clip(np.nan_to_num(p[r], nan=0.0), 0, 1).astype(np.float32)
        w = pr.copy()
        if lost is not None and not 0 <= lost < V:
            flagged = True
        elif lost is not None and q is None:
            w[lost] = 0
        elif lost is not None:
            w = np.maximum(pr - np.clip(np.nan_to_num(q[r], nan=0.0), 0, 1).astype(np.float32), np.float32(0))
        n = _steps(w)
        if n.sum() == 0:
            n = _steps(pr)
        total = int(n.sum())
        for i in rows[k:]:
            out[i] = -1
        if total == 0:
            flagged = True
            n_new.append(k)
            continue
        limit = total * int(np.floor(float(min(unit(us[b]), below)) * 2.0 ** 32)) >> 32
        out[r] = int((np.cumsum(n) <= limit).sum())
        n_new.append(k + 1)
    return n_new, out, flagged


def _case(seed, lens, V, drafter=True, spread=2.0, near=0.5):
    g = torch.Generator(device=DEV).manual_seed(seed)
    N = sum(lens)
    l = spread * torch.randn((N, V), generator=g, device=DEV)
    p = torch.softmax(l, 1)
    q = torch.softmax(l + near * torch.randn((N, V), generator=g, device=DEV), 1)
    ids = torch.randint(0, V, (max(N, 1),), generator=g, device=DEV)
    if N > 1:
        ids[1:] = torch.multinomial(q, 1, generator=g)[:-1, 0]
    cu = torch.tensor([0] + list(np.cumsum(lens)), dtype=I32, device=DEV)
    return {"target_p": p, "draft_p": q if drafter else None, "token_ids": ids[:N].to(I32), "cu_seqlens_q": cu,
            "u_accept": torch.rand((N,), generator=g, device=DEV), "u_sample": torch.rand((len(lens),), generator=g, device=DEV)}


def _verify(ia, c, stream=None):
    N, B = c["token_ids"].numel(), c["cu_seqlens_q"].numel() - 1
    out = {"n_new": torch.full((B,), -7, dtype=I32, device=DEV), "out_tokens": torch.full((N,), -7, dtype=I32, device=DEV)}
    st = _status()
    ia.inkattn_verify_drafts(ia.verify_drafts_params(**c, **out, dev_status=st), stream)
    torch.cuda.synchronize()
    return out["n_new"].tolist(), out["out_tokens"].tolist(), int(st) == ia.INKATTN_ERR_DEVICE_BOUNDS


def _check_verify(ia, c):
    want = _verify_ref(c["target_p"], c["draft_p"], c["token_ids"], c["cu_seqlens_q"], c["u_accept"], c["u_sample"])
    got = _verify(ia, c)
    assert got == (list(want[0]), list(want[1]), want[2])
    return got


@pytest.mark.parametrize("drafter", [True, False])
@pytest.mark.parametrize("lens, V", [([1], 1), ([2], 1), ([3, 1, 2], 2), ([1, 0, 5, 0], 3), ([9, 4], 67), ([9] * 5, 2048),
                                     ([9, 1, 3], 2051), ([40, 70], 513), ([9] * 3, 5003), ([9, 2], 16384), ([5, 9], 50001),
                                     ([9] * 4, 131072), ([9], 200019), ([3], (1 << 20) - 1), ([2], 1 << 20)])
def test_verify_sizes(ia, lens, V, drafter):
    for seed in range(3):
        _check_verify(ia, _case(seed, lens, V, drafter))


def test_verify_keeps_all_and_none(ia):
    c = _case(3, [9, 9], 1000)
    c["u_accept"][:9] = 0.0                      # (u q < p holds wherever p > 0)
    c["draft_p"][9] = 1.0
    c["u_accept"][9] = 0.999
    n, tokens, _ = _check_verify(ia, c)
    assert n[0] == 9 and n[1] == 1 and tokens[9] >= 0 and tokens[10:] == [-1] * 8


def test_verify_equal_distributions_fall_back_to_the_target(ia):
    """p = q: u q < p stands for every u below 1, and a draft that does not stand (p scaled under
    it everywhere) leaves no weight: the draw is from p."""
    c = _case(4, [9, 5], 3001, near=0.0)
    c["draft_p"] = c["target_p"].clone()
    n, _, _ = _check_verify(ia, c)
    assert n == [9, 5]
    c["target_p"][4] = c["draft_p"][4] * 0.5
    c["target_p"][4, int(c["token_ids"][5])] = 0.0
    n, tokens, flagged = _check_verify(ia, c)
    assert n == [5, 5] and tokens[4] >= 0 and not flagged


def test_verify_one_hot_rows_are_greedy(ia):
    """Greedy requests: one-hot rows let exactly the drafts stand that are the target's choice."""
    V, lens = 4099, [9]
    c = _case(5, lens, V, drafter=False)
    best = torch.randint(0, V, (9,), device=DEV)
    c["target_p"] = torch.nn.functional.one_hot(best, V).float()
    c["token_ids"][1:6] = best[:5].to(I32)
    c["token_ids"][6] = (best[5] + 1) % V
    n, tokens, _ = _check_verify(ia, c)
    assert n == [6] and tokens[:6] == best[:6].tolist()


def test_verify_odd_values_and_bad_indices(ia):
    """NaN, infinite and negative probabilities, rows without weight, drafts outside the vocabulary, u outside
    [0, 1)."""
    V = 2500
    c = _case(6, [3, 3, 3, 3, 2], V)
    p, q, ids = c["target_p"], c["draft_p"], c["token_ids"]
    p[0] = 0.0
    p[3, ::7], p[3, 1::7], p[3, 2::7] = float("nan"), float("inf"), -1.0
    q[3, ::5], q[3, 1::5] = float("nan"), 2.0
    ids[7] = V
    ids[10] = -1
    c["u_accept"][3:6] = torch.tensor([float("nan"), 1.0, 5.0])
    c["u_sample"][:5] = torch.tensor([0.5, 1.0, -3.0, float("nan"), 0.9999999])
    n, tokens, flagged = _check_verify(ia, c)
    assert flagged and n[0] == 0 and tokens[:3] == [-1, -1, -1]


@pytest.mark.parametrize("u", [0.0, 2.0 ** -24, 0.5, 1 - 2.0 ** -24])
def test_verify_draws_at_the_ends(ia, u):
    """The first and the last token with weight, whatever lies beside them."""
    V = 70001
    c = _case(7, [1, 1], V)
    c["target_p"][:, :100] = 0.0
    c["target_p"][:, -100:] = 0.0
    c["target_p"][1] = 0.0
    c["target_p"][1, 60000] = 1e-12
    c["u_sample"][:] = u
    _, tokens, _ = _check_verify(ia, c)
    assert 100 <= tokens[0] < V - 100 and tokens[1] == 60000


def test_verify_rows_of_wider_matrices(ia):
    c = _case(8, [9, 4], 5001)
    want = _check_verify(ia, c)
    for pad, at in ((3, 0), (8, 1), (6, 2)):
        wide = {k: torch.full((13, 5001 + pad), 0.5, device=DEV) for k in ("target_p", "draft_p")}
        for k, off in (("target_p", at), ("draft_p", at if pad == 8 else 0)):
            wide[k][:, off:off + 5001] = c[k]
            wide[k] = wide[k][:, off:off + 5001]
        assert _check_verify(ia, {**c, **wide}) == want


def test_verify_bad_offsets_are_flagged(ia):
    c = _case(9, [3, 3, 3], 200)
    c["cu_seqlens_q"] = torch.tensor([0, 5, 3, 100], dtype=I32, device=DEV)
    n, tokens, flagged = _verify(ia, c)
    assert flagged and n[1] == n[2] == 0 and n[0] >= 1 and tokens[5:] == [-7] * 4


def test_verify_follows_the_distribution(ia):
    """Drafts from q and evenly spaced draws: the emitted first tokens have the target's frequencies.  20000
    sequences of one draft; a frequency's standard deviation is at most sqrt(0.25 / 20000) = 0.0036, and 5 of
    them are allowed."""
    V, B = 8, 20000
    g = torch.Generator(device=DEV).manual_seed(1)
    p = torch.softmax(1.5 * torch.randn((V,), generator=g, device=DEV), 0)
    q = torch.softmax(1.5 * torch.randn((V,), generator=g, device=DEV), 0)
    ids = torch.zeros(2 * B, dtype=I32, device=DEV)
    ids[1::2] = torch.multinomial(q, B, replacement=True, generator=g).to(I32)
    c = {"target_p": p.expand(2 * B, V).contiguous(), "draft_p": q.expand(2 * B, V).contiguous(), "token_ids": ids,
         "cu_seqlens_q": torch.arange(0, 2 * B + 1, 2, dtype=I32, device=DEV),
         "u_accept": torch.rand((2 * B,), generator=g, device=DEV), "u_sample": torch.rand((B,), generator=g, device=DEV)}
    _, tokens, _ = _verify(ia, c)
    freq = np.bincount(np.array(tokens)[::2], minlength=V) / B
    assert np.abs(freq - p.cpu().numpy()).max() <= 5 * 0.0036


# ---------------------------------------------------------------- conv states

def _rollback_ref(x, before, keep, cu, slot):
    after = before.clone()
    for b in range(len(keep)):
        after[slot[b]] = torch.cat([before[slot[b]], x[cu[b]:cu[b] + keep[b]]])[-3:]
    return after


@pytest.mark.parametrize("widths, lens", [((8,), [1]), ((1024, 1024, 8192, 8192), [9] * 32), ((1016, 2056), [0, 1, 2, 3, 4, 17]),
                                          ((8, 16, 24, 32, 40, 1032, 48, 56), [5, 0, 2])])
@pytest.mark.parametrize("in_place", [False, True])
def test_rollback(ia, widths, lens, in_place):
    g = torch.Generator(device=DEV).manual_seed(len(lens))
    N, B, slots = sum(lens), len(lens), len(lens) + 3
    cu = [0] + list(np.cumsum(lens))
    slot = torch.randperm(slots, generator=torch.Generator().manual_seed(1))[:B]
    for trial in range(4):
        keep = [min(n, (trial + i) % 5) if trial else n for i, n in enumerate(lens)]
        # the convs' rows are columns of wider rows, as the projections' are
        rows = torch.randn((N, sum(widths) + 8), generator=g, device=DEV).to(BF16)
        at = np.cumsum([8] + list(widths))
        x = [rows[:, at[i]:at[i] + w] for i, w in enumerate(widths)]
        before = [torch.randn((slots, 3, w), generator=g, device=DEV).to(BF16) for w in widths]
        want = [_rollback_ref(a, s, keep, cu, slot) for a, s in zip(x, before)]
        after = before if in_place else [s.clone() for s in before]
        st = _status()
        ia.inkattn_conv_rollback(ia.conv_rollback_params(
            x=x, state_before=before, state_after=after, n_keep=torch.tensor(keep, dtype=I32, device=DEV),
            cu_seqlens_q=torch.tensor(cu, dtype=I32, device=DEV), state_slot=slot.to(I32).to(DEV), dev_status=st))
        torch.cuda.synchronize()
        assert int(st) == 0
        assert all(torch.equal(a, b) for a, b in zip(after, want))


def test_rollback_bad_indices_are_flagged_and_skipped(ia):
    x, before = torch.randn((6, 16), device=DEV).to(BF16), torch.randn((4, 3, 16), device=DEV).to(BF16)
    for keep, slot, cu in (([3, 1], [0, 1], [0, 2, 6]), ([1, -1], [0, 1], [0, 2, 6]), ([1, 1], [0, 4], [0, 2, 6]),
                           ([1, 1], [-1, 2], [0, 2, 6]), ([1, 1], [0, 1], [0, 2, 7]), ([1, 0], [0, 1], [0, 3, 2])):
        after, st = before.clone(), _status()
        t = lambda v: torch.tensor(v, dtype=I32, device=DEV)     # noqa: E731
        ia.inkattn_conv_rollback(ia.conv_rollback_params(x=[x], state_before=[before], state_after=[after], n_keep=t(keep),
                                                         cu_seqlens_q=t(cu), state_slot=t(slot), dev_status=st))
        torch.cuda.synchronize()
        assert int(st) == ia.INKATTN_ERR_DEVICE_BOUNDS
        good = [b for b in range(2) if 0 <= slot[b] < 4 and 0 <= cu[b] <= cu[b + 1] <= 6 and 0 <= keep[b] <= cu[b + 1] - cu[b]]
        want = before.clone()
        for b in good:
            want[slot[b]] = torch.cat([before[slot[b]], x[cu[b]:cu[b] + keep[b]]])[-3:]
        assert len(good) == 1 and torch.equal(after, want)


# ---------------------------------------------------------------- together

def _step(ia, w, x, state, V, kv):
    """A verification step: projections and prologue, decode, head, probabilities, verification, rollback."""
    from relative_bias_hybrid_gb300 import inputs as gen
    from relative_bias_hybrid_gb300.step import QkvrStep, VerifyStep
    x = dict(x, conv_state_k=state["k"], conv_state_v=state["v"])
    qk = QkvrStep(w, x, want_y=True)
    N, C = w.N_tok, w.Hkv * 128
    out = torch.empty((N, w.Hq, 128), dtype=BF16, device=DEV)
    attn = ia.attn_params(q=qk.q_out, k_cache=x["k_cache"], v_cache=x["v_cache"], k_scale=x.get("k_scale"),
                          v_scale=x.get("v_scale"), cu_seqlens_q=x["cu_seqlens_q"], seqlen_k=x["seqlen_k"],
                          block_table=x["block_table"], out=out, max_seqlen_q=max(w.q_lens), max_seqlen_k=max(w.seqlen_k),
                          r=qk.r_out, P=x["P"], rel_extent=w.rel_extent, log_scale_base=w.log_scale_base, dev_status=qk.status)
    splits = 3
    ws = torch.empty(ia.inkattn_decode_workspace_bytes(attn, splits), dtype=torch.uint8, device=DEV)
    xv = gen.make_verify_inputs(w, V, seed=5, device=DEV)
    logits = torch.empty((N, V), device=DEV)
    head = ia.linear_params(x=out.view(N, -1), w=xv["w_head"], out=logits, dev_status=qk.status)
    k_rows, v_rows = qk.y_out[:, w.Hq * 128:w.Hq * 128 + C], qk.y_out[:, w.Hq * 128 + C:w.Hq * 128 + 2 * C]
    kept = {n: torch.zeros_like(state[n]) for n in ("k", "v")}
    end = VerifyStep(w, xv, logits, [(k_rows, state["k"], kept["k"]), (v_rows, state["v"], kept["v"])])

    def run(stream=None):
        qk.run(stream)
        ia.inkattn_decode(attn, splits, ws, stream)
        ia.inkattn_combine(attn, splits, ws, stream)
        ia.inkattn_linear(head, stream)
        end.run(stream)
    return run, qk, out, logits, xv, end, kept


@pytest.mark.parametrize("kv", ["i4", "bf16"])
def test_a_whole_verification_step(ia, kv):
    """The step's results from its own parts; and the conv states and cache rows it keeps equal those of a step
    over the kept rows alone, which no draft was ever rejected from."""
    from relative_bias_hybrid_gb300 import inputs as gen
    V = 1003
    w = gen.custom("step", Hq=16, Hkv=2, q_lens=[9, 4, 1, 9], prefix_lens=[300, 70, 5, 1], rel_extent=64, log_scale_base=64.0)
    x = gen.make_qkvr_inputs(w, 256, seed=2, device=DEV, kv_dtype=kv, grid=True)
    state = {"k": x["conv_state_k"], "v": x["conv_state_v"]}
    run, qk, out, logits, xv, end, kept = _step(ia, w, x, state, V, kv)
    run()
    torch.cuda.synchronize()
    assert qk.device_status() == 0 and end.device_status() == 0
    want, bar = _probs_ref(logits, xv["temperature"])
    assert ((end.probs.double().cpu() - want).abs() <= bar).all()
    ref = _verify_ref(end.probs, xv["draft_p"], xv["token_ids"], xv["cu_seqlens_q"], xv["u_accept"], xv["u_sample"])
    assert end.n_new.tolist() == ref[0] and end.tokens.tolist() == ref[1]
    n = end.n_new.tolist()
    # the kept rows alone, from the same state, into another cache
    cu = xv["cu_seqlens_q"].tolist()
    rows = torch.cat([torch.arange(cu[b], cu[b] + n[b]) for b in range(w.B)]).to(DEV)
    w2 = gen.custom("kept", Hq=16, Hkv=2, q_lens=n, prefix_lens=w.prefix_lens, rel_extent=64, log_scale_base=64.0)
    x2 = dict(x, x=x["x"][rows], slot_mapping=x["slot_mapping"][rows], cu_seqlens_q=torch.tensor(
        [0] + list(np.cumsum(n)), dtype=I32, device=DEV), **{c: x[c].clone() for c in x if "cache" in c or "scale" in c})
    for c in x2:
        if "cache" in c or "scale" in c:
            x2[c].zero_()
    from relative_bias_hybrid_gb300.step import QkvrStep
    only = QkvrStep(w2, x2)
    only.run()
    torch.cuda.synchronize()
    assert torch.equal(kept["k"], only.state_k) and torch.equal(kept["v"], only.state_v)
    slots = x["slot_mapping"][rows].long()
    for c in x2:
        if "cache" in c or "scale" in c:
            assert torch.equal(x[c][slots // 64, :, slots % 64], x2[c][slots // 64, :, slots % 64]), c


def test_a_captured_step_replays_the_same(ia):
    from relative_bias_hybrid_gb300 import inputs as gen
    w = gen.custom("graph", Hq=16, Hkv=2, q_lens=[9, 3], prefix_lens=[200, 900], rel_extent=32)
    x = gen.make_qkvr_inputs(w, 256, seed=3, device=DEV, kv_dtype="i4")
    state = {"k": x["conv_state_k"], "v": x["conv_state_v"]}
    run, qk, out, logits, xv, end, kept = _step(ia, w, x, state, 50001, "i4")
    run()
    torch.cuda.synchronize()
    want = [t.clone() for t in (out, end.probs, end.n_new, end.tokens, kept["k"], kept["v"])]
    s = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s), torch.cuda.graph(graph, stream=s):
        run(s)
    for t in (out, end.probs, end.n_new, end.tokens, kept["k"], kept["v"]):
        t.zero_()
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert end.device_status() == 0
    for t, v in zip((out, end.probs, end.n_new, end.tokens, kept["k"], kept["v"]), want):
        assert torch.equal(t, v)


def test_two_streams_at_once(ia):
    """Two verifications in flight on two streams: each its own result."""
    cases = [_case(s, [9] * 16, 50001) for s in (1, 2)]
    want = [_verify(ia, c) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    got = []
    for _ in range(5):
        outs = []
        for c, s in zip(cases, streams):
            o = {"n_new": torch.empty(16, dtype=I32, device=DEV), "out_tokens": torch.empty(144, dtype=I32, device=DEV)}
            torch.cuda.synchronize()
            outs.append((o, ia.verify_drafts_params(**c, **o), s))
        for o, p, s in outs:
            ia.inkattn_verify_drafts(p, s)
        torch.cuda.synchronize()
        got = [(o["n_new"].tolist(), o["out_tokens"].tolist(), False) for o, _, _ in outs]
        assert got == want


def test_rollback_of_the_most_sequences(ia):
    B, C = 65535, 8
    x, before = torch.randn((B, C), device=DEV).to(BF16), torch.randn((B, 3, C), device=DEV).to(BF16)
    n = (torch.arange(B, device=DEV) % 2).to(I32)
    want = torch.where((n == 1)[:, None, None], torch.cat([before[:, 1:], x[:, None]], 1), before)
    ia.inkattn_conv_rollback(ia.conv_rollback_params(
        x=[x], state_before=[before], state_after=[before], n_keep=n, state_slot=torch.arange(B, dtype=I32, device=DEV),
        cu_seqlens_q=torch.arange(B + 1, dtype=I32, device=DEV)))
    assert torch.equal(before, want)
