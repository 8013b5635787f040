"""GPU parity of the linear layer, the grouped expert products, the router and the weighted
sum against plain 64-bit forms (torch float64 on the CPU).

Bars.  On grid inputs (x = i/8, w = j/64, bias and residual multiples of 2^-9, all small) every
partial sum is a multiple of 2^-9 below 2^14, so it is exact in fp32 in any order: the products
without a curved activation must then be bit-equal to the rounded 64-bit value, whatever the
tile, the split or the path of the store.  With a curved activation the fp32 argument v is still
exact and the tolerance is the rounding of the output (half a step) plus the fp32 evaluation of
the curve, see _curve_slack.  On Gaussian inputs the sum itself is rounded: K fp32 additions, each
off by at most one step (2^-23) of the sum of magnitudes."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

BF16, F32, I32, F64 = torch.bfloat16, torch.float32, torch.int32, torch.float64
HALF_STEP = {BF16: 2.0 ** -8, F32: 2.0 ** -24}


@pytest.fixture(scope="module")
def ia():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from relative_bias_hybrid_gb300 import build
    build.build()
    import relative_bias_hybrid_gb300.inkattn as ia
    return ia


def _grid(shape, g, lo, hi, unit, dtype=BF16):
    return (torch.randint(lo, hi + 1, shape, generator=g).to(F64) * unit).to(dtype)


def _act64(v, act):
    if act == "relu":
        return v.clamp(min=0)
    if act == "gelu":
        return 0.5 * v * torch.special.erfc(-v / 2 ** 0.5)
    if act == "silu":
        return v * torch.sigmoid(v)
    if act == "swiglu":
        a, b = v.chunk(2, dim=-1)
        return a * torch.sigmoid(a) * b
    return v


def _curve_slack(v, act):
    """Absolute error of the fp32 curve at an exact argument v.  __expf is within 2 + 1.173 |x|
    units of 2^-23 of exp(x) (its documented bound), the sum 1 + exp and the division add a unit
    each: silu is within (4 + 1.2 |v|) 2^-23 |silu|, and below -87 the exp leaves fp32's range,
    where silu is under 1e-36.  gelu takes |v| / 2 times an erfc that is within 1.5e-7 (1.3 units of
    2^-23) by its formula, and by its evaluation within about 5 units of its own value, at most 1 (the
    exponential, 2 + 1.173 x^2 times exp(-x^2), is within 2.5 units; the division and the polynomial
    2; the products 1): (1.3 + 5.5) / 2 < 4 units of |v|."""
    if act == "gelu":
        return 4 * 2.0 ** -23 * v.abs()
    if act == "silu":
        return (4 + 1.2 * v.abs()) * 2.0 ** -23 * _act64(v, "silu").abs() + 1e-36
    if act == "swiglu":
        a, b = v.chunk(2, dim=-1)
        return (5 + 1.2 * a.abs()) * 2.0 ** -23 * _act64(v, "swiglu").abs() + 1e-36 * b.abs()
    return torch.zeros_like(v)


def _check(got, v, act, residual=None, sum_slack=None):
    """got [N][F] against act(v) + residual, v exact or off by at most sum_slack."""
    y = _act64(v, act)
    slack = _curve_slack(v, act)
    if sum_slack is not None:
        # every curve here has a slope below 1.13; of the product both factors move
        if act == "swiglu":
            a, b = v.chunk(2, dim=-1)
            sa, sb = sum_slack.chunk(2, dim=-1)
            slack = slack + 1.13 * sa * b.abs() + (a.abs() + sa) * sb
        else:
            slack = slack + 1.13 * sum_slack
    if residual is not None:
        y = y + residual
        slack = slack + 2.0 ** -24 * (y.abs() + slack)          # the fp32 addition
    if act in ("none", "relu") and sum_slack is None:
        assert torch.equal(got.cpu(), y.to(F32).to(got.dtype))
        return
    err = (got.cpu().to(F64) - y).abs()
    # (the smallest normal numbers: results below them may be flushed)
    bound = slack + HALF_STEP[got.dtype] * (y.abs() + slack) + 2.0 ** -126
    assert bool((err <= bound).all()), float((err - bound).max())


def _linear_inputs(T, K, F, act, seed, grid=True):
    g = torch.Generator().manual_seed(seed)
    rows = 2 * F if act == "swiglu" else F
    if grid:
        return (_grid((T, K), g, -8, 8, 1 / 8), _grid((rows, K), g, -8, 8, 1 / 64),
                _grid((rows,), g, -512, 512, 2.0 ** -9, F32), _grid((T, F), g, -64, 64, 1 / 8))
    return (torch.randn((T, K), generator=g).to(BF16), (torch.randn((rows, K), generator=g) * K ** -0.5).to(BF16),
            torch.randn((rows,), generator=g), torch.randn((T, F), generator=g).to(BF16))


def _run_linear(ia, x, w, bias, residual, act, dtype, F, stream=None):
    N = x.shape[0]
    # the output sits between two guard rows that must stay as they are
    buf = torch.full(((N + 2) * F + 16,), 7.0, dtype=dtype, device="cuda")
    lead = (F + 15) // 16 * 16
    out = buf[lead:lead + N * F].view(N, F)
    status = torch.zeros(1, dtype=I32, device="cuda")
    dev = [t.cuda() if t is not None else None for t in (x, w, bias, residual)]
    p = ia.linear_params(x=dev[0], w=dev[1], out=out, act=act, bias=dev[2], residual=dev[3], dev_status=status)
    torch.cuda.synchronize()
    ia.inkattn_linear(p, stream)
    torch.cuda.synchronize()
    assert int(status) == 0
    assert bool((buf[:lead] == 7).all()) and bool((buf[lead + N * F:] == 7).all())
    return out


SIZES = [(1, 8, 1), (1, 8, 8), (1, 64, 256), (1, 4096, 2048), (2, 72, 7), (3, 520, 129), (9, 128, 250),
         (31, 200, 64), (32, 64, 128), (33, 1000, 264), (64, 2048, 512), (127, 56, 15), (160, 328, 1021),
         (256, 256, 256), (257, 512, 300), (288, 1024, 1024), (513, 192, 520), (1100, 96, 2600)]


@pytest.mark.parametrize("T,K,F", SIZES)
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_linear_exact_on_grid_inputs(ia, T, K, F, dtype):
    x, w, bias, residual = _linear_inputs(T, K, F, "none", seed=T + K + F)
    v = x.double() @ w.double().t()
    _check(_run_linear(ia, x, w, None, None, "none", dtype, F), v, "none")
    v = v + bias.double()
    _check(_run_linear(ia, x, w, bias, residual, "none", dtype, F), v, "none", residual.double())
    _check(_run_linear(ia, x, w, bias, None, "relu", dtype, F), v, "relu")


@pytest.mark.parametrize("T,K,F", [(1, 8, 1), (1, 4096, 2048), (9, 128, 250), (33, 1000, 264), (300, 512, 1021)])
@pytest.mark.parametrize("act", ["gelu", "silu"])
def test_linear_curved_activations(ia, T, K, F, act):
    x, w, bias, residual = _linear_inputs(T, K, F, act, seed=7 * T + F)
    v = x.double() @ w.double().t() + bias.double()
    for dtype in (BF16, F32):
        _check(_run_linear(ia, x, w, bias, None, act, dtype, F), v, act)
        _check(_run_linear(ia, x, w, bias, residual, act, dtype, F), v, act, residual.double())


@pytest.mark.parametrize("T,K,F", [(1, 8, 1), (1, 8, 16), (1, 2048, 1024), (9, 128, 45), (33, 1000, 272),
                                   (300, 512, 1040), (70, 64, 130)])
def test_linear_swiglu(ia, T, K, F):
    x, w, bias, residual = _linear_inputs(T, K, F, "swiglu", seed=11 * T + F)
    v = x.double() @ w.double().t()
    for dtype in (BF16, F32):
        _check(_run_linear(ia, x, w, None, None, "swiglu", dtype, F), v, "swiglu")
        _check(_run_linear(ia, x, w, bias, residual, "swiglu", dtype, F), v + bias.double(), "swiglu",
               residual.double())


@pytest.mark.parametrize("T,K,F,act", [(1, 8192, 512, "none"), (40, 8192, 512, "swiglu"), (700, 2048, 777, "gelu")])
def test_linear_gaussian(ia, T, K, F, act):
    x, w, bias, residual = _linear_inputs(T, K, F, act, seed=5, grid=False)
    v = x.double() @ w.double().t() + bias.double()
    mags = x.double().abs() @ w.double().abs().t() + bias.double().abs()
    for dtype in (BF16, F32):
        _check(_run_linear(ia, x, w, bias, residual, act, dtype, F), v, act, residual.double(),
               sum_slack=(K + 1) * 2.0 ** -23 * mags)


@pytest.mark.parametrize("T,K,F,act", [(161, 4104, 300, "none"), (400, 1032, 1030, "relu"), (1000, 520, 264, "swiglu"),
                                       (5000, 1600, 700, "none")])
def test_linear_fp32_output_in_parts(ia, T, K, F, act):
    """fp32 outputs over several parts of K and several items a pair: exact on grid inputs."""
    x, w, bias, residual = _linear_inputs(T, K, F, act, seed=K)
    v = x.double() @ w.double().t() + bias.double()
    _check(_run_linear(ia, x, w, bias, None if act == "relu" else residual, act, F32, F), v, act,
           None if act == "relu" else residual.double())


@pytest.mark.parametrize("T,K,F,act", [(257, 8200, 5000, "none"), (300, 8192, 3000, "relu"), (384, 8192, 5001, "none"),
                                       (350, 9000, 2500, "swiglu"), (384, 9000, 1900, "swiglu")])
def test_linear_between_one_and_two_full_tiles(ia, T, K, F, act):
    """Between 257 and 384 tokens over a long K: few tiles, split or not."""
    x, w, bias, residual = _linear_inputs(T, K, F, act, seed=F)
    v = x.double() @ w.double().t() + bias.double()
    _check(_run_linear(ia, x, w, bias, None if act == "relu" else residual, act, BF16, F), v, act,
           None if act == "relu" else residual.double())


def test_linear_fp32_output_is_summed_to_nearest(ia):
    """K = 8192 in fp32: the parts' sums keep the error of the whole output below 1e-6 of its norm
    (64 steps to nearest over each part's 32, of random sign, measure 5e-7; one long accumulation in
    the tensor cores measured 8e-6)."""
    x, w, _, _ = _linear_inputs(64, 8192, 512, "none", seed=4, grid=False)
    got = _run_linear(ia, x, w, None, None, "none", F32, 512).cpu().double()
    want = x.double() @ w.double().t()
    assert float((got - want).norm() / want.norm()) < 1e-6


def test_linear_in_place_residual_and_infinities(ia):
    """out == residual; infinities and NaN stay in their own token's row."""
    T, K, F = 40, 128, 264
    x, w, bias, residual = _linear_inputs(T, K, F, "none", seed=3)
    x[5, 7] = float("inf"); x[6, 1] = float("nan"); x[7, 3] = -float("inf")
    dev = [t.cuda() for t in (x, w, bias, residual)]
    ia.inkattn_linear(ia.linear_params(x=dev[0], w=dev[1], bias=dev[2], residual=dev[3], out=dev[3]))
    torch.cuda.synchronize()
    want = (x.double() @ w.double().t() + bias.double() + residual.double()).to(F32).to(BF16)
    got = dev[3].cpu()
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(torch.nan_to_num(got.float()), torch.nan_to_num(want.float()))


@pytest.mark.parametrize("act", ["relu", "gelu", "silu", "swiglu"])
def test_linear_activations_of_wide_arguments(ia, act):
    """Arguments from -60 to 60 in steps of 1/32, and NaN: an identity weight passes them through."""
    v = torch.arange(-1920, 1921).double() / 32
    K = 8 * ((v.numel() + 7) // 8)
    x = torch.zeros((2, K), dtype=BF16)
    x[0, :v.numel()] = v.to(BF16)                      # (rounded to bf16: the arguments are what x holds)
    x[1, 5] = float("nan")
    w = torch.eye(K, dtype=BF16)
    if act == "swiglu":
        w = torch.cat([w, w.flip(0)])
    for dtype in (BF16, F32):
        got = _run_linear(ia, x, w, None, None, act, dtype, K)
        arg = torch.cat([x[:1].double(), x[:1].double().flip(1)], 1) if act == "swiglu" else x[:1].double()
        _check(got[:1], arg, act)
        assert bool(torch.isnan(got[1]).all())         # NaN times a zero weight is a NaN everywhere


@pytest.mark.parametrize("act", ["none", "relu", "gelu", "silu", "swiglu"])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,K,F", [(3, 64, 24), (3, 1024, 24), (200, 64, 24), (200, 64, 27)])
def test_linear_infinite_sums(ia, act, dtype, T, K, F):
    """A sum of +infinity or -infinity takes the formula's value (infinity, 0 or NaN), through the
    split's join and both kinds of stores alike; the features beside it keep theirs."""
    inf = float("inf")
    rows = F * (2 if act == "swiglu" else 1)
    x, w = torch.ones((T, K), dtype=BF16), torch.zeros((rows, K), dtype=BF16)
    bias = torch.ones(rows, dtype=F32)
    bias[:6] = torch.tensor([inf, -inf, float("nan"), 3.0e38, -3.0e38, 0.0])
    if act == "swiglu":
        bias[F + 6:F + 8] = torch.tensor([inf, -inf])
    got = _run_linear(ia, x, w, bias, None, act, dtype, F).cpu()
    want = _act64(bias.double().expand(T, rows), act)
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(torch.isinf(got), torch.isinf(want.to(dtype)))
    assert torch.equal(got[torch.isinf(got)].double(), want.to(dtype)[torch.isinf(got)].double())
    live = torch.isfinite(want) & torch.isfinite(got.double())
    # half a step, and the curve: its arguments are 1, 0 or so large that a limit is reached, and at 1
    # _curve_slack's bounds are 4 (gelu), 5.2 (silu) and 6.2 (swiglu) units of 2^-23, under 8 of the value
    slack = (HALF_STEP[dtype] + 8 * 2.0 ** -23) * want.abs() + 1e-36
    assert bool(((got.double() - want).abs() <= slack)[live].all())


@pytest.mark.parametrize("T", [1, 2, 3, 4, 5, 7, 8])
@pytest.mark.parametrize("K,F", [(8, 1), (8, 5), (264, 33), (512, 7), (520, 250), (2056, 1021), (4096, 3), (4104, 700),
                                 (8200, 129)])
@pytest.mark.parametrize("act", ["none", "relu", "gelu", "swiglu"])
def test_linear_few_tokens(ia, T, K, F, act):
    """Few tokens: every count of them, rows of one, a few and many pieces of 16 bytes, odd widths."""
    x, w, bias, residual = _linear_inputs(T, K, F, act, seed=T + K + F)
    v = x.double() @ w.double().t()
    for dtype in (BF16, F32):
        for b, r in ((bias, residual), (None, None)):
            if act == "relu" and r is not None:
                continue                                       # (a sum that is not a grid value)
            got = _run_linear(ia, x, w, b, r, act, dtype, F)
            _check(got, v + b.double() if b is not None else v, act, r.double() if r is not None else None)


@pytest.mark.parametrize("T", [9, 16, 17, 63, 129, 255, 256, 257])
@pytest.mark.parametrize("K,F", [(8, 1), (64, 37), (72, 300), (512, 24), (1000, 129), (4104, 30)])
@pytest.mark.parametrize("act", ["none", "silu", "swiglu"])
def test_linear_of_small_layers(ia, T, K, F, act):
    """Small layers of more tokens, eight at a time, and the sizes from which the tensor cores take over."""
    x, w, bias, residual = _linear_inputs(T, K, F, act, seed=T + K + F)
    v = x.double() @ w.double().t()
    _check(_run_linear(ia, x, w, bias, residual, act, BF16, F), v + bias.double(), act, residual.double())
    _check(_run_linear(ia, x, w, None, None, act, F32, F), v, act)


@pytest.mark.parametrize("T,K,F,act", [(1, 8192, 8192, "none"), (2, 8192, 1000, "swiglu"), (3, 4096, 2800, "gelu"),
                                       (4, 4096, 3000, "none"), (6, 2048, 2900, "none"), (8, 2048, 3000, "silu")])
def test_linear_few_tokens_gaussian(ia, T, K, F, act):
    """Both sides of the sizes up to which the tensor cores are left out; in place, and NaN and
    infinity in one token's row leave the others as they are."""
    x, w, bias, residual = _linear_inputs(T, K, F, act, seed=T + K + F, grid=False)
    v = x.double() @ w.double().t() + bias.double()
    mags = x.double().abs() @ w.double().abs().t() + bias.double().abs()
    _check(_run_linear(ia, x, w, bias, residual, act, F32, F), v, act, residual.double(), sum_slack=K * 2.0 ** -23 * mags)
    dev = [t.cuda() for t in (x, w, bias)]
    out = residual.cuda()
    ia.inkattn_linear(ia.linear_params(x=dev[0], w=dev[1], out=out, act=act, bias=dev[2], residual=out))
    torch.cuda.synchronize()
    _check(out, v, act, residual.double(), sum_slack=K * 2.0 ** -23 * mags)
    if T > 1:
        x[T - 1, 3], x[T - 1, 7] = float("nan"), float("inf")
        dirty = _run_linear(ia, x, w, bias, residual, act, BF16, F)
        assert torch.equal(dirty[:T - 1], out[:T - 1]) and bool(torch.isnan(dirty[T - 1]).all())


def test_linear_no_tokens_and_repeatability(ia):
    x, w, bias, residual = [t.cuda() for t in _linear_inputs(64, 4096, 512, "none", seed=9, grid=False)]
    empty = torch.empty((0, 512), dtype=BF16, device="cuda")
    assert ia.inkattn_linear(ia.linear_params(x=x[:0], w=w, out=empty)) == 0
    outs = []
    for _ in range(3):
        out = torch.empty((64, 512), dtype=F32, device="cuda")
        ia.inkattn_linear(ia.linear_params(x=x, w=w, bias=bias, residual=residual, out=out))
        outs.append(out)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


# ---------------------------------------------------------------- grouped products

def _grouped(ia, counts, K, F, act="none", gather=True, dtype=BF16, seed=0, bias=True, spare=3, N_x=0):
    g = torch.Generator().manual_seed(seed)
    E, M = len(counts), int(sum(counts))
    rows = 2 * F if act == "swiglu" else F
    N_x = N_x or (max(1, M // 2) if gather else M + spare)
    x = _grid((N_x, K), g, -8, 8, 1 / 8)
    w = _grid((E, rows, K), g, -8, 8, 1 / 64)
    b = _grid((E, rows), g, -512, 512, 2.0 ** -9, F32) if bias else None
    offs = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=I32)
    tok = torch.randint(0, N_x, (M + spare,), generator=g).to(I32) if gather else None
    out = torch.full((M + spare, F), 7.0, dtype=dtype, device="cuda")
    status = torch.zeros(1, dtype=I32, device="cuda")
    dev = [None if t is None else t.cuda() for t in (x, w, b, offs, tok)]
    p = ia.grouped_linear_params(x=dev[0], w=dev[1], bias=dev[2], expert_offsets=dev[3], row_token=dev[4], out=out,
                                 act=act, dev_status=status)
    ia.inkattn_grouped_linear(p)
    torch.cuda.synchronize()
    assert int(status) == 0
    assert bool((out[M:] == 7).all())                       # rows behind the last expert's
    for e in range(E):
        lo, hi = int(offs[e]), int(offs[e + 1])
        xe = x[tok[lo:hi].long()] if gather else x[lo:hi]
        v = xe.double() @ w[e].double().t()
        if b is not None:
            v = v + b[e].double()
        _check(out[lo:hi], v, act)


COUNTS = {
    "one expert, one row": [1],
    "rows of one to three": [1, 0, 2, 3, 0, 1],
    "around the tile": [31, 32, 33, 0, 127, 128, 129, 1],
    "several tiles": [0, 257, 600, 5, 0],
    "all rows to one": [0, 0, 300, 0],
    "no rows": [0, 0, 0],
}


@pytest.mark.parametrize("name", list(COUNTS))
@pytest.mark.parametrize("gather", [True, False])
def test_grouped_row_counts(ia, name, gather):
    _grouped(ia, COUNTS[name], K=136, F=200, gather=gather, seed=len(name))
    _grouped(ia, COUNTS[name], K=512, F=272, gather=gather, act="swiglu", seed=len(name))


@pytest.mark.parametrize("K,F", [(8, 1), (64, 33), (72, 255), (1000, 257), (2048, 600)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_grouped_sizes(ia, K, F, dtype):
    _grouped(ia, [3, 70, 0, 9, 200], K=K, F=F, dtype=dtype, seed=K + F)
    _grouped(ia, [3, 70, 0, 9, 200], K=K, F=F, dtype=dtype, seed=K + F, gather=False, act="silu", bias=False)
    _grouped(ia, [3, 70, 0, 9, 200], K=K, F=F, dtype=dtype, seed=K, act="swiglu")


def test_grouped_many_experts(ia):
    g = np.random.default_rng(4)
    counts = g.integers(0, 12, size=1024).tolist()
    _grouped(ia, counts, K=64, F=136, seed=4)
    _grouped(ia, [int(c) for c in g.integers(0, 60, size=300)], K=256, F=128, act="swiglu", seed=5)


def test_grouped_split_over_k(ia):
    """Few items and a long K: the K range is split over a cluster."""
    for counts in ([1], [5, 0, 2], [40], [0, 260]):
        for F in (8, 100, 256, 400):
            _grouped(ia, counts, K=4096, F=F, seed=F)
        _grouped(ia, counts, K=4096, F=320, act="swiglu", seed=6, dtype=F32)
        _grouped(ia, counts, K=4096, F=101, act="gelu", seed=7, gather=False)


def test_grouped_repeated_row_token(ia):
    """Every row of every expert reads the same row of x."""
    _grouped(ia, [40, 3, 90], K=128, F=128, N_x=1, seed=8)


def test_grouped_bad_indices_are_flagged_and_left(ia):
    """A row_token out of range and an expert with bad offsets: flagged, their rows untouched,
    the others computed.  (The kernel checks both before it uses them.)"""
    g = torch.Generator().manual_seed(1)
    K, F, M = 64, 128, 50
    x, w = _grid((10, K), g, -8, 8, 1 / 8), _grid((2, F, K), g, -8, 8, 1 / 64)
    tok = torch.randint(0, 10, (M,), generator=g).to(I32)
    tok[3], tok[40] = 10, -1
    offs = torch.tensor([0, 20, M], dtype=I32)

    def go(tok, offs):
        out = torch.full((M, F), 7.0, dtype=BF16, device="cuda")
        status = torch.zeros(1, dtype=I32, device="cuda")
        dev = [t.cuda() for t in (x, w, offs, tok)]
        ia.inkattn_grouped_linear(ia.grouped_linear_params(x=dev[0], w=dev[1], expert_offsets=dev[2],
                                                           row_token=dev[3], out=out, dev_status=status))
        torch.cuda.synchronize()
        return out.cpu(), int(status)

    out, status = go(tok, offs)
    assert status == ia.INKATTN_ERR_DEVICE_BOUNDS
    for i in range(M):
        if i in (3, 40):
            assert bool((out[i] == 7).all())
        else:
            v = x[int(tok[i])].double() @ w[0 if i < 20 else 1].double().t()
            assert torch.equal(out[i], v.to(F32).to(BF16))
    good = tok.clamp(0, 9)
    for bad in ([0, 20, M + 1], [0, -4, M], [21, 20, M]):
        out, status = go(good, torch.tensor(bad, dtype=I32))
        assert status == ia.INKATTN_ERR_DEVICE_BOUNDS, bad
        for e in range(2):
            lo, hi = bad[e], bad[e + 1]
            if not (0 <= lo <= hi <= M):
                continue
            for i in range(lo, hi):
                assert torch.equal(out[i], (x[int(good[i])].double() @ w[e].double().t()).to(F32).to(BF16))
        covered = {i for e in range(2) if 0 <= bad[e] <= bad[e + 1] <= M for i in range(bad[e], bad[e + 1])}
        assert all(bool((out[i] == 7).all()) for i in range(M) if i not in covered)


def test_grouped_overlapping_experts_are_flagged_and_left(ia):
    """Offsets that go back: of experts 0..30, 30..10, 10..50, 50..60 the second decreases and the
    third reaches into the first one's rows; the first and the last are computed.  Many such
    experts must not make more work than the launch was sized for."""
    g = torch.Generator().manual_seed(6)
    K, F, M = 1024, 128, 60
    for offsets, good in (([0, 30, 10, 50, 60], [(0, 0, 30), (3, 50, 60)]),
                          ([0, M] * 40, [(0, 0, M)])):
        E = len(offsets) - 1
        x, w = _grid((M, K), g, -8, 8, 1 / 8), _grid((E, F, K), g, -8, 8, 1 / 64)
        out = torch.full((M, F), 7.0, dtype=BF16, device="cuda")
        status = torch.zeros(1, dtype=I32, device="cuda")
        dev = [t.cuda() for t in (x, w, torch.tensor(offsets, dtype=I32))]
        ia.inkattn_grouped_linear(ia.grouped_linear_params(x=dev[0], w=dev[1], expert_offsets=dev[2], out=out,
                                                           dev_status=status))
        torch.cuda.synchronize()
        assert int(status) == ia.INKATTN_ERR_DEVICE_BOUNDS
        want = torch.full((M, F), 7.0, dtype=BF16)
        for e, lo, hi in good:
            want[lo:hi] = (x[lo:hi].double() @ w[e].double().t()).to(F32).to(BF16)
        assert torch.equal(out.cpu(), want)


@pytest.mark.parametrize("E", [31, 32, 33, 255, 256, 257, 600, 1024])
@pytest.mark.parametrize("bad", [False, True])
def test_grouped_tiles_of_many_experts(ia, E, bad):
    """Offsets read by one warp or by eight, once or in rounds: every expert at its rows; with two
    impossible offsets, the experts beside them are flagged and left and all others computed."""
    g = torch.Generator().manual_seed(E)
    K, F = 64, 40
    counts = torch.randint(0, 4, (E,), generator=g)
    counts[E // 3] = 300                                       # several tiles
    offs = torch.cat([torch.zeros(1, dtype=torch.long), counts.cumsum(0)]).to(I32)
    M = int(offs[-1])
    x, w = _grid((M, K), g, -8, 8, 1 / 8), _grid((E, F, K), g, -8, 8, 1 / 64)
    if bad:
        offs[E // 2], offs[E - 3] = -5, M + 1
    owner = torch.full((M,), -1)
    reached = 0
    for e in range(E):
        lo, hi = int(offs[e]), int(offs[e + 1])
        if 0 <= lo <= hi <= M:
            if lo >= reached:
                owner[lo:hi] = e
            reached = max(reached, hi)
    out = torch.full((M, F), 7.0, dtype=BF16, device="cuda")
    status = torch.zeros(1, dtype=I32, device="cuda")
    ia.inkattn_grouped_linear(ia.grouped_linear_params(x=x.cuda(), w=w.cuda(), expert_offsets=offs.cuda(), out=out,
                                                       dev_status=status))
    torch.cuda.synchronize()
    assert int(status) == (ia.INKATTN_ERR_DEVICE_BOUNDS if bad else 0)
    want = torch.einsum("mk,mfk->mf", x.double(), w.double()[owner.clamp(min=0)]).to(F32).to(BF16)
    want[owner < 0] = 7.0
    assert torch.equal(out.cpu(), want)


# ---------------------------------------------------------------- router and sum

def _route(ia, logits, S, k, score="sigmoid", scale=1.0):
    T, E = logits.shape[0], logits.shape[1] - S
    o = {"topk_ids": torch.full((T, k), -7, dtype=I32), "weights": torch.full((T, k + S), -7.0),
         "expert_offsets": torch.full((E + 1,), -7, dtype=I32), "row_token": torch.full((T * k,), -7, dtype=I32),
         "token_rows": torch.full((T, k), -7, dtype=I32)}
    o = {n: t.cuda() for n, t in o.items()}
    dev = logits.cuda()
    p = ia.route_params(logits=dev, n_shared=S, score=score, scale=scale, **o)
    n = ia.inkattn_route_workspace_bytes(p)
    ws = torch.full((n,), 0xAB, dtype=torch.uint8, device="cuda") if n else None
    ia.inkattn_route(p, ws)
    torch.cuda.synchronize()
    return {n: t.cpu() for n, t in o.items()}


def _check_route(got, logits, S, k, score, scale=1.0):
    T, E = logits.shape[0], logits.shape[1] - S
    clean = torch.where(torch.isnan(logits), torch.full_like(logits, -float("inf")), logits).double()
    best = torch.sort(clean[:, :E], dim=1, descending=True, stable=True)
    ids = best.indices[:, :k]
    assert torch.equal(got["topk_ids"].long(), ids)
    counts = torch.bincount(ids.reshape(-1), minlength=E)
    assert torch.equal(got["expert_offsets"].long(), torch.cat([torch.zeros(1, dtype=torch.long), counts.cumsum(0)]))
    order = torch.sort(ids.reshape(-1), stable=True).indices
    assert torch.equal(got["row_token"].long(), order // k)
    rows = torch.empty_like(order)
    rows[order] = torch.arange(T * k)
    assert torch.equal(got["token_rows"].long().reshape(-1), rows)
    z = torch.cat([best.values[:, :k], clean[:, E:]], 1)
    if score == "sigmoid":
        s = torch.sigmoid(z)
    else:
        m = z.amax(1, keepdim=True)
        s = torch.where(z == m, torch.ones_like(z), torch.exp(z - m))
        s[z == -float("inf")] = 0.0
    total = s.sum(1, keepdim=True)
    w = torch.where(total > 0, scale * s / total, torch.zeros_like(s))
    # Units of 2^-23: expf 2; its argument is one fp32 subtraction l - m, off by 2^-24 |l - m|, with m
    # the largest logit (sigmoid: or 0, if that is less); 1 + e, the quotients and the products one
    # each; the sum of at most 32 terms 5 levels deep: 16 + |l - m| in all.  Below 2^-126 values may
    # be flushed.
    m = z.amax(1, keepdim=True)
    if score == "sigmoid":
        m = m.clamp(max=0.0)
    arg = (z - m).abs().nan_to_num(0.0, 0.0, 0.0)
    err = (got["weights"].double() - w).abs()
    assert bool((err <= (16 + arg) * 2.0 ** -23 * w.abs() + abs(scale) * 2.0 ** -125).all()), float(err.max())


@pytest.mark.parametrize("T,E,S,k", [(1, 1, 0, 1), (1, 256, 2, 6), (2, 2, 1, 2), (5, 16, 16, 16), (31, 33, 0, 3),
                                     (288, 256, 2, 6), (300, 64, 1, 8), (683, 256, 2, 6), (700, 200, 0, 6), (1023, 1024, 1, 16), (1024, 60, 2, 6), (1025, 60, 2, 6),
                                     (1500, 1024, 3, 4), (4097, 129, 2, 1), (9000, 384, 2, 8), (20001, 256, 2, 6), (200000, 20, 0, 2)])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_route(ia, T, E, S, k, score):
    g = torch.Generator().manual_seed(T + E)
    logits = torch.randn((T, E + S), generator=g) * 2
    _check_route(_route(ia, logits, S, k, score), logits, S, k, score)
    tied = (logits * 2).round() / 2                          # many equal logits, -0 among them
    tied[tied == 0] *= torch.where(torch.rand((T, E + S), generator=g) < 0.5, -1.0, 1.0)[tied == 0]
    _check_route(_route(ia, tied, S, k, score, scale=2.5), tied, S, k, score, scale=2.5)


@pytest.mark.parametrize("T,E,S,k", [(500, 64, 1, 6), (501, 64, 1, 6), (375, 300, 0, 8), (376, 300, 0, 8), (1000, 384, 2, 3),
                                     (1001, 385, 2, 3), (1024, 20, 0, 2), (1025, 20, 0, 2), (1024, 6, 1, 1), (700, 513, 0, 4),
                                     (701, 1000, 1, 5), (33, 1024, 16, 16)])
def test_route_around_one_block(ia, T, E, S, k):
    """Batches that one block places, just not any more, and few choices of many tokens."""
    g = torch.Generator().manual_seed(T + E)
    logits = torch.randn((T, E + S), generator=g)
    logits[::3] = torch.round(logits[::3] * 2) / 2             # ties
    _check_route(_route(ia, logits, S, k), logits, S, k, "sigmoid")


@pytest.mark.parametrize("T", [7, 1000])
def test_route_same_choice_for_every_token(ia, T):
    """Every token takes the same experts: all rows in k groups."""
    logits = torch.zeros((T, 96))
    _check_route(_route(ia, logits, 0, 6), logits, 0, 6, "sigmoid")
    logits[:, [90, 5, 17]] = 3.0
    _check_route(_route(ia, logits, 0, 3), logits, 0, 3, "sigmoid")


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_route_infinities_and_nan(ia, score):
    """-infinity, NaN, +infinity and huge logits; a token whose every logit is -infinity gets
    zero weights and the lowest indices."""
    inf, nan = float("inf"), float("nan")
    E, S, k = 40, 2, 4
    logits = torch.randn((8, E + S), generator=torch.Generator().manual_seed(2))
    logits[0, :] = -inf
    logits[1, :E] = nan
    logits[2, 3], logits[2, 30] = inf, nan
    logits[3, :E - 2] = -inf
    logits[4, :] = -300.0
    logits[5, 7] = 3e38
    logits[6, E:] = nan
    logits[7, :] = nan
    got = _route(ia, logits, S, k, score)
    _check_route(got, logits, S, k, score)
    assert got["topk_ids"][0].tolist() == [0, 1, 2, 3] and bool((got["weights"][0] == 0).all())


def test_route_no_tokens(ia):
    got = _route(ia, torch.zeros((0, 12)), 2, 3)
    assert got["expert_offsets"].tolist() == [0] * 11


@pytest.mark.parametrize("T,k,S,F", [(1, 1, 0, 8), (1, 6, 2, 8192), (3, 8, 2, 1032), (9, 16, 16, 264), (100, 3, 1, 2056),
                                     (700, 6, 0, 520)])
def test_expert_combine(ia, T, k, S, F):
    g = torch.Generator().manual_seed(T + F)
    M = T * k
    y, sh = torch.randn((M, F), generator=g).to(BF16), torch.randn((S, T, F), generator=g).to(BF16)
    w = torch.randn((T, k + S), generator=g)
    rows = torch.randperm(M, generator=g).to(I32).reshape(T, k)
    rows[0, 0] = -1                                          # a dropped row
    out = torch.full((T + 1, F), 7.0, dtype=BF16, device="cuda")
    status = torch.zeros(1, dtype=I32, device="cuda")
    dev = [t.cuda() for t in (y, sh, w, rows)]
    ia.inkattn_expert_combine(ia.expert_combine_params(y=dev[0], shared=dev[1] if S else None, weights=dev[2],
                                                       token_rows=dev[3], out=out[:T], dev_status=status))
    torch.cuda.synchronize()
    assert int(status) == 0 and bool((out[T] == 7).all())
    picked = torch.where((rows >= 0)[..., None], y[rows.clamp(min=0).long()].double(), torch.zeros(1, dtype=F64))
    terms = torch.cat([picked * w[:, :k, None].double(), sh.double().transpose(0, 1) * w[:, k:, None].double()], 1)
    want, mags = terms.sum(1), terms.abs().sum(1)
    slack = (k + S) * 2.0 ** -24 * mags                      # one rounding a term
    err = (out[:T].cpu().double() - want).abs()
    assert bool((err <= slack + 2.0 ** -8 * (want.abs() + slack) + 2.0 ** -126).all())


def test_expert_combine_bad_rows_and_no_nan_from_dropped_ones(ia):
    T, k, F = 3, 2, 16
    y = torch.full((4, F), float("nan"), dtype=BF16)
    y[1] = 2.0
    rows = torch.tensor([[1, -1], [4, 1], [-2, -1]], dtype=I32)
    w = torch.full((T, k), 0.5)
    w[0, 1] = float("nan")                                    # the weight of a dropped row
    out = torch.empty((T, F), dtype=BF16, device="cuda")
    status = torch.zeros(1, dtype=I32, device="cuda")
    dev = [t.cuda() for t in (y, w, rows)]
    ia.inkattn_expert_combine(ia.expert_combine_params(y=dev[0], weights=dev[1], token_rows=dev[2], out=out,
                                                       dev_status=status))
    torch.cuda.synchronize()
    assert int(status) == ia.INKATTN_ERR_DEVICE_BOUNDS
    assert torch.equal(out.cpu().float(), torch.tensor([1.0, 1.0, 0.0])[:, None].expand(T, F))


@pytest.mark.parametrize("T,k,S,F", [(2501, 1, 0, 1000), (2500, 1, 1, 1024), (2497, 2, 0, 520), (2463, 3, 1, 1032),
                                     (2600, 2, 1, 2056), (40001, 1, 0, 64), (40000, 2, 0, 56), (20003, 3, 1, 136),
                                     (77777, 1, 1, 8), (50001, 7, 2, 24)])
def test_expert_combine_of_many_tokens(ia, T, k, S, F):
    """More blocks than run at once: several tokens a thread where they have few rows, and several
    a block where the rows are narrow; with dropped and bad rows among them."""
    g = torch.Generator(device="cuda").manual_seed(T + F)
    M = T * k
    y, sh = (torch.randn(s, generator=g, device="cuda").to(BF16) for s in ((M, F), (S, T, F)))
    w = torch.randn((T, k + S), generator=g, device="cuda")
    rows = torch.randperm(M, generator=g, device="cuda").to(I32).reshape(T, k)
    rows[::7, 0] = -1
    for bad in (False, True):
        if bad:
            rows[T - 1, 0], rows[5, k - 1] = M, -2
        out = torch.full((T + 1, F), 7.0, dtype=BF16, device="cuda")
        status = torch.zeros(1, dtype=I32, device="cuda")
        ia.inkattn_expert_combine(ia.expert_combine_params(y=y, shared=sh if S else None, weights=w, token_rows=rows,
                                                           out=out[:T], dev_status=status))
        torch.cuda.synchronize()
        assert int(status) == (ia.INKATTN_ERR_DEVICE_BOUNDS if bad else 0) and bool((out[T] == 7).all())
        want, mags = torch.zeros((T, F), dtype=F64, device="cuda"), torch.zeros((T, F), dtype=F64, device="cuda")
        for j in range(k + S):
            if j < k:
                r = rows[:, j].long()
                term = torch.where(((r >= 0) & (r < M))[:, None], y[r.clamp(0, M - 1)].double() * w[:, j, None].double(), 0.0)
            else:
                term = sh[j - k].double() * w[:, j, None].double()
            want, mags = want + term, mags + term.abs()
        slack = (k + S) * 2.0 ** -24 * mags                  # one rounding a term
        err = (out[:T].double() - want).abs()
        assert bool((err <= slack + 2.0 ** -8 * (want.abs() + slack) + 2.0 ** -126).all())
