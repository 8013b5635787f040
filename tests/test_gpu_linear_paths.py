"""The tensor-core kernel behind inkattn_linear and inkattn_grouped_linear (k_linear), path by path, at
sizes that really reach it.  inkattn_linear gives few tokens and small layers to k_linear_few (always
up to 2 tokens; up to 256 tokens where the layer is small enough), so every test here names the
kernel that it is about and asserts, from a captured graph, that the call launches it; more than
256 tokens never go to k_linear_few, and neither do grouped products.

Whether the K range is split shows in the grid: two CTAs for each item (256 weight rows, 128 for
SWIGLU, times a tile of at least 32 tokens) and each part of K, as long as these are fewer than the SMs."""
import os
import re
import subprocess
import sys
import warnings

import pytest
import torch

from test_gpu_layer_products import BF16, F32, F64, HALF_STEP, I32, _act64, _grid, _linear_inputs, _run_linear

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
ACTS = {"none": 0, "relu": 1, "gelu": 2, "silu": 3, "swiglu": 4}
U = 2.0 ** -24


@pytest.fixture(scope="module")
def ia():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from relative_bias_hybrid_gb300 import build
    build.build()
    import relative_bias_hybrid_gb300.inkattn as ia
    return ia


def launches(call, tmp_path):
    """(mangled kernel name, blocks) of every launch of call, from the graph that it is captured into."""
    graph = torch.cuda.CUDAGraph(keep_graph=True)
    graph.enable_debug_mode()
    with torch.cuda.graph(graph):
        call()
    path = os.path.join(str(tmp_path), f"graph{len(os.listdir(str(tmp_path)))}.dot")
    with warnings.catch_warnings():
        warnings.simplefilter("ignore")                        # (it announces the file)
        graph.debug_dump(path)
    found = re.findall(r"\| (_ZN7inkattn\w+)\\<\\<\\<(\d+),", open(path).read())
    return [(name, int(blocks)) for name, blocks in found]


def is_linear(name, act, dtype, residual):
    return name.startswith(f"_ZN7inkattn8k_linearILi{ACTS[act]}ELb{int(dtype == F32)}ELb{int(residual)}E")


def the_launch(ia, tmp_path, T, K, F, act, dtype, residual):
    """The launch of a linear layer of these sizes: it must be k_linear's kernel for them.  Its blocks."""
    rows = F * (2 if act == "swiglu" else 1)
    x, w, out = (torch.zeros(s, dtype=d, device="cuda") for s, d in
                 (((T, K), BF16), ((rows, K), BF16), ((T, F), dtype)))
    res = torch.zeros((T, F), dtype=BF16, device="cuda") if residual else None
    p = ia.linear_params(x=x, w=w, out=out, act=act, residual=res)
    (name, blocks), = launches(lambda: ia.inkattn_linear(p), tmp_path)
    assert is_linear(name, act, dtype, residual), name
    return blocks


def items(F, act, tiles):
    feat = 128 if act == "swiglu" else 256
    return (F + feat - 1) // feat * tiles


def curve_slack(v, act, dtype):
    """Absolute error of the curve at an exact argument v, before the output's rounding.  In units of 2^-24.
    fp32: SILU 11 of the value and GELU 18 + 1.25 v^2 (see test_gpu_linear_curves.py).
    bf16, SILU v / (1 + 2^(-v log2 e)): the exponent has two roundings (2 |v|), 2^x is within 2^-22 (4), the
    sum and the product round once each (2), the reciprocal is within a step (2): 8 + 2 |v| of the value,
    and below 2^-126 it may be 0.  bf16, GELU v h or v - v h, absolute in h: the formula (2.5 / 2); t = 1 / (1 +
    c |v|) within 3 of itself, times 3.5 (the formula's slope against t) times h <= 1/2 (5.3); five
    steps of values up to 0.73 (3.7); 2^x 4 h + 2.5 v^2 / 2 h (2.5); the product (0.5): 14 |v|."""
    if act == "silu":
        y = v * torch.sigmoid(v)
        return 11 * U * y.abs() + 2.0 ** -141 if dtype == F32 else (8 + 2 * v.abs()) * U * y.abs() + 2.0 ** -119
    if act == "gelu":
        y = _act64(v, "gelu")
        return (18 + 1.25 * v * v) * U * y.abs() + 2.0 ** -141 if dtype == F32 else 14 * U * v.abs()
    if act == "swiglu":
        a, b = v.chunk(2, dim=-1)
        return (curve_slack(a, "silu", dtype) + U * (a * torch.sigmoid(a)).abs()) * b.abs() + 2.0 ** -141
    return torch.zeros_like(v)


def check(got, v, act, residual=None):
    """got against act(v) + residual at the exact argument v: bit for bit where the curve is straight."""
    y, slack = _act64(v, act), curve_slack(v, act, got.dtype)
    if residual is not None:
        y = y + residual
        slack = slack + U * (y.abs() + slack)                  # the fp32 addition
    got = got.cpu()
    if act in ("none", "relu"):
        assert torch.equal(got, y.to(F32).to(got.dtype))
        return
    over = (got.to(F64) - y).abs() - (slack + HALF_STEP[got.dtype] * (y.abs() + slack) + 2.0 ** -134)
    assert bool((over <= 0).all()), float(over.max())


# ---------------------------------------------------------------- infinite sums, wide arguments

# More than 256 tokens: k_linear.  The short K cannot be split (fewer than four steps of 64); the long
# one of few items is.  64 tokens of 256 features read 4 MB of weights eight times: far above what
# k_linear_few takes for more than eight tokens.
INF_SHAPES = [(300, 64, 24, False), (300, 64, 27, False), (300, 64, 260, False), (64, 8192, 256, True),
              (64, 8192, 253, True)]


@pytest.mark.parametrize("act", list(ACTS))
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("with_residual", [False, True])
@pytest.mark.parametrize("T,K,F,split", INF_SHAPES)
def test_infinite_sums(ia, tmp_path, act, dtype, with_residual, T, K, F, split):
    """A sum of +infinity or -infinity takes the formula's value (infinity, 0 or NaN) through the unsplit
    epilogue and the split's join, with stores of whole words and single values; the features beside
    it keep theirs."""
    blocks = the_launch(ia, tmp_path, T, K, F, act, dtype, with_residual)
    if split:
        assert blocks > 2 * items(F, act, 2)                   # (64 tokens are two tiles at most)
    inf, rows = float("inf"), F * (2 if act == "swiglu" else 1)
    x, w = torch.ones((T, K), dtype=BF16), torch.zeros((rows, K), dtype=BF16)
    bias = torch.ones(rows, dtype=F32)
    bias[:6] = torch.tensor([inf, -inf, float("nan"), 3.0e38, -3.0e38, 0.0])
    if act == "swiglu":
        bias[F + 6:F + 8] = torch.tensor([inf, -inf])
    residual = torch.full((T, F), 0.5, dtype=BF16) if with_residual else None
    got = _run_linear(ia, x, w, bias, residual, act, dtype, F).cpu()
    want = _act64(bias.double().expand(T, rows), act) + (0.5 if with_residual else 0.0)
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(torch.isinf(got), torch.isinf(want.to(dtype)))
    assert torch.equal(got[torch.isinf(got)].double(), want.to(dtype)[torch.isinf(got)].double())
    live = torch.isfinite(want) & torch.isfinite(got.double())
    # half a step, and the curves at 0, at 1 and at their limits: at 1, 14 units of 2^-24 (gelu) of at least
    # 0.73, 11 (silu) and 12 (swiglu) of the value, and the residual's rounding: under 24 units in all
    slack = (HALF_STEP[dtype] + 24 * U) * want.abs() + 1e-36
    assert bool(((got.double() - want).abs() <= slack)[live].all())


@pytest.mark.parametrize("act", ["relu", "gelu", "silu", "swiglu"])
@pytest.mark.parametrize("T,split", [(300, False), (32, True)])
def test_activations_of_wide_arguments(ia, tmp_path, act, T, split):
    """Arguments from -60 to 60, and NaN, through an identity weight of 2568 features: 11 blocks of
    them (SWIGLU 21), which 32 tokens, one tile, split over K."""
    v = torch.arange(-1280, 1281).double() * (60.0 / 1280)
    K = 8 * ((v.numel() + 7) // 8)
    x = torch.zeros((T, K), dtype=BF16)
    x[:, :v.numel()] = v.to(BF16)                      # (the arguments are what x holds)
    x[1, 5] = float("nan")
    w = torch.eye(K, dtype=BF16)
    if act == "swiglu":
        w = torch.cat([w, w.flip(0)])
    for dtype in (BF16, F32):
        blocks = the_launch(ia, tmp_path, T, K, K, act, dtype, False)
        if split:
            assert blocks > 2 * items(K, act, 1)
        got = _run_linear(ia, x, w, None, None, act, dtype, K)
        rows = torch.tensor([0, 2, T // 2, T - 1])
        a = x[rows].double()
        check(got[rows.cuda()], torch.cat([a, a.flip(1)], 1) if act == "swiglu" else a, act)
        assert bool(torch.isnan(got[1]).all())         # NaN times a zero weight is a NaN everywhere


# ---------------------------------------------------------------- residuals

# 5000 tokens are 20 tiles of at most 256: 80 items of 1021 features, 160 of 2000, 100 of 600 with SWIGLU;
# fp32 outputs, in tiles of 160: 128 items of 1021.  More than the 76 pairs of SMs, so that pairs
# take a second item, whose first residual values are requested while the first is stored.
@pytest.mark.parametrize("T,K,F,act,dtype,in_place", [
    (5000, 128, 1021, "none", BF16, True), (5000, 128, 1021, "none", BF16, False), (5000, 72, 2000, "none", BF16, True),
    (5000, 200, 2000, "none", BF16, False), (5003, 128, 600, "swiglu", BF16, True), (5003, 128, 599, "swiglu", BF16, True),
    (5003, 136, 599, "swiglu", BF16, False), (5000, 64, 1024, "gelu", BF16, True), (5000, 64, 1021, "silu", BF16, False),
    (5000, 600, 1021, "none", F32, False), (5003, 136, 599, "swiglu", F32, False), (5000, 64, 1024, "gelu", F32, False),
    (300, 64, 33, "none", BF16, True), (300, 128, 1024, "none", BF16, True), (321, 128, 261, "swiglu", BF16, True)])
def test_residual_of_several_items(ia, tmp_path, T, K, F, act, dtype, in_place):
    """A residual through the unsplit epilogue, which requests its values a block and an item ahead: also
    where the output is the residual array itself, so that requested values lie beside stored ones."""
    blocks = the_launch(ia, tmp_path, T, K, F, act, dtype, True)
    if T >= 5000:
        assert blocks < 2 * items(F, act, (T + (159 if dtype == F32 else 255)) // (160 if dtype == F32 else 256))
    x, w, bias, residual = _linear_inputs(T, K, F, act, seed=T + K + F)
    v = x.double() @ w.double().t() + bias.double()
    if in_place:
        dev = [t.cuda() for t in (x, w, bias, residual)]
        ia.inkattn_linear(ia.linear_params(x=dev[0], w=dev[1], bias=dev[2], residual=dev[3], out=dev[3], act=act))
        torch.cuda.synchronize()
        check(dev[3], v, act, residual.double())
    else:
        check(_run_linear(ia, x, w, bias, residual, act, dtype, F), v, act, residual.double())


@pytest.mark.parametrize("T,K,F", [(700, 128, 264), (700, 128, 261)])
def test_in_place_residual_and_infinities(ia, tmp_path, T, K, F):
    """out == residual; infinities and NaN of a token or a residual stay in their own place."""
    the_launch(ia, tmp_path, T, K, F, "none", BF16, True)
    x, w, bias, residual = _linear_inputs(T, K, F, "none", seed=3)
    x[5, 7], x[300, 1], x[699, 3] = float("inf"), float("nan"), -float("inf")
    residual[44, 7], residual[45, F - 1], residual[260, 0] = float("inf"), float("nan"), -float("inf")
    dev = [t.cuda() for t in (x, w, bias, residual)]
    ia.inkattn_linear(ia.linear_params(x=dev[0], w=dev[1], bias=dev[2], residual=dev[3], out=dev[3]))
    torch.cuda.synchronize()
    want = (x.double() @ w.double().t() + bias.double() + residual.double()).to(F32).to(BF16)
    got = dev[3].cpu()
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(torch.nan_to_num(got.float()), torch.nan_to_num(want.float()))


# ---------------------------------------------------------------- behind other calls

@pytest.mark.parametrize("T,K,split", [(300, 512, False), (64, 2048, True)])
def test_calls_wait_for_the_work_before_them(ia, tmp_path, T, K, split):
    """A product reads what the calls just before it on the stream wrote, over and over: k_linear sets
    itself up, and each of its roles waits, before the kernel in front has finished."""
    blocks = the_launch(ia, tmp_path, T, K, K, "none", BF16, True)
    if split:
        assert blocks > 2 * items(K, "none", 2)
    g = torch.Generator().manual_seed(1)
    eye = torch.eye(K, dtype=BF16, device="cuda")
    a = _grid((T, K), g, -8, 8, 1 / 8).cuda()
    b, first = torch.empty_like(a), a.clone()
    p = [ia.linear_params(x=a, w=eye, out=b), ia.linear_params(x=b, w=eye, out=a, residual=b)]
    for _ in range(12):                                        # a <- 2 a, exactly, each round
        ia.inkattn_linear(p[0])
        ia.inkattn_linear(p[1])
    torch.cuda.synchronize()
    assert torch.equal(a.double(), first.double() * 2 ** 12)


def test_kernels_of_every_length_wait_for_each_other(ia, tmp_path):
    """Short kernels that let their successor start early in front of long ones and behind them, on
    the same buffers: k_linear_few doubles four rows, k_linear copies all, the grouped products
    gather them in another order (rows of two experts, whose weights are 1 and 2), the weighted sum
    brings them back halved where they were doubled."""
    T, K = 300, 512
    g = torch.Generator().manual_seed(2)
    eye = torch.eye(K, dtype=BF16, device="cuda")
    a = _grid((T, K), g, -8, 8, 1 / 8).cuda()
    want = a.clone()
    few, b = torch.empty((4, K), dtype=BF16, device="cuda"), torch.empty_like(a)
    rows = torch.empty_like(a)
    order = torch.randperm(T, generator=g)
    place = torch.empty_like(order)
    place[order] = torch.arange(T)
    tok, place = order.to(I32).cuda(), place.to(I32).cuda()[:, None].contiguous()
    offs = torch.tensor([0, 131, T], dtype=I32, device="cuda")
    w2 = torch.stack([eye, 2 * eye])
    weights = torch.where(place < 131, 1.0, 0.5).contiguous()
    calls = [(ia.inkattn_linear, ia.linear_params(x=a[:4], w=eye, out=few)),
             (ia.inkattn_linear, ia.linear_params(x=few, w=eye, out=a[:4], residual=few)),
             (ia.inkattn_linear, ia.linear_params(x=a, w=eye, out=b)),
             (ia.inkattn_grouped_linear, ia.grouped_linear_params(x=b, w=w2, expert_offsets=offs, row_token=tok, out=rows)),
             (ia.inkattn_expert_combine, ia.expert_combine_params(y=rows, weights=weights, token_rows=place, out=a))]

    def once():
        for call, p in calls:
            call(p)

    names = [n for n, _ in launches(once, tmp_path)]
    assert ["k_linear_few" in n for n in names] == [True, True, False, False, False]
    assert is_linear(names[2], "none", BF16, False) and is_linear(names[3], "none", BF16, False)
    for _ in range(10):
        once()
    torch.cuda.synchronize()
    want[:4] *= 2 ** 10
    assert torch.equal(a, want)


FIRST = r"""
import sys
sys.path.insert(0, sys.argv[1])
import torch
import relative_bias_hybrid_gb300.inkattn as ia
BF, I = torch.bfloat16, torch.int32
T, K, E = 300, 64, 4
g = torch.Generator().manual_seed(0)
x = (torch.randint(-8, 9, (T, K), generator=g) / 8).to(BF).cuda()
eye = torch.eye(K, dtype=BF, device="cuda")
r = dict(topk_ids=torch.empty((T, 1), dtype=I, device="cuda"), weights=torch.empty((T, 1), device="cuda"),
         expert_offsets=torch.empty(E + 1, dtype=I, device="cuda"), row_token=torch.empty(T, dtype=I, device="cuda"),
         token_rows=torch.empty((T, 1), dtype=I, device="cuda"))
logits = torch.randn((T, E), generator=g).cuda()
y, rows, back = (torch.zeros_like(x) for _ in range(3))
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    ia.inkattn_linear(ia.linear_params(x=x, w=eye, out=y))
    ia.inkattn_route(ia.route_params(logits=logits, **r))
    ia.inkattn_grouped_linear(ia.grouped_linear_params(x=y, w=eye.expand(E, K, K).contiguous(), out=rows,
                              expert_offsets=r["expert_offsets"], row_token=r["row_token"]))
    ia.inkattn_expert_combine(ia.expert_combine_params(y=rows, weights=r["weights"], token_rows=r["token_rows"], out=back))
assert not bool(back.any())
for _ in range(3):
    back.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(back, x)
print("FIRST CALLS CAPTURED")
"""


def test_first_calls_of_a_process_can_be_captured(ia):
    """What the library asks of the runtime once, it may ask during a capture."""
    r = subprocess.run([sys.executable, "-c", FIRST, ROOT], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "FIRST CALLS CAPTURED" in r.stdout, r.stdout[-2000:] + r.stderr[-4000:]


# ---------------------------------------------------------------- the size of the error

def _norm_error(got, want):
    return float((got.cpu().double() - want).norm() / want.norm())


# k_linear_few with 1, 4 and 16 warps a row (K up to 512; longer; a K of 4096 and more with at most 304
# groups of rows), then k_linear: split, unsplit, and one part of K alone.
@pytest.mark.parametrize("T,K,F,few", [(4, 512, 500, True), (8, 2048, 700, True), (2, 8192, 258, True), (64, 8192, 512, False),
                                       (300, 8192, 2048, False), (700, 1000, 1021, False), (2100, 512, 3000, False)])
def test_error_of_the_whole_output(ia, tmp_path, T, K, F, few):
    """fp32 outputs to 1e-6 of their norm (as rounding to nearest of random sign gives with up to 128 terms
    in a row: 2^-24 / sqrt 3 * sqrt(128 / 2) = 2.8e-7; and the tensor cores' parts of 512: 5e-7 measured where
    they were chosen).  bf16 outputs: what rounding the exact values costs, within a hundredth of it, and
    2e-5 for sums that the tensor cores did not round to nearest (1e-5 at K = 8192)."""
    x, w, _, _ = _linear_inputs(T, K, F, "none", seed=T + K, grid=False)
    want = x.double() @ w.double().t()
    for dtype in (F32, BF16):
        out = torch.empty((T, F), dtype=dtype, device="cuda")
        dev = [x.cuda(), w.cuda()]
        p = ia.linear_params(x=dev[0], w=dev[1], out=out)
        (name, _), = launches(lambda: ia.inkattn_linear(p), tmp_path)
        assert ("k_linear_few" in name) == few
        err = _norm_error(_run_linear(ia, x, w, None, None, "none", dtype, F), want)
        bound = 1e-6 if dtype == F32 else 1.01 * _norm_error(want.to(F32).to(BF16), want) + 2e-5
        assert err <= bound, (err, bound)


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_error_of_grouped_products(ia, gather, dtype):
    """The same bounds, rows of 5 experts, K = 4096."""
    g = torch.Generator().manual_seed(3)
    counts, K, F = [40, 0, 300, 1, 90], 4096, 600
    M = sum(counts)
    x, w = torch.randn((M, K), generator=g).to(BF16), (torch.randn((5, F, K), generator=g) * K ** -0.5).to(BF16)
    tok = torch.randperm(M, generator=g) if gather else torch.arange(M)
    offs = torch.tensor([0, *torch.tensor(counts).cumsum(0).tolist()], dtype=I32)
    out = torch.empty((M, F), dtype=dtype, device="cuda")
    ia.inkattn_grouped_linear(ia.grouped_linear_params(x=x.cuda(), w=w.cuda(), expert_offsets=offs.cuda(), out=out,
                                                       row_token=tok.to(I32).cuda() if gather else None))
    torch.cuda.synchronize()
    want = torch.cat([x[tok[offs[e]:offs[e + 1]]].double() @ w[e].double().t() for e in range(5)])
    err = _norm_error(out, want)
    bound = 1e-6 if dtype == F32 else 1.01 * _norm_error(want.to(F32).to(BF16), want) + 2e-5
    assert err <= bound, (err, bound)


@pytest.mark.parametrize("T,K,F,act,dtype", [(288, 8192, 2048, "none", BF16), (2000, 4096, 1024, "swiglu", BF16),
                                             (300, 4096, 1021, "gelu", F32), (64, 8192, 512, "none", BF16)])
def test_every_call_gives_the_same_bits(ia, T, K, F, act, dtype):
    """Twenty calls, others between them: no sum depends on which CTA came first."""
    x, w, bias, residual = [t.cuda() for t in _linear_inputs(T, K, F, act, seed=9, grid=False)]
    outs = [torch.empty((T, F), dtype=dtype, device="cuda") for _ in range(2)]
    other = torch.empty((40, F), dtype=dtype, device="cuda")
    first = None
    for i in range(20):
        out = outs[i & 1].zero_()
        ia.inkattn_linear(ia.linear_params(x=x, w=w, bias=bias, residual=residual, out=out, act=act))
        ia.inkattn_linear(ia.linear_params(x=x[:40], w=w, bias=bias, out=other, act=act))
        if first is None:
            first = out.clone()
        assert torch.equal(out, first)
