"""The activations of fp32 outputs against 64 bits, to a few units of the last place over the whole
range of their argument, from both kernels behind inkattn_linear and from inkattn_grouped_linear.

The arguments are fp32 values passed through exactly: each is the sum of three bf16 pieces, and a
weight matrix of three identities adds them up again, one nonzero product at a time, so that every
partial sum is an fp32 number."""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF16, F32, I32, F64 = torch.bfloat16, torch.float32, torch.int32, torch.float64
U = 2.0 ** -24                                        # half a step of fp32


@pytest.fixture(scope="module")
def ia():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from relative_bias_hybrid_gb300 import build
    build.build()
    import relative_bias_hybrid_gb300.inkattn as ia
    return ia


def _pieces(v):
    """v (fp32) as [3][n] bf16 whose sum is v exactly."""
    out, rest = [], v.to(F64)
    for _ in range(3):
        out.append(rest.to(F32).to(BF16))
        rest = rest - out[-1].to(F64)
    assert bool((rest == 0).all())
    return torch.stack(out)


def _through(ia, v, act, T, grouped=False):
    """The last of T rows of act over the arguments v (swiglu: gates v, ups v reversed)."""
    n = v.numel()
    assert n % 8 == 0
    x = _pieces(v).reshape(1, -1).expand(T, -1).contiguous().cuda()
    eye = torch.eye(n, dtype=BF16)
    w = torch.cat([eye] * 3, 1)
    if act == "swiglu":
        w = torch.cat([w, w.flip(0)])
    w, out = w.cuda(), torch.empty((T, n), device="cuda")
    if grouped:
        offs = torch.tensor([0, T], dtype=I32, device="cuda")
        ia.inkattn_grouped_linear(ia.grouped_linear_params(x=x, w=w[None], out=out, act=act, expert_offsets=offs))
    else:
        ia.inkattn_linear(ia.linear_params(x=x, w=w, out=out, act=act))
    torch.cuda.synchronize()
    return out[T - 1].cpu().to(F64)


def _silu(v):
    return v * torch.sigmoid(v)


RANGES = [(-103.0, -87.4), (-87.3, -60.0), (-60.0, -20.0), (-20.0, -6.0), (-6.0, -2.0), (-2.0, -1e-3), (1e-3, 2.0),
          (2.0, 90.0)]


def _arguments(lo, hi):
    return torch.linspace(lo, hi, 608, dtype=F64).to(F32)


# 1 token goes to k_linear_few (up to two tokens always do); 300 rows are more than that kernel takes
# (256), and grouped products never go there.
@pytest.mark.parametrize("T,grouped", [(1, False), (300, False), (40, True)])
@pytest.mark.parametrize("lo,hi", RANGES)
def test_silu_of_fp32_outputs(ia, T, grouped, lo, hi):
    """v e / (1 + e) or v / (1 + e) with e = exp(-|v|), in units of 2^-24 of the value: expf is within two
    of its steps (4 units); v e rounds once (1); 1 + e takes over at most half of e's error (2) and
    rounds (1); the reciprocal is within a step (2), the last product half (1): 11.  Below -87.3 e
    itself is subnormal, within 2 * 2^-149, times |v| <= 103: under 2^-141."""
    v = _arguments(lo, hi)
    got, want = _through(ia, v, "silu", T, grouped), _silu(v.to(F64))
    over = (got - want).abs() - (11 * U * want.abs() + 2.0 ** -141)
    assert bool((over <= 0).all()), float((((got - want) / want).abs() / U).max())


@pytest.mark.parametrize("T,grouped", [(1, False), (300, False), (40, True)])
@pytest.mark.parametrize("lo,hi", RANGES)
def test_gelu_of_fp32_outputs(ia, T, grouped, lo, hi):
    """v h or v - v h with h = erfc(|v| / sqrt 2) / 2 = E t P(t), E = 2^(-v^2 log2(e) / 2).  In units of 2^-24
    of h: 1 + c |v| rounds once (1) and its reciprocal is within a step (2), which t P(t) multiplies by
    at most 2.3, its slope against t at t = 1 (erfc(x) exp(x^2) falls by 1.13 x, and x is 2 (1 / t - 1)): 7; the
    fit 1, the eight steps of P 2, whose values are all below 1/2 of P's own: 10.  E: ex2 is within 2^-22
    (4), and its argument, of two roundings and a constant (2.5 units), is v^2 / 2 in natural logarithms
    (1.25 v^2).  The three products a rounding each (3).  For v > 0 that is h / (1 - h) < 1 times as much of
    v - v h.  In all 18 units, and below 0 also 1.25 v^2.  From |v| = 13 on E is subnormal, within 2 * 2^-149,
    times |v| <= 103: under 2^-141."""
    v = _arguments(lo, hi)
    d = v.to(F64)
    got, want = _through(ia, v, "gelu", T, grouped), 0.5 * d * torch.special.erfc(-d / 2 ** 0.5)
    units = torch.where(d > 0, torch.full_like(d, 18.0), 1.25 * d * d + 18)
    over = (got - want).abs() - (units * U * want.abs() + 2.0 ** -141)
    assert bool((over <= 0).all()), float(over.max())


@pytest.mark.parametrize("T,grouped", [(1, False), (300, False), (40, True)])
@pytest.mark.parametrize("lo,hi", RANGES)
def test_swiglu_of_fp32_outputs(ia, T, grouped, lo, hi):
    """As SILU, and one more rounding for the product with the up value."""
    v = _arguments(lo, hi)
    d = v.to(F64)
    got, want = _through(ia, v, "swiglu", T, grouped), _silu(d) * d.flip(0)
    over = (got - want).abs() - (12 * U * want.abs() + 2.0 ** -141 * (1 + d.flip(0).abs()))
    assert bool((over <= 0).all()), float((((got - want) / want).abs() / U).max())
