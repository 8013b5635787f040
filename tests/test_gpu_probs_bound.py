"""The error of inkattn_token_probs against what its arithmetic allows, in units of U = 2^-23 (a rounding is half
of one).  With D = (m - l) / t of an element and B the batches of 16 logits a thread takes one after the other:

  an exponential: 2 for the exponential unit; its argument (l - m) log2(e) / t is rounded in the constant
      (0.11), the quotient, the difference and the product (0.5 each): 1.61 D.  Factors between maxima (batch to
      thread, thread to CTA, CTA to row) are exponentials too, and their differences add up to D.
  a thread's sum: 2 additions in a group, at most 4 a batch: 2 B + 1; a factor (2) and its product (0.5) for every
      batch behind the first that raises the maximum: 2.5 (B - 1).
  the row's sum: a factor and its product from thread to CTA (2.5, rows read twice alone), 9 halvings (4.5), a
      factor and its product from CTA to row (2.5), 7 additions (3.5).
  all of an element's terms of the sum, 2 + 4.5 B - 1.5 + 13 = 4.5 B + 13.5, and 1.61 D weighted with the
      probabilities: the mean of D is the row's entropy less the log of its sum, at most ln V.
  a value: its exponential (2), the quotient by the sum and the product (0.5 each): 3; held rows have the factor
      of their CTA beside it (2), one batch of 32 and none to raise: less in the sum.

In all 4.5 B + 16.5 + 1.61 ln V + 1.61 D.  Rows of less than eight CTAs have B <= 4 and V <= 131072: 53.5 + 1.61 D;
of eight B <= V / 65536 + 1, so at most 64 + V 2^-14 + 2 D up to 2^20 logits, which the header states."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

U = 2.0 ** -23
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module")
def ia():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from relative_bias_hybrid_gb300 import build
    build.build()
    import relative_bias_hybrid_gb300.inkattn as ia
    return ia


def _run(ia, logits, temperature):
    probs = torch.full(logits.shape, float("nan"), device="cuda")
    ia.inkattn_token_probs(ia.token_probs_params(logits=logits, probs=probs, temperature=temperature))
    return probs


def _logits(T, V, dtype, order):
    g = torch.Generator(device="cuda").manual_seed(V + T)
    x = 3 * torch.randn((T, V), generator=g, device="cuda")
    if order == "rising":                       # every batch of a thread raises its maximum
        x = x.sort(1).values
    elif order == "even":                       # nearly equal: the largest entropy
        x = x * 0.01
    return x.to(dtype), 0.3 + torch.rand((T,), generator=g, device="cuda")


@pytest.mark.parametrize("order", ["any", "rising", "even"])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T, V", [(1, 3), (9, 50001), (1, 131072), (320, 8200), (310, 16411), (200, 50001), (40, 131072),
                                  (3, 524291), (2, 1 << 20)])
def test_values_are_within_the_stated_error(ia, T, V, dtype, order):
    l, t = _logits(T, V, dtype, order)
    got = _run(ia, l, t).double()
    d = (l.double().max(1, keepdim=True).values - l.double()) / t.double()[:, None]
    want = torch.exp(-d)
    want /= want.sum(1, keepdim=True)
    bar = want * (64 + V * 2.0 ** -14 + 2 * d) * U + 2.0 ** -125
    assert bool(((got - want).abs() <= bar).all()), float((((got - want).abs() - 2.0 ** -125) / want / U).max())


@pytest.mark.parametrize("order", ["any", "rising", "even"])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T, V", [(1, 3), (1, 1), (9, 50001), (1, 131072), (60, 16384), (100, 2049), (300, 4096)])
def test_held_rows_sum_to_one(ia, T, V, dtype, order):
    """Rows whose weights stay in registers: the values stored are those summed, so a row's sum is off by its
    roundings alone, whatever the exponentials are: a thread's additions (5), 9 halvings (4.5), the product with
    the CTA's factor (0.5), 7 additions (3.5), the quotient and the product (0.5 each).  2^-125 for each value
    that may have underflown."""
    l, t = _logits(T, V, dtype, order)
    total = _run(ia, l, t).double().sum(1)
    assert float((total - 1).abs().max()) <= 14.5 * U + V * 2.0 ** -125


@pytest.mark.parametrize("T, V", [(9, 1003), (320, 8200), (2, 262147)])
def test_the_smallest_and_largest_temperatures_of_the_stated_error(ia, T, V):
    """t = 2^-127, whose log2(e) / t is finite, with logits that far apart; and t = 2^126, with logits less than
    2^128 apart."""
    g = torch.Generator(device="cuda").manual_seed(V)
    z = (3 * torch.randn((T, V), generator=g, device="cuda").double()).clamp(-1.9, 1.9)
    for e in (-127, -126, -100, 100, 126):
        l = (z * 2.0 ** e).float()
        t = torch.full((T,), 2.0 ** e, dtype=torch.float64).float().cuda()
        got = _run(ia, l, t).double()
        d = (l.double().max(1, keepdim=True).values - l.double()) / t.double()[:, None]
        want = torch.exp(-d)
        want /= want.sum(1, keepdim=True)
        bar = want * (64 + V * 2.0 ** -14 + 2 * d) * U + 2.0 ** -125
        assert bool(((got - want).abs() <= bar).all()), (e, float(((got - want).abs() / want / U).max()))
        assert math.isfinite(float(got.sum()))
