"""The oracle's 4-bit cache rows, pinned by hand: the scale chosen, ties, saturation, the codes' places,
and the layout that the header states."""
import os
import re

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _row(values):
    from helpers import to_bits
    x = np.zeros(128)
    x[:len(values)] = values
    return to_bits(x)[None]


def test_scales_are_the_upper_bytes_of_fp16(oracle_mod):
    want = (np.arange(0xC7).astype(np.uint16) << 7).view(np.float16).astype(np.float64)
    assert np.array_equal(oracle_mod.i4_scales(), want)
    assert want[0xC6] == 896 and 72 * 896 < 65504


@pytest.mark.parametrize("top, scale", [
    (7.0, 1.0),                       # 7 * 1 holds it exactly
    (7.03125, 1.125),                 # the next bf16 does not fit: the next scale
    (1.0, 0.15625),                   # 1/7 = 0.1428..: 0.140625 < 1/7 <= 0.15625
    (2.0 ** -17 * 7, 2.0 ** -17),     # the smallest scale
    (2.0 ** -30, 2.0 ** -17),         # below it: still that scale
    (0.0, 0.0),
    (6272.0, 896.0),                  # the largest value that fits
    (1e30, 896.0),                    # beyond: saturates
])
def test_scale_of_a_group(oracle_mod, top, scale):
    codes, b = oracle_mod.quantize_rows_i4(_row([0.0] * 32 + [-top]))
    assert oracle_mod.i4_scales()[b[0, 1]] == scale
    assert b[0, 0] == b[0, 2] == b[0, 3] == 0


def test_rounding_ties_to_even_and_saturation(oracle_mod):
    x = [7.0, 0.5, 1.5, 2.5, -0.5, -1.5, -2.5, 3.49, -6.53125, 6.5, 0.49]
    codes, b = oracle_mod.quantize_rows_i4(_row(x))
    got = oracle_mod.dequantize_i4(codes, b)[0]
    assert got[:11].tolist() == [7, 0, 2, 2, 0, -2, -2, 3, -7, 6, 0]
    codes, b = oracle_mod.quantize_rows_i4(_row([1e30, -1e30, 1.0, float("nan")]))
    assert oracle_mod.dequantize_i4(codes, b)[0, :4].tolist() == [6272.0, -6272.0, 0.0, 0.0]


def test_places_of_the_codes(oracle_mod):
    x = np.zeros(128)
    x[:8] = [-7, -5, -3, -1, 1, 3, 5, 7]
    codes, b = oracle_mod.quantize_rows_i4(_row(x))
    u = [1, 3, 5, 7, 9, 11, 13, 15]
    word = sum(u[2 * i] << (4 * i) | u[2 * i + 1] << (16 + 4 * i) for i in range(4))
    assert codes[0, :4].tolist() == [(word >> (8 * i)) & 255 for i in range(4)]
    assert (codes[0, 4:] == 0x88).all()               # n = 0 is u = 8


def test_values_are_exact_in_bf16_and_fp16(oracle_mod):
    s = oracle_mod.i4_scales()
    v = np.outer(np.arange(-7, 8), s).ravel()
    assert np.array_equal(v.astype(np.float16).astype(np.float64), v)
    assert np.array_equal(oracle_mod.bf16_bits_to_f64(oracle_mod.round_bf16(v)), v)


def test_fused_expansion_is_exact():
    """(64 + u) s - 72 s as the kernels take it: 72 s is an fp16 (so the multiply-add rounds n s once, and n s
    is an fp16)."""
    s = (np.arange(0xC7).astype(np.uint16) << 7).view(np.float16)
    off = s.astype(np.float64) * 72
    assert np.array_equal(off.astype(np.float16).astype(np.float64), off)


def test_header_states_the_type():
    text = open(os.path.join(ROOT, "include", "inkattn.h")).read()
    assert re.search(r"#define INKATTN_KV_I4 4\b", text)
