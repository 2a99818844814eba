"""int8 codes of values at half and at other odd multiples of a 254th of their row's largest, where the code
hangs on the factor's one rounding: exact rational arithmetic against the device, for every bf16
mantissa of the largest value."""
from fractions import Fraction

import numpy as np
import pytest

import sort_ref as ref
from test_gpu_sort import Rows, sync

pytestmark = pytest.mark.gpu


def to_fp32(q):
    """The fp32 value next to a positive rational in the normal range, ties to even."""
    e = 0
    while q >= 2 ** 24:
        q, e = q / 2, e + 1
    while q < 2 ** 23:
        q, e = q * 2, e - 1
    n = q.numerator // q.denominator
    rest = q - n
    if rest > Fraction(1, 2) or (rest == Fraction(1, 2) and n % 2):
        n += 1
    return Fraction(n) * Fraction(2) ** e


def nearest(q):
    """The integer next to a rational, ties to even."""
    n = q.numerator // q.denominator
    rest = q - n
    return n + (rest > Fraction(1, 2) or (rest == Fraction(1, 2) and n % 2 == 1))


def rows_of(exponent):
    """bf16 rows, one for each mantissa of the largest value a: a, its halves, and the bf16 values next to
    (2 n + 1) a / 254, of both signs."""
    rows = []
    for mantissa in range(128, 256):
        a = float(mantissa) * 2.0 ** exponent
        border = ref.bf16_round((np.arange(1, 254, 2) * (a / 254)).astype(np.float32))
        rows.append(np.concatenate([[a, a / 2, -a / 2], border, -border]))
    return np.array(rows, np.float32)


def definition(x):
    codes, scales = [], []
    for row in x:
        a = max(abs(Fraction(float(v))) for v in row)
        r = to_fp32(Fraction(127) / a)
        codes.append([nearest(Fraction(float(v)) * r) for v in row])
        scales.append(float(to_fp32(a / 127)))
    return np.array(codes), np.array(scales, np.float32)


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("exponent", [-12, 3])
def test_halves_of_every_largest_value(c3gpu, exponent, dtype):
    import torch

    x = rows_of(exponent)
    rows, cols = x.shape
    X = Rows(rows, cols, dtype, values=x)
    assert (X.numpy() == x).all()
    codes = torch.zeros(rows, ref.padded(cols), dtype=torch.int8, device="cuda:0")
    scales = torch.zeros(rows, device="cuda:0")
    c3gpu.c3_i8_quantize(X.ptr(), dtype, rows, cols, cols, codes, scales)
    sync()
    want = definition(x)
    assert {int(c) for c in want[0][:, 1]} == {63, 64}  # the half falls on either side, by the factor's rounding
    np.testing.assert_array_equal(codes.cpu().numpy()[:, :cols], want[0])
    np.testing.assert_array_equal(scales.cpu().numpy(), want[1])
