"""The oracle of the cache in 8 bits against exact fractions and the numbers of e4m3."""
from fractions import Fraction

import numpy as np
import pytest
import torch

import oracle
from oracle import codes as C


def test_e4m3_numbers_are_those_of_the_type():
    b = torch.arange(256, dtype=torch.int32).to(torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    v = C.e4m3_numbers()
    assert np.array_equal(np.isnan(b), np.isnan(v)) and np.array_equal(b[~np.isnan(b)], v[~np.isnan(v)])
    assert np.nanmax(v) == 448 and np.sum(~np.isnan(v)) == 254 and len(set(v[~np.isnan(v)])) == 253


def bf16(x):
    return torch.from_numpy(np.asarray(x, np.float32)).bfloat16().double().numpy()


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_codes_are_the_nearest(fmt):
    rng = np.random.default_rng(3)
    x = bf16(rng.standard_normal((40, 16)) * np.exp(3 * rng.standard_normal((40, 1))))
    x[0] = 0
    x[1, :4] = bf16([127.0, 0.5, 1.5, -2.5])            # int8: halfway values, which go to the even code
    x[1, 4:] = 0
    x[2, :4] = bf16([448.0, 17.0, 19.0, 2.0 ** -10])    # e4m3: between 16 and 18, 18 and 20, 0 and 2^-9
    x[2, 4:] = 0
    codes, scales = oracle.oracle_encode(x, fmt)
    num = [Fraction(float(v)) for v in C.values(np.arange(256).astype(np.uint8).view(np.int8), fmt) if np.isfinite(v)]
    for r in range(len(x)):
        a = max(abs(Fraction(float(v))) for v in x[r])
        assert scales[r] == np.float32(float(a)) / np.float32(C.M[fmt])
        for v, c in zip(x[r], C.values(codes[r], fmt)):
            t = Fraction(float(v)) * Fraction(C.M[fmt]) / a if a else Fraction(0)
            gap = min(abs(t - y) for y in num)
            assert abs(t - Fraction(float(c))) == gap
    if fmt == "int8":
        assert codes[1, :4].tolist() == [127, 0, 2, -2]
    else:
        assert C.values(codes[2], fmt)[:4].tolist() == [448.0, 16.0, 20.0, 0.0]


def test_rows_that_are_not_finite():
    x = np.ones((3, 16))
    x[0, 3], x[1, 0], x[2, 5] = np.nan, np.inf, -np.inf
    for fmt in C.M:
        codes, scales = oracle.oracle_encode(x, fmt)
        assert not codes.any() and np.isnan(scales).all()
