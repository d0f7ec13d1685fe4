"""The polynomial 2^x of the windowed attention's kernels (ex2_poly): its error with the coefficients as
they stand in the source, exactly and in the kernel's own fp32 steps, without a GPU."""
import os
import re
from fractions import Fraction

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
F = np.float32


@pytest.fixture(scope="module")
def source():
    with open(os.path.join(ROOT, "sparse_dynamic_routing_b200", "csrc", "gm_common.cuh")) as f:
        return f.read()


@pytest.fixture(scope="module")
def coefficients(source):
    c = re.search(r"constexpr float C\[6\] = \{([^}]*)\}", source).group(1)
    return [F(x.strip().rstrip("f")) for x in c.split(",")]


def stated(source):
    """The two errors that the comment gives."""
    exact, fp32 = re.search(r"\((\S+) with these coefficients, (\S+) evaluated in fp32", source).groups()
    return float(exact), float(fp32)


def fma(a, b, c):
    """fp32 a * b + c with one rounding (the product is exact in 64 bits, the sum's second rounding is
    2^-29 of a step)."""
    return (a.astype(np.float64) * np.float64(b) + np.float64(c)).astype(F)


def test_exact_error(source, coefficients):
    f = np.linspace(-0.5, 0.5, 200001).astype(np.longdouble)
    p = np.zeros_like(f)
    for c in coefficients[::-1]:
        p = p * f + np.longdouble(float(c))
    worst = float(np.abs(p / np.exp2(f) - 1).max())
    assert worst <= stated(source)[0] <= 1.05 * worst, worst


def test_error_in_fp32(source, coefficients):
    rng = np.random.default_rng(1)
    x = np.concatenate([rng.uniform(-126, 127, 2_000_000), rng.uniform(-2, 2, 1_000_000), np.arange(-126, 128),
                        np.arange(-126, 127) + 0.5]).astype(F)
    rounding = F(12582912.0)
    t = (x + rounding).astype(F)
    n = (t - rounding).astype(F)
    assert (np.abs(x - n) <= 0.5).all()
    f = (x - n).astype(F)  # exact: both are multiples of x's last place
    p = np.full_like(f, coefficients[5])
    for c in coefficients[4::-1]:
        p = fma(p, f, c)
    bits = t.view(np.uint32).astype(np.uint64)
    scale = ((bits << 23) + 0x3F800000 & 0xFFFFFFFF).astype(np.uint32).view(F)
    assert np.array_equal(scale.astype(np.float64), np.exp2(n.astype(np.float64)))
    got = p.astype(np.longdouble) * scale  # a product with a power of two: exact down to 2^-126
    worst = float(np.abs(got / np.exp2(x.astype(np.longdouble)) - 1).max())
    assert worst <= stated(source)[1] <= 1.05 * worst, worst
    assert worst <= 2.0 ** -22
    assert Fraction(float(coefficients[0])) == 1 + Fraction(1, 2 ** 23)  # 2^x of an integer x is one step too large
