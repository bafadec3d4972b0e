"""The two polynomials of the gates (csrc/glr_gate.cuh), with the coefficients that stand
there, against 64 bits over their whole ranges, in exact and in fp32 arithmetic."""
import os
import re

import numpy as np
import pytest

from gated_delta_rule_52_gb300 import build

N = 1 << 20


def _horner(name):
    """Leading coefficient and the others, as the function of this name applies them."""
    src = open(os.path.join(build.CSRC, "glr_gate.cuh")).read()
    body = src[src.index(f"void {name}("):]
    rest = re.search(r"constexpr float c\[\d\] = \{([^}]*)\};", body).group(1).split(",")
    lead = re.search(r"fma_n<n>\(q, \w, ([\d.]+)f, c\[0\]\);", body).group(1)
    return [np.float32(t.strip().rstrip("f")) for t in (lead, *rest)]


def _errors(coefficients, x, want):
    exact, single = np.full_like(x, coefficients[0]), np.full(x.shape, coefficients[0], np.float32)
    for c in coefficients[1:]:
        exact = exact * x + float(c)
        single = (single.astype(np.float64) * x + float(c)).astype(np.float32)   # one rounding, as an fma's
    return np.abs(exact / want - 1).max(), np.abs(single / want - 1).max()


@pytest.mark.parametrize("name,exact,single", [("atanh_poly_n", 2.2e-8, 6.4e-8), ("exp2_decay_n", 1.1e-8, 7.6e-8)])
def test_polynomials(name, exact, single):
    if name == "atanh_poly_n":
        s = np.sqrt(np.linspace(1 / N, 1 / 9, N).astype(np.float32).astype(np.float64))
        x, want = s * s, 2 * np.arctanh(s) / s / np.log(2)
        x = x.astype(np.float32).astype(np.float64)
    else:
        x = np.linspace(-0.5, 0, N).astype(np.float32).astype(np.float64)
        want = 2.0 ** x
    got = _errors(_horner(name), x, want)
    assert got[0] <= exact and got[1] <= single, got
