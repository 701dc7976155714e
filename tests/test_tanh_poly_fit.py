"""The FMA-pipe tanh of the capped scores (cap_pair in csrc/score.cuh) uses the float32 coefficients printed by
exact_tiled_attention_41_b200/fit_tanh_poly.py: re-run the fit, compare with the header, and check the accuracy of
the plain and of the folded evaluation in float32."""

import os
import re

import numpy as np
import pytest

from exact_tiled_attention_41_b200 import fit_tanh_poly as F
from tests.conftest import ROOT


def _header(degree):
    src = open(os.path.join(ROOT, "exact_tiled_attention_41_b200", "csrc", "score.cuh")).read()
    body = re.search(r"#define FA_TANH%d \{(.*)\}" % degree, src).group(1)
    return [np.float32(float(x.rstrip("f"))) for x in body.replace(" ", "").split(",")]


@pytest.mark.parametrize("limit,degree", F.RANGES)
def test_header_constants_are_the_fit(limit, degree):
    assert _header(degree) == F.coefficients_f32(limit, degree)
    assert _header(degree)[0] > 0        # a masked score, -inf, stays -inf


@pytest.mark.parametrize("limit,degree", F.RANGES)
def test_error_in_float32(limit, degree):
    # x is off by nothing, u = x^2 by one rounding, each Horner step and the last product by one more
    assert F.fp32_error(limit, degree) <= (5.1e-7 if degree == 2 else 2e-7)


@pytest.mark.parametrize("inv", [2.0 ** -13, 0.0011, 0.0044, 0.3, 2.0 ** 13])
@pytest.mark.parametrize("limit,degree", F.RANGES[:2])
def test_folded_coefficients_stay_normal_and_accurate(limit, degree, inv):
    # out tanh(inv s) = s (a_0 + a_1 w + ...), w = s^2, a_k = c_k out inv^(2k + 1) as the host folds them
    out = 43.28
    c = [float(x) for x in _header(degree)][::-1]
    a = [np.float32(ck * out * inv ** (2 * k + 1)) for k, ck in enumerate(c)]
    assert all(abs(x) >= np.finfo(np.float32).tiny for x in a)
    s = np.linspace(1e-3, 1.0, 200001).astype(np.float32) * np.float32(limit / inv)
    w = s * s
    p = np.full_like(w, a[-1])
    for x in a[-2::-1]:
        p = p * w + x
    want = out * np.tanh(inv * s.astype(np.float64))
    assert np.max(np.abs(s * p / want - 1.0)) <= (6e-7 if degree == 2 else 3e-7)
