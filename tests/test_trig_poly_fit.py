"""The rotary tables' sines and cosines (sin_cos_turn in csrc/rotary.cu) use the float32 coefficients printed by
exact_tiled_attention_41_b200/fit_trig_poly.py: re-run the fit, compare with the source, and check a float32 model of
the whole evaluation, quarter turns included."""

import os
import re

import numpy as np
import pytest

from exact_tiled_attention_41_b200 import fit_trig_poly as F
from tests.conftest import ROOT


def _source(var):
    src = open(os.path.join(ROOT, "exact_tiled_attention_41_b200", "csrc", "rotary.cu")).read()
    body = src[src.index("void sin_cos_turn("):]
    body = body[: body.index("\n}\n")]
    first = re.search(r"float %s = fmaf\((\S+)f, u, (\S+)f\);" % var, body)
    rest = re.findall(r"^    %s = fmaf\(%s, u, (\S+)f\)" % (var, var), body, flags=re.M)
    return [np.float32(float(x)) for x in list(first.groups()) + rest]


@pytest.mark.parametrize("name,var", [("sin", "s"), ("cos", "c")])
def test_source_constants_are_the_fit(name, var):
    assert _source(var) == F.coefficients_f32(name)


@pytest.mark.parametrize("name", ["sin", "cos"])
def test_error_in_float32(name):
    assert F.fp32_error(name) <= 1.2e-7        # values up to 1: two half steps of fp32


def test_model_over_the_whole_turn():
    frac = np.random.RandomState(0).randint(0, 1 << 32, 500000, dtype=np.uint64).astype(np.uint32)
    frac[:9] = [0, 1, 0x1FFFFFFF, 0x20000000, 0x40000000, 0x80000000, 0xC0000000, 0xE0000000, 0xFFFFFFFF]
    quarter = (frac + np.uint32(0x20000000)) >> np.uint32(30)
    left = (frac - (quarter << np.uint32(30))).astype(np.int32)
    y = left.astype(np.float32) * np.float32(1.4629180792671596e-9)
    u = y * y
    out = {}
    for name, var in (("sin", "s"), ("cos", "c")):
        c = _source(var)
        p = np.full_like(u, c[0])
        for a in c[1:]:
            p = p * u + a
        out[name] = p * y if name == "sin" else p
    odd = (quarter & 1).astype(bool)
    sn = np.where(odd, out["cos"], out["sin"]) * np.where(quarter & 2, -1, 1)
    cs = np.where(odd, out["sin"], out["cos"]) * np.where((quarter + 1) & 2, -1, 1)
    a = frac.astype(np.float64) * (2 * np.pi / 2 ** 32)
    assert np.abs(sn - np.sin(a)).max() <= 2e-7 and np.abs(cs - np.cos(a)).max() <= 2e-7
