"""Calls of the rotary entry points that must not pass silently, and the relative accuracy of small sines."""

import numpy as np
import pytest
import torch

import oracle.modifiers as M
from exact_tiled_attention_41_b200 import abi, attention as A
from tests.gpu_helpers import f64
from tests.test_gpu_rotary import normal, tables

pytestmark = pytest.mark.gpu


def test_in_place_rotation_is_refused_where_autograd_would_miss_it():
    cos, sin, _, _ = tables(16, 32)
    cos, sin = cos.cuda(), sin.cuda()
    x = normal(1, 2, 9, 3, 64).cuda().requires_grad_()
    h = x * 2                                            # not a leaf
    for t in (x, h):
        before = t.detach().clone()
        with pytest.raises(ValueError, match="grad"):
            A.apply_rotary(t, cos, sin, out=t)
        with pytest.raises(ValueError, match="grad"):
            A.apply_rotary(t, cos, sin, out=torch.empty_like(t))
        with pytest.raises(ValueError, match="grad"):
            A.apply_rotary(t.detach(), cos, sin, out=t)
        assert torch.equal(t, before)
    with torch.no_grad():
        want = A.apply_rotary(h, cos, sin)
        assert A.apply_rotary(h, cos, sin, out=h) is h
    assert torch.equal(h, want)


def test_a_tensor_that_autograd_saved_may_not_change_under_it():
    cos, sin, _, _ = tables(16, 32)
    x = normal(2, 2, 9, 3, 64).cuda()
    scale = torch.ones(64, device="cuda", dtype=torch.bfloat16, requires_grad=True)
    y = (x * scale).sum()                                # saves x
    A.apply_rotary(x, cos.cuda(), sin.cuda(), out=x)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()
    with torch.inference_mode():                         # tensors without a version counter
        z = normal(2, 2, 9, 3, 64).cuda()
        A.apply_rotary(z, cos.cuda(), sin.cuda(), out=z)
    assert torch.equal(z, x)


def test_positions_that_the_host_knows_to_be_past_the_tables_are_refused():
    x = normal(3, 2, 6, 2, 64).cuda()
    cos, sin, _, _ = tables(10, 32)
    cos, sin = cos.cuda(), sin.cuda()
    A.apply_rotary(x, cos, sin, 4)
    for offset in (5, 10, 1 << 20, 1 << 31, 1 << 32, (1 << 32) + 1):
        with pytest.raises(ValueError, match="position"):
            A.apply_rotary(x, cos, sin, offset)
        with pytest.raises(ValueError, match="position"):
            A.RotaryFunction.apply(x, cos, sin, offset)
    cu = torch.tensor([0, 3, 6], dtype=torch.int32).cuda()
    for offset in (1 << 31, 1 << 32):
        with pytest.raises(ValueError, match="position"):
            A.apply_rotary(x[0], cos, sin, offset, cu_seqlens=cu)
    q, kc = normal(4, 2, 2, 2, 64).cuda(), normal(5, 2, 64, 2, 64).cuda()
    before = kc.clone()
    call = lambda n, **kw: A.flash_attn_with_kvcache(q, kc, kc.clone(), n, k=q, v=q, rotary_cos=cos, rotary_sin=sin, **kw)  # noqa: E731
    for n in (9, 10, 63):
        for kw in (dict(causal=True), dict()):
            with pytest.raises(ValueError, match="position"):
                call(n, **kw)
    assert torch.equal(kc, before)
    call(8)
    call(8, causal=True)
    assert abi.fa_get_device_status() == 0


def test_a_full_cache_asks_for_no_position_of_keys_that_it_does_not_take():
    # 64 rows, all in use: nothing is appended, and the query stands at position 64, the tables' last
    cos, sin, _, _ = tables(65, 32)
    q, kc = normal(6, 1, 1, 2, 64).cuda(), normal(7, 1, 64, 2, 64).cuda()
    k = normal(8, 1, 3, 2, 64).cuda()
    before = kc.clone()
    A.flash_attn_with_kvcache(q, kc, kc.clone(), 64, k=k, v=k, rotary_cos=cos.cuda(), rotary_sin=sin.cuda())
    assert torch.equal(kc, before) and abi.fa_get_device_status() == 0


@pytest.mark.parametrize("scaling,factor", [("none", 1.0), ("linear", 32.0), ("base", 16.0), ("by_parts", 32.0)])
def test_small_sines_are_as_accurate_as_large_ones(scaling, factor):
    rows, rd, base = 300, 128, 1e6
    cos, sin = A.rotary_tables(rows, rd, base, scaling, factor, original_seqlen=4096)
    c, s = M.rotary_tables(rows, rd, base, scaling, factor, original=4096)
    # The turn of a position is kept to 2^-63 (and 2^-53 of itself): an angle off by pos 2 pi 2^-63.  Then float32: the
    # angle's conversion and product, its square, and the polynomial with its last product, 4 half steps relative; a
    # quarter turn on, the cosine's polynomial, 2 half steps of 1.  Where the angle comes back near a multiple of a quarter
    # turn, the bound on the angle in turns counts, not its relative size.
    pos = np.arange(rows)[:, None]
    angle = pos * (2 * np.pi * 2.0 ** -63) + 2.0 ** -50 * pos
    for got, want in ((cos, c), (sin, s)):
        err = np.abs(f64(got) - want)
        assert (err <= 5 * 2.0 ** -24 * np.abs(want) + angle).all()
