"""Calls of the rotary entry points that must not pass silently."""

import pytest
import torch

from exact_tiled_attention_41_b200 import attention as A
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
