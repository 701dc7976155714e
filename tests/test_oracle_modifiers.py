"""Pins of oracle/modifiers.py: closed forms, reductions to the plain oracle, central differences, torch autograd."""

import numpy as np
import pytest
import torch

import oracle
from oracle import modifiers as M


def _rand(seed, *shapes):
    r = np.random.RandomState(seed)
    return [r.randn(*s) for s in shapes]


def test_without_modifiers_it_is_the_plain_oracle():
    q, k, v, do = _rand(0, (2, 5, 4, 8), (2, 7, 2, 8), (2, 7, 2, 8), (2, 5, 4, 8))
    o, lse = oracle.mha_forward(q, k, v, 0.3, True, (3, -1))
    dq, dk, dv = oracle.mha_backward(q, k, v, do, 0.3, True, (3, -1))
    for b, r in enumerate(M.attention(q, k, v, 0.3, True, (3, -1), do=do)):
        for n, want in (("o", o), ("lse", lse), ("dq", dq), ("dk", dk), ("dv", dv)):
            np.testing.assert_allclose(r[n], want[b], rtol=1e-12, atol=1e-13)


def test_a_wide_cap_changes_nothing_and_a_narrow_one_bounds_the_scores():
    q, k = _rand(1, (6, 8), (9, 8))
    x, _ = M.scores(q, k, 0.5)
    np.testing.assert_allclose(M.scores(q, k, 0.5, softcap=1e6)[0], x, rtol=1e-9)
    assert np.abs(M.scores(q, k, 50.0, softcap=2.0)[0]).max() <= 2.0


def test_bias_is_the_distance_from_the_bottom_right_diagonal():
    q, k = np.zeros((2, 4)), np.zeros((5, 4))
    x, _ = M.scores(q, k, 1.0, slope=0.5)
    np.testing.assert_array_equal(x, -0.5 * np.array([[3, 2, 1, 0, 1], [4, 3, 2, 1, 0]]))


def test_equal_keys_leave_the_bias_alone():
    # with identical keys the scores differ by the bias only: weights exp(-slope d) / sum
    q, v = _rand(2, (1, 4), (6, 4))
    k = np.ones((6, 4))
    r = M.head(q, k, v, 0.7, np.ones((1, 6), bool), softcap=3.0, slope=0.25)
    w = np.exp(-0.25 * np.arange(5, -1, -1.0))
    np.testing.assert_allclose(r["o"][0], (w / w.sum()) @ v, rtol=1e-12)


@pytest.mark.parametrize("softcap,slope", [(1.5, None), (0.0, 0.3), (2.0, -0.2), (0.7, 0.4)])
@pytest.mark.parametrize("causal,Lq,Lk", [(False, 3, 5), (True, 5, 3), (True, 4, 4)])
def test_gradients_are_differences(softcap, slope, causal, Lq, Lk):
    q, k, v, do = _rand(3, (Lq, 4), (Lk, 4), (Lk, 4), (Lq, 4))
    mask = oracle.allowed_mask(Lq, Lk, causal)
    r = M.head(q, k, v, 0.6, mask, softcap, slope, do)
    h = 1e-6
    for name, a in (("dq", q), ("dk", k), ("dv", v)):
        num = np.zeros_like(a)
        for idx in np.ndindex(a.shape):
            keep = a[idx]
            f = []
            for d in (h, -h):
                a[idx] = keep + d
                f.append((M.head(q, k, v, 0.6, mask, softcap, slope)["o"] * do).sum())
            a[idx] = keep
            num[idx] = (f[0] - f[1]) / (2 * h)
        np.testing.assert_allclose(r[name], num, atol=2e-8 * max(1.0, np.abs(num).max()))


def test_gradients_are_autograds_and_shared_heads_are_summed():
    q, k, v, do = _rand(4, (2, 5, 4, 8), (2, 6, 2, 8), (2, 6, 2, 8), (2, 5, 4, 8))
    slopes = np.random.RandomState(5).rand(2, 4)
    res = M.attention(q, k, v, 0.4, False, softcap=1.2, slopes=slopes, do=do)
    tq, tk, tv = (torch.tensor(a, requires_grad=True) for a in (q, k, v))
    kk, vv = tk.repeat_interleave(2, 2), tv.repeat_interleave(2, 2)
    x = 1.2 * torch.tanh(torch.einsum("bihd,bjhd->bhij", tq, kk) * 0.4 / 1.2)
    i, j = torch.arange(5)[:, None], torch.arange(6)[None, :]
    x = x - torch.tensor(slopes)[:, :, None, None] * (i + 1 - j).abs()
    o = torch.einsum("bhij,bjhd->bihd", torch.softmax(x, -1), vv)
    grads = torch.autograd.grad(o, (tq, tk, tv), torch.tensor(do))
    for b in range(2):
        for n, g in zip(("dq", "dk", "dv"), grads):
            np.testing.assert_allclose(res[b][n], g[b].numpy(), rtol=1e-9, atol=1e-12)


def test_rows_without_keys():
    q, k, v, do = _rand(6, (4, 8), (2, 8), (2, 8), (4, 8))
    r = M.head(q, k, v, 0.5, oracle.allowed_mask(4, 2, True), 1.0, 0.1, do)
    assert (r["o"][:2] == 0).all() and np.isneginf(r["lse"][:2]).all() and (r["dq"][:2] == 0).all()
    assert np.isfinite(r["dk"]).all() and np.isfinite(r["dv"]).all()


@pytest.mark.parametrize("interleaved", [True, False])
def test_rotation_keeps_lengths_and_depends_on_differences_only(interleaved):
    x, y = _rand(7, (1, 2, 32), (1, 2, 32))
    cos, sin = M.rotary_tables(50, 16)
    a = M.rotate(x, cos, sin, np.array([11]), interleaved)
    np.testing.assert_allclose(np.linalg.norm(a, axis=-1), np.linalg.norm(x, axis=-1))
    np.testing.assert_array_equal(a[..., 16:], x[..., 16:])
    dots = [(M.rotate(x, cos, sin, np.array([p + 7]), interleaved) * M.rotate(y, cos, sin, np.array([p]), interleaved)).sum()
            for p in (0, 5, 42)]
    np.testing.assert_allclose(dots, dots[0], rtol=1e-12)
    back = M.rotate(a, cos, sin, np.array([11]), interleaved, inverse=True)
    np.testing.assert_allclose(back, x, atol=1e-14)


def test_rotation_by_hand():
    # position 1, rotary_dim 4: angles 1 and 0.01
    cos, sin = M.rotary_tables(2, 4)
    np.testing.assert_allclose(cos[1], np.cos([1.0, 0.01]))
    x = np.array([[[1.0, 2.0, 3.0, 4.0]]])
    c, s = cos[1], sin[1]
    np.testing.assert_allclose(M.rotate(x, cos, sin, np.array([1]), True)[0, 0],
                               [c[0] - 2 * s[0], 2 * c[0] + s[0], 3 * c[1] - 4 * s[1], 4 * c[1] + 3 * s[1]])
    np.testing.assert_allclose(M.rotate(x, cos, sin, np.array([1]), False)[0, 0],
                               [c[0] - 3 * s[0], 2 * c[1] - 4 * s[1], 3 * c[0] + s[0], 4 * c[1] + 2 * s[1]])


def test_scaled_tables():
    plain = M.rotary_tables(64, 32)
    lin = M.rotary_tables(256, 32, scaling="linear", factor=4.0)
    np.testing.assert_allclose(lin[0][::4], plain[0], atol=1e-12)
    # base change: the fastest pair keeps its speed, the slowest is slowed by the factor
    chg = M.rotary_tables(2, 32, scaling="base", factor=8.0)
    fast, slow = np.arctan2(chg[1][1], chg[0][1])[[0, -1]]
    np.testing.assert_allclose(fast, 1.0)
    np.testing.assert_allclose(slow, 10000.0 ** (-30 / 32) / 8, rtol=1e-9)
    # by parts: pairs with many turns in the original context stay, those with few are slowed
    part = M.rotary_tables(2, 64, scaling="by_parts", factor=8.0, original=4096)
    ang = np.arctan2(part[1][1], part[0][1])
    want = 10000.0 ** (-np.arange(32) / 32)
    turns = 4096 * want / (2 * np.pi)
    np.testing.assert_allclose(ang[turns > 32], want[turns > 32], rtol=1e-9)
    np.testing.assert_allclose(ang[turns < 1], want[turns < 1] / 8, rtol=1e-9)
    mid = (turns > 1) & (turns < 32)
    assert mid.any() and (ang[mid] < want[mid]).all() and (ang[mid] > want[mid] / 8).all()
