"""Capped scores over the whole accepted range of caps and scores, on the GPU against the fp64 oracle."""

import numpy as np
import pytest
import torch

from exact_tiled_attention_41_b200 import abi, attention as A, workloads as W
from tests.gpu_helpers import f64
from tests.test_gpu_score_mod import NONE, check_cache, check_dense, slopes_of

pytestmark = pytest.mark.gpu

CAPS = [1e2, 1e4, 1e6, 1e8, 1e18]


@pytest.mark.parametrize("softcap", CAPS)
@pytest.mark.parametrize("D,kind", [(64, None), (128, "mixed"), (256, None)])
def test_cache_call_under_large_caps(D, kind, softcap):
    lens = [1, 63, 256, 700]
    w = W.kvcache_update(len(lens), 3, 8, 2, D, 1024, lens, seqlen_new=3, seed=D)
    w.tensors["q"].mul_(2)
    check_cache(w, True, NONE, softcap, None if kind is None else slopes_of(8, kind=kind))


@pytest.mark.parametrize("softcap", CAPS)
@pytest.mark.parametrize("D,kind,window", [(64, None, (3, 2)), (128, "mixed", NONE), (256, None, (1, 0))])
def test_gradients_under_large_caps(D, kind, window, softcap):
    # few keys a row: Delta is formed from the probabilities there
    w = W.dense(2, 60, 60, 4, 2, D, False, seed=D)
    w.tensors["q"].mul_(2)
    for det in (False, True):
        check_dense(w, window, softcap, None if kind is None else slopes_of(4, kind=kind), det, causal=kind is not None)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("softcap", [100.0, 1e5, 1e7])
def test_rows_at_the_cap_beside_rows_far_below_it(D, softcap):
    # every fifth query reaches the cap; the others in the same warp score a few units and must not feel it
    w = W.dense(2, 150, 150, 2, 2, D, True, seed=D + 1)
    w.tensors["q"][:, ::5] *= softcap
    for det in (False, True):
        check_dense(w, NONE, softcap, None, det)
    c = W.kvcache_update(3, 4, 4, 2, D, 512, [5, 200, 508], seqlen_new=4, seed=D)
    c.tensors["q"][:, ::2] *= softcap
    check_cache(c, True, NONE, softcap, None)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("softcap,slope", [(1.0, None), (1.0, 0.01), (60.0, None)])
def test_raw_scores_beyond_float32(D, softcap, slope):
    """q.k overflows to +-inf in float32: the tanh is +-1 there, in every path, and its derivative 0."""
    S = 150
    w = W.dense(1, S, S, 1, 1, D, True, seed=D)
    t = w.tensors
    sign = torch.ones(S)
    sign[1::3] = -1
    t["k"][0, :, 0] = 2e20 * sign[:, None].to(torch.bfloat16)
    t["q"][0, :, 0] = 2e20 * ((-1.0) ** torch.arange(S))[:, None].to(torch.bfloat16)
    slopes = None if slope is None else torch.tensor([slope])
    sl = None if slope is None else slopes.cuda()
    d = {n: x.cuda() for n, x in t.items()}
    x = softcap * np.outer((-1.0) ** np.arange(S), sign.numpy())
    if slope is not None:
        x = x - slope * np.abs(np.arange(S)[:, None] - np.arange(S)[None, :])
    x = np.where(np.tril(np.ones((S, S), bool)), x, -np.inf)
    m = x.max(1, keepdims=True)
    p = np.exp(x - m)
    lse = m[:, 0] + np.log(p.sum(1))
    p /= p.sum(1, keepdims=True)
    o, v, do = p @ f64(t["v"])[0, :, 0], f64(t["v"])[0, :, 0], f64(t["do"])[0, :, 0]
    # P rounded to bf16, the result rounded once more; the exponents are exact but for float32 roundings of the score
    o_tol = 2.0 ** -7 * (p @ np.abs(v)) + 1e-6
    lse_tol = 2.0 ** -20 * (1 + np.abs(lse))
    out, l = A.flash_attn_func(d["q"], d["k"], d["v"], w.scale, True, NONE, softcap, sl)
    assert (np.abs(f64(out)[0, :, 0] - o) <= o_tol).all() and (np.abs(f64(l)[0, 0] - lse) <= lse_tol).all()
    for det in (False, True):
        dq, dk, dv = A.flash_attn_backward(d["do"], d["q"], d["k"], d["v"], out, l, w.scale, True, NONE, det, softcap, sl)
        assert (dq == 0).all() and (dk == 0).all()
        assert (np.abs(f64(dv)[0, :, 0] - p.T @ do) <= 2.0 ** -7 * (p.T @ np.abs(do)) + 1e-6).all()
    n = torch.tensor([S], dtype=torch.int32, device="cuda")
    out, l = A.flash_attn_with_kvcache(d["q"], d["k"], d["v"], n, w.scale, True, softcap=softcap, alibi_slopes=sl)
    assert (np.abs(f64(out)[0, :, 0] - o) <= o_tol).all() and (np.abs(f64(l)[0, 0] - lse) <= lse_tol).all()
    assert abi.fa_get_device_status() == 0


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("softcap,scale", [(1e-18, 1e-21), (1e-12, 2e-16), (1e-19, 1e-20)])
@pytest.mark.parametrize("grow", [1, 4, 8, 13, 20, 60])
def test_tiny_caps_and_scales_under_a_mask(D, softcap, scale, grow):
    # the scores are nothing beside 1, whatever their ratio to the cap, so every allowed key weighs the same
    w = W.dense(1, 200, 200, 2, 1, D, True, seed=grow)
    w.scale = scale
    w.tensors["q"].mul_(grow)
    check_dense(w, (90, -1), softcap, None)
