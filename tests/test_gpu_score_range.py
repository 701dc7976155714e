"""Capped scores over the whole accepted range of caps and scores, on the GPU against the fp64 oracle."""

import math

import numpy as np
import pytest
import torch

import oracle.modifiers as M
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


# ------------------------------------------------------------------------------------------- Delta
def gradients(lens, Hq, Hkv, D, softcap, slopes, seed, det=True, only=None):
    """Gradients (and the oracle's) of sequence `only` of a packed causal batch."""
    w = W.varlen(lens, lens, Hq, Hkv, D, True, seed=seed)
    w.tensors["q"].mul_(2)
    t = {n: x.cuda() for n, x in w.tensors.items()}
    sl = None if slopes is None else slopes.cuda()
    where = (t["cu_q"], t["cu_k"], max(lens), max(lens))
    out, lse = A.flash_attn_varlen_func(t["q"], t["k"], t["v"], *where, w.scale, True, NONE, softcap, sl)
    g = A.flash_attn_varlen_backward(t["do"], t["q"], t["k"], t["v"], out, lse, *where, w.scale, True, NONE, det, softcap, sl)
    cu = w.tensors["cu_q"].tolist()
    a, b = cu[only], cu[only + 1]
    cut = {n: w.tensors[n][a:b] for n in ("q", "k", "v", "do")}
    ref = M.attention(*([f64(cut[n])] for n in ("q", "k", "v")), w.scale, True, NONE, softcap,
                      None if slopes is None else slopes.numpy(), [f64(cut["do"])])[0]
    return [x[a:b] for x in g], ref, cut


def check_norms(g, ref):
    # three roundings to bf16 at most, 1.6e-3 of the norm each on average (see test_gradients_of_rows_with_few_keys)
    for name, x in zip(("dq", "dk", "dv"), g):
        assert np.linalg.norm(f64(x) - ref[name]) <= 4e-3 * np.linalg.norm(ref[name]), name


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("kind", [None, "falling"])
@pytest.mark.parametrize("det", [False, True])
def test_gradients_of_a_short_document_packed_beside_a_long_one(D, kind, det):
    slopes = None if kind is None else slopes_of(4, kind=kind)
    g, ref, _ = gradients([3000, 3, 2100], 4, 2, D, 20.0, slopes, D, det, 1)
    check_norms(g, ref)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("softcap", [0.0, 20.0])
@pytest.mark.parametrize("steep", [4.0, 1.0, -2.0])
def test_gradients_under_steep_slopes_in_a_long_sequence(D, softcap, steep):
    # each row puts its weight on a few keys: the nearest, or the farthest
    g, ref, _ = gradients([100, 1800, 2200], 4, 2, D, softcap, torch.tensor([steep] * 4), D + 1, True, 1)
    check_norms(g, ref)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_gradients_of_a_sequence_do_not_depend_on_the_batch_around_it(D):
    slopes = slopes_of(4, kind="mixed")
    for n in (5, 60, 130):
        long, _, cut = gradients([n, 2500, 2500], 4, 2, D, 8.0, slopes, n, True, 0)
        t = {k: x.cuda()[None].contiguous() for k, x in cut.items()}
        scale = 1.0 / math.sqrt(D)
        out, lse = A.flash_attn_func(t["q"], t["k"], t["v"], scale, True, NONE, 8.0, slopes.cuda())
        alone = A.flash_attn_backward(t["do"], t["q"], t["k"], t["v"], out, lse, scale, True, NONE, True, 8.0, slopes.cuda())
        for x, y in zip(long, alone):
            assert torch.equal(x, y[0])
