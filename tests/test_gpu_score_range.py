"""Capped scores over the whole accepted range of caps and scores, on the GPU against the fp64 oracle."""

import pytest

from exact_tiled_attention_41_b200 import workloads as W
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
