"""Capped and biased attention on the GPU against the fp64 oracle, element by element within the bounds that
oracle/modifiers.py derives from the roundings: dense, packed and cached, forward and both backwards."""

import math

import numpy as np
import pytest
import torch

import oracle.modifiers as M
from exact_tiled_attention_41_b200 import abi, attention as A, workloads as W
from tests.gpu_helpers import f64

pytestmark = pytest.mark.gpu

NONE = (-1, -1)


def slopes_of(Hq, B=None, kind="falling"):
    s = torch.tensor([2.0 ** (-8.0 * (h + 1) / Hq) for h in range(Hq)])
    if kind == "mixed":       # a zero, a negative and a steep one
        s[0], s[-1] = 0.0, 2.5
        if Hq > 2:
            s[1] = -0.01
    if B is not None:
        s = torch.stack([s * (1.0 + 0.5 * b) for b in range(B)])
    return s


def compare(got, want, name):
    g, w, tol = f64(got), want[name], want[name + "_tol"]
    assert g.shape == w.shape
    if name == "lse":
        np.testing.assert_array_equal(np.isneginf(g), np.isneginf(w))
        g, w = np.where(np.isneginf(w), 0.0, g), np.where(np.isneginf(w), 0.0, w)
    assert np.isfinite(g).all(), name
    over = np.abs(g - w) - tol
    assert over.max(initial=-1.0) <= 0, f"{name}: off by {np.abs(g - w).flat[over.argmax()]:.3e}, allowed {tol.flat[over.argmax()]:.3e}"


def check_dense(w, window, softcap, slopes, det=False, causal=None):
    causal = w.causal if causal is None else causal
    t = {n: x.cuda() for n, x in w.tensors.items()}
    sl = None if slopes is None else slopes.cuda()
    out, lse = A.flash_attn_func(t["q"], t["k"], t["v"], w.scale, causal, window, softcap, sl)
    grads = A.flash_attn_backward(t["do"], t["q"], t["k"], t["v"], out, lse, w.scale, causal, window, det, softcap, sl)
    torch.cuda.synchronize()
    assert abi.fa_get_device_status() == 0
    ref = M.attention(*(f64(w.tensors[n]) for n in ("q", "k", "v")), w.scale, causal, window, softcap,
                      None if slopes is None else slopes.numpy(), f64(w.tensors["do"]))
    for b, r in enumerate(ref):
        for name, x in zip(("o", "lse", "dq", "dk", "dv"), (out, lse) + grads):
            compare(x[b], r, name)


MODS = [(20.0, None), (0.0, "falling"), (1.5, "mixed")]


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("softcap,kind", MODS)
@pytest.mark.parametrize("Sq,Sk,causal,window,det", [
    (1, 1, True, NONE, False),
    (130, 130, True, NONE, False),
    (300, 300, True, NONE, True),
    (257, 97, True, NONE, False),          # rows without a key
    (97, 389, False, NONE, True),
    (200, 333, True, (70, -1), False),
    (333, 200, False, (50, 30), False),
])
def test_dense(D, softcap, kind, Sq, Sk, causal, window, det):
    w = W.dense(2, Sq, Sk, 4, 2, D, causal, seed=Sq + D)
    check_dense(w, window, softcap, None if kind is None else slopes_of(4, kind=kind), det)


@pytest.mark.parametrize("Hq,Hkv", [(6, 2), (5, 1), (3, 3)])
def test_grouped_heads_and_slopes_of_each_sequence(Hq, Hkv):
    w = W.dense(3, 140, 140, Hq, Hkv, 128, True, seed=Hq)
    check_dense(w, NONE, 5.0, slopes_of(Hq, B=3))


def test_scores_far_beyond_the_cap_and_around_every_tanh_branch():
    # queries scaled so that |score| / cap runs from 0 to about 30
    w = W.dense(1, 260, 260, 2, 2, 64, False, seed=9)
    w.tensors["q"][:, 130:] *= 8.0
    w.tensors["q"][:, 200:] *= 4.0
    check_dense(w, NONE, 1.0, None)
    check_dense(w, NONE, 1.0, None, det=True)


@pytest.mark.parametrize("softcap", [1e-6, 0.01, 20.0, 33.5, 50.0, 55.0, 56.0, 300.0])
@pytest.mark.parametrize("slope", [None, 0.7, -0.7])
def test_saturated_scores_on_both_sides_of_the_widest_fixed_reference(softcap, slope):
    # one key vector for all keys: rows of +c u score +cap with every key, rows of -c u score -cap, whole rows of either
    # end of the range; and rows that mix the ends
    w = W.dense(1, 190, 190, 1, 1, 64, True, seed=11)
    u = w.tensors["k"][0, :1, 0].clone()
    w.tensors["k"][0, :, 0] = u
    w.tensors["k"][0, 1::7, 0] = -u
    for i in range(190):
        w.tensors["q"][0, i, 0] = u * (-1) ** (i // 3) * max(softcap, 1.0) * (1.0 if i % 2 else 0.02)
    w.tensors["v"].mul_(1e4)
    check_dense(w, NONE, softcap, None if slope is None else torch.tensor([slope]), det=True)


@pytest.mark.parametrize("softcap,kind", MODS)
@pytest.mark.parametrize("D", [64, 128, 256])
def test_packed_batch_with_empty_sequences(D, softcap, kind):
    lq, lk = [0, 1, 130, 257, 5, 0, 64], [3, 1, 130, 100, 300, 0, 65]
    w = W.varlen(lq, lk, 4, 2, D, True, seed=D)
    t = {n: x.cuda() for n, x in w.tensors.items()}
    slopes = None if kind is None else slopes_of(4, B=len(lq), kind=kind)
    sl = None if slopes is None else slopes.cuda()
    where = (t["cu_q"], t["cu_k"], max(lq), max(lk))
    for causal, window, det in ((True, NONE, False), (False, (40, 20), True)):
        out, lse = A.flash_attn_varlen_func(t["q"], t["k"], t["v"], *where, w.scale, causal, window, softcap, sl)
        grads = A.flash_attn_varlen_backward(t["do"], t["q"], t["k"], t["v"], out, lse, *where, w.scale, causal, window,
                                             det, softcap, sl)
        torch.cuda.synchronize()
        assert abi.fa_get_device_status() == 0
        cq, ck = w.tensors["cu_q"].tolist(), w.tensors["cu_k"].tolist()
        cut = lambda n, cu: [f64(w.tensors[n])[a:b] for a, b in zip(cu, cu[1:])]  # noqa: E731
        ref = M.attention(cut("q", cq), cut("k", ck), cut("v", ck), w.scale, causal, window, softcap,
                          None if slopes is None else slopes.numpy(), cut("do", cq))
        for b, r in enumerate(ref):
            for name, x in zip(("o", "dq", "dk", "dv"), (out,) + grads):
                cu = cq if name in ("o", "dq") else ck
                compare(x[cu[b]:cu[b + 1]], r, name)
            compare(lse[:, cq[b]:cq[b + 1]], r, "lse")


def test_no_modifier_gives_the_bits_of_the_plain_call():
    w = W.dense(2, 300, 300, 4, 2, 128, True, seed=2)
    t = {n: x.cuda() for n, x in w.tensors.items()}
    out, lse = A.flash_attn_func(t["q"], t["k"], t["v"], w.scale, True)
    out0, lse0 = torch.empty_like(out), torch.empty_like(lse)
    assert abi.fa_fwd_ex(t["q"], t["k"], t["v"], out0, lse0, 2, 4, 2, 300, 300, 128, w.scale, 1, -1, -1) == 0
    assert torch.equal(out, out0) and torch.equal(lse, lse0)


def test_both_backwards_give_the_same_dk_and_dv_and_the_deterministic_one_repeats():
    for D in (64, 128, 256):
        w = W.dense(2, 333, 333, 4, 2, D, True, seed=3)
        t = {n: x.cuda() for n, x in w.tensors.items()}
        sl = slopes_of(4).cuda()
        out, lse = A.flash_attn_func(t["q"], t["k"], t["v"], w.scale, True, NONE, 3.0, sl)
        args = (t["do"], t["q"], t["k"], t["v"], out, lse, w.scale, True, NONE)
        a, b, c = (A.flash_attn_backward(*args, det, 3.0, sl) for det in (True, True, False))
        assert all(torch.equal(x, y) for x, y in zip(a, b))
        assert torch.equal(a[1], c[1]) and torch.equal(a[2], c[2])


def test_steep_slopes_over_a_long_context():
    # each row sees a handful of keys; the far ones underflow, and the reference maximum must not suffer
    w = W.dense(1, 1500, 1500, 2, 1, 64, True, seed=4)
    for causal in (True, False):
        check_dense(w, NONE, 0.0, torch.tensor([8.0, -0.05]), causal=causal)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("det", [False, True])
@pytest.mark.parametrize("Sq,Sk,window,softcap,kind", [(150, 150, (1, 0), 20.0, None), (90, 400, (2, 1), 0.0, "falling"),
                                                       (2, 300, NONE, 30.0, "falling"), (40, 40, NONE, 0.0, "mixed")])
def test_gradients_of_rows_with_few_keys(D, det, Sq, Sk, window, softcap, kind):
    # Rounding to bf16 is off by 2^-8 / sqrt(3) / m for a mantissa m in [1, 2), 1.6e-3 of the value on average.  dS, the
    # products' result and the stored gradient make three of them at most: 2.8e-3 of the norm, 4e-3 with room for a sample
    # of a few rows.  Delta from the rounded output alone would add 5e-3 here.
    w = W.dense(3, Sq, Sk, 4, 2, D, True, seed=D + Sq)
    w.tensors["q"].mul_(2)
    t = {n: x.cuda() for n, x in w.tensors.items()}
    slopes = None if kind is None else slopes_of(4, kind=kind)
    sl = None if slopes is None else slopes.cuda()
    out, lse = A.flash_attn_func(t["q"], t["k"], t["v"], w.scale, True, window, softcap, sl)
    grads = A.flash_attn_backward(t["do"], t["q"], t["k"], t["v"], out, lse, w.scale, True, window, det, softcap, sl)
    ref = M.attention(*(f64(w.tensors[n]) for n in ("q", "k", "v")), w.scale, True, window, softcap,
                      None if slopes is None else slopes.numpy(), f64(w.tensors["do"]))
    for name, x in zip(("dq", "dk", "dv"), grads):
        want = np.stack([r[name] for r in ref])
        assert np.linalg.norm(f64(x) - want) <= 4e-3 * np.linalg.norm(want), name


def test_captured_replayed_and_on_another_stream():
    w = W.dense(2, 200, 200, 4, 2, 128, True, seed=5)
    t = {n: x.cuda() for n, x in w.tensors.items()}
    sl = slopes_of(4).cuda()

    def step():
        out, lse = A.flash_attn_func(t["q"], t["k"], t["v"], w.scale, True, NONE, 4.0, sl)
        return (out, lse) + A.flash_attn_backward(t["do"], t["q"], t["k"], t["v"], out, lse, w.scale, True, NONE, True, 4.0, sl)

    want = [x.clone() for x in step()]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = step()
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step()
    t["q"].mul_(0.5)
    g.replay()
    torch.cuda.synchronize()
    half = [x.clone() for x in got]
    assert all(torch.equal(a, b) for a, b in zip(half, step()))
    assert not torch.equal(half[0], want[0])


def test_autograd_and_slopes_without_a_gradient():
    w = W.dense(2, 130, 130, 4, 2, 64, True, seed=6)
    t = {n: x.cuda() for n, x in w.tensors.items()}
    q, k, v = (t[n].requires_grad_() for n in "qkv")
    sl = slopes_of(4)
    out = A.FlashAttnFunction.apply(q, k, v, w.scale, True, NONE, True, 6.0, sl.cuda())
    out.backward(t["do"])
    ref = M.attention(*(f64(w.tensors[n]) for n in ("q", "k", "v")), w.scale, True, NONE, 6.0, sl.numpy(), f64(w.tensors["do"]))
    for b, r in enumerate(ref):
        compare(out[b], r, "o")
        for name, x in (("dq", q), ("dk", k), ("dv", v)):
            compare(x.grad[b], r, name)
    with pytest.raises(ValueError):
        A.FlashAttnFunction.apply(q, k, v, w.scale, True, NONE, True, 0.0, sl.cuda().requires_grad_())


def test_bad_slopes_are_refused():
    q = torch.zeros(2, 8, 4, 64, dtype=torch.bfloat16, device="cuda")
    z = lambda *shape: torch.zeros(shape, device="cuda")  # noqa: E731
    for bad, err in ((z(3), ValueError), (z(3, 4), ValueError), (z(4).half(), TypeError), (z(8)[::2], ValueError)):
        with pytest.raises(err):
            A.flash_attn_func(q, q, q, alibi_slopes=bad)
    with pytest.raises(ValueError):
        A.flash_attn_func(q, q, q, alibi_slopes=torch.zeros(4))
    for cap in (-1.0, math.nan, math.inf):
        with pytest.raises(abi.FAError):
            A.flash_attn_func(q, q, q, softcap=cap)


# ------------------------------------------------------------------------------------------- KV cache
def check_cache(w, causal, window, softcap, slopes, num_splits=0):
    t = w.tensors
    dev = {n: x.cuda() for n, x in t.items()}
    out, lse = A.flash_attn_with_kvcache(dev["q"], dev["k_cache"], dev["v_cache"], dev["cache_seqlens"], w.scale, causal,
                                         num_splits, True, dev.get("k_new"), dev.get("v_new"), dev.get("cache_batch_idx"),
                                         dev.get("block_table"), window, softcap, None if slopes is None else slopes.cuda())
    torch.cuda.synchronize()
    assert abi.fa_get_device_status() == 0
    kc, vc = f64(dev["k_cache"]), f64(dev["v_cache"])       # after the append
    sn = w.meta["seqlen_new"]
    keys, vals = [], []
    for b, n in enumerate(t["cache_seqlens"].tolist()):
        n += sn
        if w.meta["page"]:
            rows = t["block_table"][b].long().numpy()
            keys.append(kc[rows].reshape(-1, *kc.shape[2:])[:n])
            vals.append(vc[rows].reshape(-1, *vc.shape[2:])[:n])
        else:
            keys.append(kc[b, :n])
            vals.append(vc[b, :n])
    ref = M.attention(list(f64(t["q"])), keys, vals, w.scale, causal, window, softcap,
                      None if slopes is None else slopes.numpy())
    for b, r in enumerate(ref):
        compare(out[b], r, "o")
        compare(lse[b], r, "lse")


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("softcap,kind", MODS)
@pytest.mark.parametrize("Sq,new,page,causal,window", [
    (1, 0, 0, False, NONE), (1, 1, 256, True, NONE), (3, 3, 0, True, (100, -1)), (5, 2, 256, False, (33, 12)),
])
def test_cache(D, softcap, kind, Sq, new, page, causal, window):
    lens = [0, 1, 63, 255, 256, 700]
    w = W.kvcache_update(len(lens), Sq, 8, 2, D, 1024, lens, seqlen_new=new, page=page, seed=D + Sq)
    slopes = None if kind is None else slopes_of(8, B=len(lens), kind=kind)
    check_cache(w, causal, window, softcap, slopes)


@pytest.mark.parametrize("num_splits", [1, 3, 16])
def test_cache_does_not_depend_on_the_split(num_splits):
    w = W.kvcache_update(2, 4, 7, 7, 128, 2048, [2044, 513], seqlen_new=4, seed=8)
    check_cache(w, True, NONE, 8.0, slopes_of(7), num_splits)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("softcap,kind", MODS + [(80.0, "falling")])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_rows_outside_a_sequence_do_not_reach_it(D, softcap, kind, bad):
    """A neighbouring sequence full of NaN or infinities, and such padding behind the last one, change no bit of the
    others (dq of the backward that adds in any order: within two roundings)."""
    lq, lk = [130, 57, 70], [140, 57, 33]
    w = W.varlen(lq + [20], lk + [20], 4, 2, D, True, seed=D)
    good = {n: x.cuda() for n, x in w.tensors.items()}
    cq, ck = (torch.tensor(np.cumsum([0] + n), dtype=torch.int32) for n in (lq, lk))
    filled = {n: x.clone() for n, x in good.items()}
    for n, cu in (("q", cq), ("k", ck), ("v", ck), ("do", cq)):
        filled[n][cu[1]:cu[2]] = bad
        filled[n][cu[3]:] = bad
    sl = None if kind is None else slopes_of(4, kind=kind).cuda()
    where = (cq.cuda(), ck.cuda(), max(lq), max(lk))
    for causal, window, det in ((True, NONE, True), (False, (20, 10), False), (False, (3, 2), True)):
        res = []
        for t in (good, filled):
            out, lse = A.flash_attn_varlen_func(t["q"], t["k"], t["v"], *where, w.scale, causal, window, softcap, sl)
            res.append((out, lse.t()) + A.flash_attn_varlen_backward(t["do"], t["q"], t["k"], t["v"], out, lse, *where,
                                                                     w.scale, causal, window, det, softcap, sl))
        assert abi.fa_get_device_status() == 0
        for name, a, b, cu in zip(("o", "lse", "dq", "dk", "dv"), *res, (cq, cq, cq, ck, ck)):
            for s in (0, 2):
                x, y = a[cu[s]:cu[s + 1]], b[cu[s]:cu[s + 1]]
                if name == "dq" and not det:
                    assert ((x.float() - y.float()).abs() <= 2.0 ** -7 * x.float().abs() + 1e-5).all()
                else:
                    assert torch.equal(x, y), name


@pytest.mark.parametrize("D", [64, 128, 256])
def test_padding_behind_the_last_sequence_is_left_as_it_was(D):
    lq, lk = [3, 130], [130, 65]
    w = W.varlen(lq + [9], lk + [9], 4, 2, D, True, seed=D + 1)
    t = {n: x.cuda() for n, x in w.tensors.items()}
    cq, ck = (torch.tensor(np.cumsum([0] + n), dtype=torch.int32).cuda() for n in (lq, lk))
    out, lse = torch.full_like(t["q"], 7.0), torch.full((4, t["q"].shape[0]), 7.0, device="cuda")
    grads = [torch.full_like(t[n], 7.0) for n in ("q", "k", "v")]
    sl = slopes_of(4).cuda()
    nb = abi.fa_varlen_bwd_workspace_size(2, t["q"].shape[0], t["k"].shape[0], 4, 2, D)
    ws = torch.empty(max(nb, 256), dtype=torch.uint8, device="cuda")
    sizes = (2, max(lq), max(lk), t["q"].shape[0], t["k"].shape[0], 4, 2, D, w.scale, True, -1, -1)
    assert abi.fa_varlen_fwd_mod(t["q"], t["k"], t["v"], out, lse, cq, ck, *sizes, 5.0, sl, 0, ws, nb) == 0
    for det in (False, True):
        assert abi.fa_varlen_bwd_mod(t["q"], t["k"], t["v"], out, t["do"], lse, *grads, cq, ck, *sizes, det, 5.0, sl, 0, ws, nb) == 0
        for x, n in ((out, 133), (lse.t(), 133), (grads[0], 133), (grads[1], 195), (grads[2], 195)):
            # the backward that adds into an fp32 dq converts all of its rows: zeros there, with and without modifiers
            zeros = x is grads[0] and not det
            assert (x[n:] == (0.0 if zeros else 7.0)).all() and (x[:n] != 7.0).any()
            if zeros:
                x.fill_(7.0)
    assert abi.fa_get_device_status() == 0
