"""Rotary positions on the GPU against the fp64 oracle: the stand-alone rotation and its gradient, the tables, the
cache call that rotates for itself, and a training step and a decoding loop that use them together."""

import numpy as np
import pytest
import torch

import oracle.modifiers as M
from exact_tiled_attention_41_b200 import abi, attention as A, workloads as W
from tests.gpu_helpers import f64

pytestmark = pytest.mark.gpu


def normal(seed, *shape):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16)


def tables(rows, rd):
    cos, sin = M.rotary_tables(rows, rd)
    cos, sin = torch.tensor(cos, dtype=torch.float32), torch.tensor(sin, dtype=torch.float32)
    return cos, sin, f64(cos), f64(sin)


def check(y, x, cos, sin, positions, interleaved, inverse=False):
    want = M.rotate(x, cos, sin, positions, interleaved, inverse)
    tol = M.rotate_tol(x, want, cos, sin, positions, interleaved)
    assert (np.abs(f64(y) - want) <= tol).all()
    rd = 2 * cos.shape[1]
    np.testing.assert_array_equal(f64(y)[..., rd:], x[..., rd:])


@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("D,rd", [(64, 64), (64, 16), (64, 48), (128, 128), (128, 96), (256, 256), (256, 80)])
@pytest.mark.parametrize("B,S,H", [(1, 1, 1), (2, 7, 3), (3, 33, 16), (2, 65, 40)])
def test_dense(interleaved, D, rd, B, S, H):
    x = normal(D + rd + S, B, S, H, D)
    cos, sin, c, s = tables(S + 9, rd)
    off = torch.arange(B, dtype=torch.int32) * 4
    pos = (np.arange(S)[None, :] + off.numpy()[:, None]).reshape(-1)
    flat = f64(x).reshape(-1, H, D)
    for inverse in (False, True):
        y = A.apply_rotary(x.cuda(), cos.cuda(), sin.cuda(), off.cuda(), interleaved, inverse)
        check(y.reshape(-1, H, D), flat, c, s, pos, interleaved, inverse)
    y = A.apply_rotary(x.cuda(), cos.cuda(), sin.cuda(), 9, interleaved)
    check(y.reshape(-1, H, D), flat, c, s, np.tile(np.arange(S) + 9, B), interleaved)
    assert abi.fa_get_device_status() == 0


@pytest.mark.parametrize("interleaved", [True, False])
def test_strided_in_place_and_transposed(interleaved):
    cos, sin, c, s = tables(40, 32)
    qkv = normal(1, 2, 33, 9, 64)
    dev = qkv.cuda()
    part = dev[:, :, 2:7]
    y = A.apply_rotary(part, cos.cuda(), sin.cuda(), 0, interleaved)
    pos = np.tile(np.arange(33), 2)
    check(y.reshape(-1, 5, 64), f64(qkv)[:, :, 2:7].reshape(-1, 5, 64), c, s, pos, interleaved)
    assert A.apply_rotary(part, cos.cuda(), sin.cuda(), 0, interleaved, out=part) is part
    assert torch.equal(part, y)
    assert torch.equal(dev[:, :, :2].cpu(), qkv[:, :, :2]) and torch.equal(dev[:, :, 7:].cpu(), qkv[:, :, 7:])
    heads_first = qkv[:, :, 2:7].cuda().permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3)   # (B, H, S, D) in memory
    out = torch.empty_like(heads_first)
    A.apply_rotary(heads_first, cos.cuda(), sin.cuda(), 0, interleaved, out=out)
    assert torch.equal(out, y)
    wide = qkv[:, :1, :1].cuda().expand(2, 33, 5, 64)                                          # broadcast input
    y = A.apply_rotary(wide, cos.cuda(), sin.cuda(), 0, interleaved)
    check(y.reshape(-1, 5, 64), f64(wide).reshape(-1, 5, 64), c, s, pos, interleaved)


@pytest.mark.parametrize("interleaved", [True, False])
def test_packed_batch(interleaved):
    lens = [0, 5, 0, 1, 70, 33, 0]
    total = sum(lens)
    cu = torch.tensor(np.cumsum([0] + lens), dtype=torch.int32)
    x = normal(2, total + 6, 4, 128)          # six rows behind the last sequence
    cos, sin, c, s = tables(90, 64)
    off = torch.tensor([3, 0, 1, 17, 2, 11, 4], dtype=torch.int32)
    pos = np.concatenate([np.arange(n) + o for n, o in zip(lens, off.tolist())])
    out = torch.full_like(x, 7.0).cuda()
    A.apply_rotary(x.cuda(), cos.cuda(), sin.cuda(), off.cuda(), interleaved, cu_seqlens=cu.cuda(), out=out)
    check(out[:total], f64(x)[:total], c, s, pos, interleaved)
    assert (out[total:] == 7.0).all()
    many = torch.arange(0, total + 1, dtype=torch.int32)      # as many sequences as tokens
    y = A.apply_rotary(x.cuda(), cos.cuda(), sin.cuda(), 5, interleaved, cu_seqlens=many.cuda())
    check(y[:total], f64(x)[:total], c, s, np.full(total, 5), interleaved)
    empty = A.apply_rotary(x.cuda()[:0], cos.cuda(), sin.cuda(), cu_seqlens=cu.cuda() * 0)
    assert empty.shape == (0, 4, 128)
    assert abi.fa_get_device_status() == 0


def test_positions_outside_the_tables_are_reported_and_become_zeros():
    x = normal(3, 2, 6, 2, 64).cuda()
    cos, sin, c, s = tables(8, 32)
    y = A.apply_rotary(x, cos.cuda(), sin.cuda(), torch.tensor([4, -2], dtype=torch.int32).cuda())
    torch.cuda.synchronize()
    assert abi.fa_get_device_status() == abi.FA_ERR_INVALID_ARG
    assert (y[0, 4:, :, :32] == 0).all() and (y[1, :2, :, :32] == 0).all()
    assert torch.equal(y[..., 32:], x[..., 32:])
    check(y[0, :4], f64(x[0, :4]), c, s, np.arange(4, 8), True)
    check(y[1, 2:], f64(x[1, 2:]), c, s, np.arange(4), True)
    assert abi.fa_get_device_status() == 0


@pytest.mark.parametrize("rows,rd", [(1, 16), (77, 32), (4097, 64), (33, 256)])
@pytest.mark.parametrize("scaling", ["none", "linear", "base", "by_parts"])
def test_tables(rows, rd, scaling):
    kw = dict(factor=7.5, amplitude=1.2) if scaling != "none" else {}
    cos, sin = A.rotary_tables(rows, rd, 50000.0, scaling, original_seqlen=2048, low_rotations=1.0, high_rotations=20.0, **kw)
    c, s = M.rotary_tables(rows, rd, 50000.0, scaling, original=2048, low=1.0, high=20.0, **kw)
    assert cos.shape == (rows, rd // 2) and cos.is_contiguous() and sin.is_contiguous()
    # the angle to 2^-25 of a half turn (times pi), sine and cosine to 3 half steps of fp32 at 1, one product
    for got, want in ((cos, c), (sin, s)):
        assert np.abs(f64(got) - want).max() <= 1.2 * (np.pi * 2.0 ** -25 + 3 * 2.0 ** -24)


def test_tables_at_far_positions():
    # 2^20 positions: an fp32 product of position and frequency would be off by 0.06
    rows, rd = (1 << 20) + 3, 32
    cos, sin = A.rotary_tables(rows, rd)
    f = 10000.0 ** (-2 * np.arange(rd // 2, dtype=np.longdouble) / rd)
    for p in (0, 1, 131071, rows - 1):
        np.testing.assert_allclose(f64(cos[p]), np.cos(p * f).astype(float), atol=3e-7)
        np.testing.assert_allclose(f64(sin[p]), np.sin(p * f).astype(float), atol=3e-7)


def test_gradient_is_the_opposite_rotation():
    x = normal(4, 2, 9, 3, 64).cuda().requires_grad_()
    cos, sin, c, s = tables(32, 48)
    off = torch.tensor([2, 20], dtype=torch.int32).cuda()
    for interleaved in (True, False):
        x.grad = None
        y = A.RotaryFunction.apply(x, cos.cuda(), sin.cuda(), off, interleaved)
        dy = normal(5, 2, 9, 3, 64)
        y.backward(dy.cuda())
        pos = np.concatenate([np.arange(9) + 2, np.arange(9) + 20])
        check(x.grad.reshape(-1, 3, 64), f64(dy).reshape(-1, 3, 64), c, s, pos, interleaved, inverse=True)
        # and the difference quotient along a direction: the rotation is linear
        d = f64(normal(6, 2, 9, 3, 64)).reshape(-1, 3, 64)
        lin = (M.rotate(d, c, s, pos, interleaved) * f64(dy).reshape(-1, 3, 64)).sum()
        assert abs((f64(x.grad).reshape(-1, 3, 64) * d).sum() - lin) <= 2.0 ** -8 * np.abs(f64(x.grad).reshape(-1, 3, 64) * d).sum()


@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("D,rd", [(64, 64), (128, 32), (256, 144)])
@pytest.mark.parametrize("page", [0, 256])
@pytest.mark.parametrize("Sq,new,causal,window", [(1, 1, False, (-1, -1)), (3, 3, True, (-1, -1)), (2, 5, False, (50, -1)),
                                                   (4, 1, False, (-1, -1))])
def test_the_cache_call_gives_the_bits_of_the_separate_calls(interleaved, D, rd, page, Sq, new, causal, window):
    lens = [0, 1, 250, 600]
    w = W.kvcache_update(4, Sq, 8, 2, D, 1024, lens, seqlen_new=new, page=page, seed=D + Sq)
    t = {n: x.cuda() for n, x in w.tensors.items()}
    cos, sin, _, _ = tables(1024, rd)
    cos, sin = cos.cuda(), sin.cuda()
    rest = dict(block_table=t.get("block_table"), window_size=window, softcap=9.0)
    kc, vc = t["k_cache"].clone(), t["v_cache"].clone()
    q0 = t["q"].clone()
    out, lse = A.flash_attn_with_kvcache(t["q"], kc, vc, t["cache_seqlens"], w.scale, causal, k=t["k_new"], v=t["v_new"],
                                         rotary_cos=cos, rotary_sin=sin, rotary_interleaved=interleaved, **rest)
    assert torch.equal(t["q"], q0)
    k = A.apply_rotary(t["k_new"], cos, sin, t["cache_seqlens"], interleaved)
    if causal or window != (-1, -1):
        q = A.apply_rotary(t["q"], cos, sin, t["cache_seqlens"], interleaved)
    else:
        q = A.apply_rotary(t["q"].transpose(0, 1).reshape(Sq * 4, 1, 8, D), cos, sin, t["cache_seqlens"].repeat(Sq), interleaved)
        q = q.reshape(Sq, 4, 8, D).transpose(0, 1).contiguous()
    kc2, vc2 = t["k_cache"].clone(), t["v_cache"].clone()
    out2, lse2 = A.flash_attn_with_kvcache(q, kc2, vc2, t["cache_seqlens"], w.scale, causal, k=k, v=t["v_new"], **rest)
    assert torch.equal(out, out2) and torch.equal(lse, lse2)
    assert torch.equal(kc.view(torch.int16), kc2.view(torch.int16)) and torch.equal(vc.view(torch.int16), vc2.view(torch.int16))
    assert abi.fa_get_device_status() == 0


def test_cache_rows_by_index_and_a_full_cache():
    # cache rows named by cache_batch_idx; a sequence without room keeps its cache and attends to what it holds
    lens = [5, 64, 63]
    w = W.kvcache_update(3, 1, 4, 2, 64, 64, lens, seqlen_new=1, seed=2, cache_batch_idx=[4, 0, 2], cache_batch=5)
    t = {n: x.cuda() for n, x in w.tensors.items()}
    cos, sin, _, _ = tables(65, 32)
    cos, sin = cos.cuda(), sin.cuda()
    kc, vc = t["k_cache"].clone(), t["v_cache"].clone()
    out, lse = A.flash_attn_with_kvcache(t["q"], kc, vc, t["cache_seqlens"], w.scale, True, k=t["k_new"], v=t["v_new"],
                                         cache_batch_idx=t["cache_batch_idx"], rotary_cos=cos, rotary_sin=sin)
    q = A.apply_rotary(t["q"], cos, sin, t["cache_seqlens"])
    k = A.apply_rotary(t["k_new"], cos, sin, t["cache_seqlens"])
    kc2, vc2 = t["k_cache"].clone(), t["v_cache"].clone()
    out2, lse2 = A.flash_attn_with_kvcache(q, kc2, vc2, t["cache_seqlens"], w.scale, True, k=k, v=t["v_new"],
                                           cache_batch_idx=t["cache_batch_idx"])
    assert torch.equal(out, out2) and torch.equal(lse, lse2)
    assert torch.equal(kc.view(torch.int16), kc2.view(torch.int16)) and torch.equal(vc.view(torch.int16), vc2.view(torch.int16))
    assert torch.equal(kc[0].view(torch.int16), t["k_cache"][0].view(torch.int16))     # the full row
    assert not torch.equal(kc[4, 5], t["k_cache"][4, 5]) and abi.fa_get_device_status() == 0


def test_cache_call_reports_positions_past_the_tables():
    w = W.kvcache_update(2, 1, 4, 2, 64, 512, [100, 300], seqlen_new=1, seed=1)
    t = {n: x.cuda() for n, x in w.tensors.items()}
    cos, sin, _, _ = tables(200, 64)
    A.flash_attn_with_kvcache(t["q"], t["k_cache"], t["v_cache"], t["cache_seqlens"], w.scale, k=t["k_new"], v=t["v_new"],
                              rotary_cos=cos.cuda(), rotary_sin=sin.cuda())
    torch.cuda.synchronize()
    assert abi.fa_get_device_status() == abi.FA_ERR_INVALID_ARG
    assert (t["k_cache"][1, 300] == 0).all() and (t["k_cache"][0, 100] != 0).any()
    assert torch.equal(t["v_cache"][1, 300], t["v_new"][1, 0])


def test_refusals():
    x = torch.zeros(2, 4, 2, 64, dtype=torch.bfloat16, device="cuda")
    cos = torch.zeros(16, 16, device="cuda")
    bad = [
        (ValueError, dict(cos=cos[:, :12].contiguous(), sin=cos[:, :12].contiguous())),      # rotary_dim 24
        (ValueError, dict(cos=cos, sin=cos[:8].contiguous())),
        (ValueError, dict(cos=cos.cpu(), sin=cos.cpu())),
        (ValueError, dict(cos=torch.zeros(16, 40, device="cuda"), sin=torch.zeros(16, 40, device="cuda"))),
        (TypeError, dict(cos=cos.half(), sin=cos.half())),
        (TypeError, dict(x=x.float())),
        (ValueError, dict(x=x[0])),
        (ValueError, dict(x=x.transpose(2, 3).contiguous().transpose(2, 3))),                # head dimension not contiguous
        (ValueError, dict(seqlen_offsets=torch.zeros(3, dtype=torch.int32, device="cuda"))),
        (TypeError, dict(seqlen_offsets=torch.zeros(2, dtype=torch.int64, device="cuda"))),
        (ValueError, dict(out=torch.zeros(2, 4, 2, 128, dtype=torch.bfloat16, device="cuda"))),
        (abi.FAError, dict(out=torch.zeros(2, 4, 1, 64, dtype=torch.bfloat16, device="cuda").expand(2, 4, 2, 64))),
        (abi.FAError, dict(seqlen_offsets=-1)),
        (abi.FAError, dict(x=torch.zeros(2, 4, 2, 96, dtype=torch.bfloat16, device="cuda"))),
        (abi.FAError, dict(x=torch.zeros(2 * 4 * 2 * 64 + 4, dtype=torch.bfloat16, device="cuda")[4:].view(2, 4, 2, 64))),
    ]
    for err, kw in bad:
        args = dict(x=x, cos=cos, sin=cos)
        args.update(kw)
        with pytest.raises(err):
            A.apply_rotary(**args)
    with pytest.raises(ValueError):
        A.rotary_tables(16, 32, scaling="quadratic")
    for kw in (dict(rotary_dim=24), dict(base=1.0), dict(scaling="linear", factor=0.5), dict(scaling="by_parts", factor=2.0),
               dict(seqlen=0), dict(rotary_dim=512)):
        with pytest.raises(abi.FAError):
            A.rotary_tables(**{**dict(seqlen=16, rotary_dim=32), **kw})
    q = torch.zeros(1, 1, 2, 64, dtype=torch.bfloat16, device="cuda")
    cache = torch.zeros(1, 64, 2, 64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(abi.FAError):      # rotary needs the new keys
        A.flash_attn_with_kvcache(q, cache, cache.clone(), 3, rotary_cos=cos, rotary_sin=cos)
    with pytest.raises(ValueError):
        A.flash_attn_with_kvcache(q, cache, cache.clone(), 3, k=q, v=q, rotary_cos=cos)
    with pytest.raises(ValueError):       # new keys of another head count
        A.flash_attn_with_kvcache(q, cache, cache.clone(), 3, k=q[:, :, :1].contiguous(), v=q[:, :, :1].contiguous())


def test_training_step_through_rotary_and_capped_attention():
    B, S, Hq, Hkv, D, rd, cap = 2, 150, 4, 2, 64, 32, 4.0
    qkv0, do = normal(7, B, S, Hq + 2 * Hkv, D), normal(8, B, S, Hq, D)
    cos, sin = A.rotary_tables(S, rd)
    slopes = torch.tensor([0.5, 0.25, 0.1, 0.02], device="cuda")
    qkv = qkv0.cuda().requires_grad_()
    qk = A.RotaryFunction.apply(qkv[:, :, :Hq + Hkv], cos, sin, 0, False)
    q, k, v = qk[:, :, :Hq].contiguous(), qk[:, :, Hq:].contiguous(), qkv[:, :, Hq + Hkv:].contiguous()
    out = A.FlashAttnFunction.apply(q, k, v, None, True, (-1, -1), False, cap, slopes)
    out.backward(do.cuda())
    # the oracle on the queries and keys that the rotation gave; then the rotation of its gradients back
    ref = M.attention(f64(q), f64(k), f64(v), D ** -0.5, True, (-1, -1), cap, f64(slopes), f64(do))
    c, s = f64(cos), f64(sin)
    g = f64(qkv.grad)
    for b, r in enumerate(ref):
        assert (np.abs(f64(out[b]) - r["o"]) <= r["o_tol"]).all()
        d = np.concatenate([r["dq"], r["dk"]], 1)
        tol = np.concatenate([r["dq_tol"], r["dk_tol"]], 1)
        want = M.rotate(d, c, s, np.arange(S), False, inverse=True)
        # each value mixes two: bounded by both tolerances, and one more rounding
        spread = np.abs(M.rotate(tol, np.abs(c), -np.abs(s), np.arange(S), False)) + np.abs(M.rotate(tol, np.abs(c), np.abs(s), np.arange(S), False)) \
            + M.rotate_tol(d, want, c, s, np.arange(S), False)
        assert (np.abs(g[b, :, :Hq + Hkv] - want) <= spread).all()
        assert (np.abs(g[b, :, Hq + Hkv:] - r["dv"]) <= r["dv_tol"]).all()


def test_decoding_loop_matches_the_prompt_in_one_pass():
    # tokens one by one through the cache call = one causal pass over the rotated sequence
    B, S, Hq, Hkv, D, rd, cap = 2, 40, 4, 2, 128, 64, 5.0
    q, k, v = (normal(i, B, S, h, D).cuda() for i, h in ((9, Hq), (10, Hkv), (11, Hkv)))
    cos, sin = A.rotary_tables(64, rd)
    slopes = torch.tensor([0.3, 0.1, 0.05, 0.01], device="cuda")
    kc, vc = torch.zeros(B, 64, Hkv, D, dtype=torch.bfloat16, device="cuda"), torch.zeros(B, 64, Hkv, D, dtype=torch.bfloat16, device="cuda")
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    outs = []
    for i in range(S):
        o, _ = A.flash_attn_with_kvcache(q[:, i:i + 1].contiguous(), kc, vc, lens, causal=True, k=k[:, i:i + 1].contiguous(),
                                         v=v[:, i:i + 1].contiguous(), rotary_cos=cos, rotary_sin=sin, softcap=cap,
                                         alibi_slopes=slopes)
        lens += 1
        outs.append(o)
    qr, kr = A.apply_rotary(q, cos, sin), A.apply_rotary(k, cos, sin)
    assert torch.equal(kc[:, :S], kr)
    ref = M.attention(f64(qr), f64(kr), f64(v), D ** -0.5, True, (-1, -1), cap, f64(slopes))
    out = f64(torch.cat(outs, 1))
    full, _ = A.flash_attn_func(qr, kr, v, None, True, (-1, -1), cap, slopes)
    for b, r in enumerate(ref):
        assert (np.abs(out[b] - r["o"]) <= r["o_tol"]).all()
        assert (np.abs(f64(full[b]) - r["o"]) <= r["o_tol"]).all()


def test_captured_cache_call_replays_at_the_next_length():
    B, Hq, Hkv, D = 2, 4, 2, 64
    q, k, v = (normal(i, B, 1, h, D).cuda() for i, h in ((12, Hq), (13, Hkv), (14, Hkv)))
    cos, sin = A.rotary_tables(64, 64)
    kc, vc = normal(15, B, 64, Hkv, D).cuda(), normal(16, B, 64, Hkv, D).cuda()
    lens = torch.tensor([5, 17], dtype=torch.int32, device="cuda")
    step = lambda a, b: A.flash_attn_with_kvcache(q, a, b, lens, k=k, v=v, rotary_cos=cos, rotary_sin=sin, softcap=3.0)  # noqa: E731
    step(kc.clone(), vc.clone())
    ka, va = kc.clone(), vc.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out, lse = step(ka, va)
    for _ in range(3):
        g.replay()
        want, wl = step(kc, vc)
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(lse, wl) and torch.equal(ka, kc) and torch.equal(va, vc)
        lens += 1


@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("rd", [64, 32])
def test_padding_of_a_packed_batch_gets_zeros_in_new_tensors(interleaved, rd):
    """Rows behind the last sequence (and before the first) are zeros in a new output and in the gradient, whatever
    the memory held."""
    cos, sin, c, s = tables(40, rd)
    cu = torch.tensor([2, 30, 30, 41], dtype=torch.int32).cuda()
    x = normal(21, 60, 3, 64).cuda().requires_grad_()
    pos = np.concatenate([np.arange(28), np.arange(11)])
    dy = normal(22, 60, 3, 64)
    dy[41:] = float("nan")
    dy = dy.cuda()
    poison = [torch.full_like(x, float("nan"), requires_grad=False) for _ in range(4)]
    del poison                                        # the next tensors of this size lie there
    y = A.RotaryFunction.apply(x, cos.cuda(), sin.cuda(), 0, interleaved, cu)
    g, = torch.autograd.grad(y, x, dy)
    for t, src, inverse in ((y.detach(), x.detach(), False), (g, dy, True)):
        assert (t[:2] == 0).all() and (t[41:] == 0).all()
        check(t[2:41], f64(src)[2:41], c, s, pos, interleaved, inverse=inverse)


def test_rotary_gradient_is_first_order():
    cos, sin, _, _ = tables(8, 32)
    x = normal(23, 1, 4, 2, 64).cuda().requires_grad_()
    y = A.RotaryFunction.apply(x, cos.cuda(), sin.cuda())
    g, = torch.autograd.grad(y, x, torch.ones_like(y, requires_grad=True), create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        g.sum().backward()
