"""Cases for measuring attention with capped and biased scores, and rotary positions.

Three kinds of operator, each in its plain form (``own`` false: elementary torch operations) and through
the framework's entry points (``own`` true):

* attention whose scores are capped by a tanh and / or biased by the distance of query and key:
      x_ij = cap tanh(scale q_i.k_j / cap) - slope_h |i + Lk - Lq - j|,   O = softmax(x) V
  as a training step (forward and gradients; equal lengths or packed sequences), as a forward pass over a
  chunk of a long prompt, and against a KV cache;
* rotary positions applied to queries and keys, their gradient, and the same inside the cache call, which
  rotates the new queries and keys and appends the keys and values;
* the cos / sin tables of those positions, scaled for long contexts.
"""

import math

import numpy as np
import torch

own = False


# --------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # the dense prefill workload of bench.py as a training step with capped scores
        dict(name="train_cap_dense", op="train", n=4, lo=2048, hi=2048, sq=0, hq=16, hkv=16, d=128, causal=True,
             wl=-1, wr=-1, cap=30.0, alibi=False, det=False, packed=False, lens=0),
        # a long training step with grouped heads and a distance bias: the largest
        dict(name="train_alibi_gqa", op="train", n=2, lo=4096, hi=4096, sq=0, hq=32, hkv=8, d=128, causal=True,
             wl=-1, wr=-1, cap=0.0, alibi=True, det=False, packed=False, lens=0),
        # a packed batch of unequal documents, both modifiers, the widest heads
        dict(name="train_both_packed", op="train", n=16, lo=128, hi=2048, sq=0, hq=16, hkv=16, d=256, causal=True,
             wl=-1, wr=-1, cap=50.0, alibi=True, det=False, packed=True, lens=7),
        # a small odd step: more queries than keys (the first rows see no key), a window, reproducible gradients
        dict(name="train_small_odd", op="train", n=3, lo=97, hi=97, sq=150, hq=6, hkv=2, d=64, causal=True,
             wl=40, wr=-1, cap=20.0, alibi=True, det=True, packed=False, lens=0),
        # one chunk of a long prompt against the keys before it, window on the left, forward only
        dict(name="prefill_cap_window", op="prefill", n=1, lo=8192, hi=8192, sq=1024, hq=32, hkv=8, d=64,
             causal=True, wl=4096, wr=-1, cap=50.0, alibi=False, det=False, packed=False, lens=0),
        # one user's next token: latency
        dict(name="decode_one", op="decode", n=1, lo=1234, hi=1234, cap_keys=4096, page=0, sq=1, new=1, hq=16,
             hkv=4, d=128, causal=False, wl=-1, cap=30.0, alibi=False, rd=64, inter=False, lens=0),
        # a serving batch on pages: rotary, append and capped scores in one call
        dict(name="decode_paged", op="decode", n=32, lo=1024, hi=8192, cap_keys=8448, page=256, sq=1, new=1, hq=32,
             hkv=8, d=128, causal=True, wl=-1, cap=30.0, alibi=False, rd=128, inter=True, lens=3),
        # four tokens at once (drafted ones being checked) with a distance bias, wide heads, contiguous cache
        dict(name="decode_alibi_tokens", op="decode", n=16, lo=512, hi=2048, cap_keys=2052, page=0, sq=4, new=4,
             hq=16, hkv=16, d=256, causal=True, wl=-1, cap=0.0, alibi=True, rd=0, inter=False, lens=5),
        # queries and keys of a training step, a slice of the packed projection; and their gradient
        dict(name="rotary_train", op="rotary", n=4, lo=2048, hi=2048, h=32, spare=16, d=128, rd=128, inter=False,
             offset=0, packed=False, lens=0),
        # the new tokens of a small serving batch: latency; positions differ for each sequence
        dict(name="rotary_tokens", op="rotary", n=8, lo=1, hi=1, h=32, spare=0, d=64, rd=32, inter=True,
             offset=1000, packed=False, lens=0),
        # the table of an ordinary context
        dict(name="table_short", op="table", rows=4096, rd=64, scaling="none"),
        # the table of a context 32 times as long as the original one
        dict(name="table_long", op="table", rows=131072, rd=128, scaling="by_parts"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["train", "train", "train", "prefill", "decode", "decode", "decode", "rotary", "rotary", "table"])
    d = rng.choice([64, 128, 256])
    hkv = rng.choice([1, 2, 3, 4, 8])
    hq = hkv * rng.choice([1, 1, 2, 3, 4, 8])
    cap, alibi = rng.choice([(0.0, True), (20.0, False), (30.0, True), (50.0, False), (50.0, True)])
    if op in ("train", "prefill"):
        packed = rng.random() < 0.5
        n = _log(rng, 1, 16)
        hi = _log(rng, 17, 4096)
        while n * hq * hi * hi > 4e8:   # keeps the plain form's scores at a few GB
            hi = max(1, int(hi * 0.8))
        lo = rng.choice([0, 1, hi // 2]) if packed else hi
        sq = 0 if packed or rng.random() < 0.5 else _log(rng, 1, hi)
        causal = rng.random() < 0.6
        wl = rng.choice([-1, -1, _log(rng, 1, 1024)])
        wr = -1 if causal else rng.choice([-1, -1, _log(rng, 1, 256)])
        return dict(op=op, n=n, lo=lo, hi=hi, sq=sq, hq=hq, hkv=hkv, d=d, causal=causal, wl=wl, wr=wr, cap=cap,
                    alibi=alibi, det=rng.random() < 0.3, packed=packed, lens=rng.randrange(1 << 20))
    if op == "decode":
        n = _log(rng, 1, 32)
        hi = _log(rng, 2, 8192)
        while n * hi * hkv * d > 2.5e8:
            hi = max(1, int(hi * 0.8))
        sq = rng.choice([1, 1, 1, 2, 4, 5])
        new = rng.choice([0, sq])
        page = rng.choice([0, 256, 512])
        cap_keys = hi + sq
        if page:
            cap_keys = -(-cap_keys // page) * page
        rd = rng.choice([0, d, d // 2, 16 * rng.randrange(1, d // 16 + 1)]) if new else 0
        return dict(op=op, n=n, lo=rng.choice([0, 1, hi // 2, hi]), hi=hi, cap_keys=cap_keys, page=page, sq=sq, new=new,
                    hq=hq, hkv=hkv, d=d, causal=sq > 1 or rng.random() < 0.5, wl=rng.choice([-1, -1, _log(rng, 1, 4096)]),
                    cap=cap, alibi=alibi, rd=rd, inter=rng.random() < 0.5, lens=rng.randrange(1 << 20))
    if op == "rotary":
        packed = rng.random() < 0.4
        n, hi, h = _log(rng, 1, 64), _log(rng, 1, 8192), _log(rng, 1, 64)
        while n * hi * h * d > 5e7:
            hi = max(1, int(hi * 0.8))
        return dict(op=op, n=n, lo=rng.choice([0, 1, hi // 2]) if packed else hi, hi=hi, h=h,
                    spare=rng.choice([0, 0, 1, h]), d=d, rd=rng.choice([d, d // 2, 16 * rng.randrange(1, d // 16 + 1)]),
                    inter=rng.random() < 0.5, offset=rng.choice([0, 0, _log(rng, 1, 100000)]), packed=packed,
                    lens=rng.randrange(1 << 20))
    return dict(op="table", rows=_log(rng, 1, 131072), rd=16 * rng.randrange(1, 9),
                scaling=rng.choice(["none", "linear", "base", "by_parts"]))


def _lengths(case):
    """Sequence lengths of a case: part of the case, not of the seed, so that its work is known."""
    n, lo, hi = case["n"], case["lo"], case["hi"]
    if lo == hi:
        return [hi] * n
    r = np.random.RandomState(case["lens"])
    lens = [int(x) for x in r.randint(lo, hi + 1, n)]
    lens[int(r.randint(n))] = hi   # never a batch of empty sequences only
    return lens


def _pairs(lq, lk, causal, wl, wr):
    """Allowed (query, key) pairs of one sequence."""
    i = np.arange(lq, dtype=np.int64) + (lk - lq)
    last = np.full(lq, lk - 1, dtype=np.int64)
    first = np.zeros(lq, dtype=np.int64)
    if causal:
        wr = 0
    if wr >= 0:
        last = np.minimum(last, i + wr)
    if wl >= 0:
        first = np.maximum(first, i - wl)
    return int(np.maximum(last - first + 1, 0).sum())


def work(case):
    op = case["op"]
    if op == "table":
        return dict(bytes=case["rows"] * case["rd"] // 2 * 8, flops=case["rows"] * case["rd"] // 2 * 2)
    lens = _lengths(case)
    if op == "rotary":
        rows = sum(lens) * case["h"]
        # forward and gradient: each reads its input and writes its output; the table rows once
        return dict(bytes=2 * 2 * 2 * rows * case["d"] + max(lens) * case["rd"] // 2 * 8,
                    flops=2 * 3 * rows * case["rd"])
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    if op == "decode":
        lk = [x + case["new"] for x in lens]
        rows = sum(_pairs(case["sq"], x, case["causal"], case["wl"], -1) for x in lk)
        seen = 0   # keys that some query of the sequence sees
        for x in lk:
            first = max(0, x - case["sq"] - case["wl"]) if case["wl"] >= 0 else 0
            seen += max(0, x - first)
        size = seen * hkv * d * 2 * 2 + case["n"] * (case["sq"] * hq * (d * 4 + 4) + case["new"] * hkv * d * 2 * 2)
        return dict(bytes=size, flops=4 * rows * hq * d)
    sq = case["sq"]
    lq = [sq or x for x in lens]
    pairs = sum(_pairs(a, b, case["causal"], case["wl"], case["wr"]) for a, b in zip(lq, lens))
    q_size, k_size = sum(lq) * hq * d * 2, sum(lens) * hkv * d * 2
    if op == "prefill":
        return dict(bytes=2 * q_size + 2 * k_size + sum(lq) * hq * 4, flops=4 * pairs * hq * d)
    # q, out, dout, dq and k, v, dk, dv; 2 products forward, 5 backward
    return dict(bytes=4 * q_size + 4 * k_size + sum(lq) * hq * 4, flops=14 * pairs * hq * d)


# --------------------------------------------------------------------------------------------- inputs
def _normal(g, shape, std=1.0):
    x = torch.empty(shape, dtype=torch.float32, device="cuda").normal_(0.0, std, generator=g)
    return x.to(torch.bfloat16)


def _slopes(heads):
    """Slopes 2^(-8 (h + 1) / heads) of the distance bias, one for each query head."""
    return torch.tensor([2.0 ** (-8.0 * (h + 1) / heads) for h in range(heads)], dtype=torch.float32, device="cuda")


def _cos_sin(rows, rd, base=10000.0):
    """Rotary tables as a user's program holds them, computed in 64 bits."""
    f = base ** (-torch.arange(0, rd, 2, dtype=torch.float64, device="cuda") / rd)
    a = torch.arange(rows, dtype=torch.float64, device="cuda")[:, None] * f[None, :]
    return torch.cos(a).float(), torch.sin(a).float()


def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    r = np.random.RandomState(seed % (1 << 31))
    s = dict(case=case)
    op = case["op"]
    if op == "table":
        s.update(base=float(10.0 ** r.uniform(4.0, 6.0)), factor=float(r.uniform(2.0, 32.0)),
                 amplitude=float(r.uniform(1.0, 1.4)))
        return s
    lens = _lengths(case)
    cu = torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32, device="cuda")
    if op == "rotary":
        heads = case["h"] + case["spare"]
        rows = case["hi"] + case["offset"] + 2 * case["n"]
        s["cos"], s["sin"] = _cos_sin(rows, case["rd"])
        if case["packed"]:
            s["x"] = _normal(g, (sum(lens), heads, case["d"]))[:, :case["h"]]
            s["dy"] = _normal(g, (sum(lens), case["h"], case["d"]))
            s["cu"] = cu
        else:
            s["x"] = _normal(g, (case["n"], case["hi"], heads, case["d"]))[:, :, :case["h"]]
            s["dy"] = _normal(g, (case["n"], case["hi"], case["h"], case["d"]))
            s["cu"] = None
        s["offset"] = 0
        if case["offset"]:   # another first position for each sequence
            s["offset"] = torch.from_numpy(r.randint(0, case["offset"] + 1, case["n"]).astype(np.int32)).cuda()
        return s
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    s["scale"] = 1.0 / math.sqrt(d)
    s["slopes"] = _slopes(hq) if case["alibi"] else None
    if op == "decode":
        n, sq, new, page, cap_keys = case["n"], case["sq"], case["new"], case["page"], case["cap_keys"]
        s["q"] = _normal(g, (n, sq, hq, d), 2.0)
        if page:
            blocks = cap_keys // page
            s["table"] = torch.from_numpy(r.permutation(n * blocks + 2)[:n * blocks].reshape(n, blocks).astype(np.int32)).cuda()
            shape = (n * blocks + 2, page, hkv, d)
        else:
            s["table"] = None
            shape = (n, cap_keys, hkv, d)
        s["k_cache"], s["v_cache"] = _normal(g, shape), _normal(g, shape)
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        s["k"] = _normal(g, (n, new, hkv, d)) if new else None
        s["v"] = _normal(g, (n, new, hkv, d)) if new else None
        s["cos"], s["sin"] = _cos_sin(cap_keys, case["rd"]) if case["rd"] else (None, None)
        return s
    # scores of a few units, as heads that look at something have, so that the cap is felt
    sq = case["sq"]
    if case["packed"]:
        lead = (sum(lens),)
        s.update(cu=cu, hi=max(lens))
        s["q"], s["k"], s["v"] = _normal(g, lead + (hq, d), 2.0), _normal(g, lead + (hkv, d)), _normal(g, lead + (hkv, d))
    else:
        s["q"] = _normal(g, (case["n"], sq or case["hi"], hq, d), 2.0)
        s["k"], s["v"] = _normal(g, (case["n"], case["hi"], hkv, d)), _normal(g, (case["n"], case["hi"], hkv, d))
    if op == "train":
        s["do"] = _normal(g, tuple(s["q"].shape))
    return s


# --------------------------------------------------------------------------------------------- one pass
def run(state):
    case = state["case"]
    op = case["op"]
    if op == "table":
        return _run_table(case, state)
    if op == "rotary":
        return _run_rotary(case, state)
    if op == "decode":
        return _run_decode(case, state)
    return _run_attention(case, state)


def _run_attention(case, s):
    window, cap, train = (case["wl"], case["wr"]), case["cap"], case["op"] == "train"
    if own:
        from exact_tiled_attention_41_b200 import attention as A
        if case["packed"]:
            where = (s["cu"], s["cu"], s["hi"], s["hi"])
            out, lse = A.flash_attn_varlen_func(s["q"], s["k"], s["v"], *where, s["scale"], case["causal"], window,
                                                softcap=cap, alibi_slopes=s["slopes"])
            if not train:
                return out, lse
            grads = A.flash_attn_varlen_backward(s["do"], s["q"], s["k"], s["v"], out, lse, *where, s["scale"],
                                                 case["causal"], window, case["det"], softcap=cap,
                                                 alibi_slopes=s["slopes"])
        else:
            out, lse = A.flash_attn_func(s["q"], s["k"], s["v"], s["scale"], case["causal"], window, softcap=cap,
                                         alibi_slopes=s["slopes"])
            if not train:
                return out, lse
            grads = A.flash_attn_backward(s["do"], s["q"], s["k"], s["v"], out, lse, s["scale"], case["causal"], window,
                                          case["det"], softcap=cap, alibi_slopes=s["slopes"])
        return (out, lse) + tuple(grads)
    q, k, v, do = s["q"], s["k"], s["v"], s.get("do")
    if case["packed"]:   # sequences side by side, padded to the longest
        cu = s["cu"].long()
        lens = cu[1:] - cu[:-1]
        col = torch.arange(s["hi"], device="cuda")
        inside = col[None, :] < lens[:, None]
        at = (cu[:-1, None] + col[None, :]).clamp(max=q.shape[0] - 1)
        q, k, v = q[at], k[at], v[at]
        do = do[at] if train else None
        lq = lk = lens
    else:
        lq = torch.full((q.shape[0],), q.shape[1], device="cuda")
        lk = torch.full((q.shape[0],), k.shape[1], device="cuda")
    got = _plain_attention(q, k, v, do, lq, lk, s["scale"], case["causal"], window, cap, s["slopes"])
    if case["packed"]:
        got = [x[inside] if i != 1 else x.transpose(1, 2)[inside].t().contiguous() for i, x in enumerate(got)]
    return tuple(x.to(torch.bfloat16) if i != 1 else x for i, x in enumerate(got))


def _plain_attention(q, k, v, do, lq, lk, scale, causal, window, cap, slopes):
    """Attention of n sequences in 32 bits, scores and all, and with ``do`` its gradients."""
    n, sq, hq, d = q.shape
    sk, hkv = k.shape[1], k.shape[2]
    q = q.float().transpose(1, 2)
    k = k.float().repeat_interleave(hq // hkv, 2).transpose(1, 2)
    v = v.float().repeat_interleave(hq // hkv, 2).transpose(1, 2)
    x = torch.matmul(q, k.transpose(2, 3)) * scale
    t = None
    if cap > 0:
        t = torch.tanh(x / cap)
        x = t * cap
    i = torch.arange(sq, device="cuda")[None, :, None]
    j = torch.arange(sk, device="cuda")[None, None, :]
    far = i + (lk - lq)[:, None, None] - j        # how far the key lies behind the query
    if slopes is not None:
        x = x - slopes[None, :, None, None] * far.abs()[:, None]
    keep = (i < lq[:, None, None]) & (j < lk[:, None, None])
    if causal:
        keep = keep & (far >= 0)
    if window[0] >= 0:
        keep = keep & (far <= window[0])
    if window[1] >= 0:
        keep = keep & (far >= -window[1])
    x = x.masked_fill(~keep[:, None], -math.inf)
    m = x.amax(3, keepdim=True)
    m = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    x = torch.exp(x - m)
    total = x.sum(3, keepdim=True)
    lse = (m + torch.log(total))[..., 0]
    p = x / torch.where(total > 0, total, torch.ones_like(total))
    out = torch.matmul(p, v).transpose(1, 2)
    if do is None:
        return out, lse
    do = do.float().transpose(1, 2) * (torch.arange(sq, device="cuda")[None, :] < lq[:, None])[:, None, :, None]
    dv = torch.matmul(p.transpose(2, 3), do)
    ds = torch.matmul(do, v.transpose(2, 3))
    ds = p * (ds - (p * ds).sum(3, keepdim=True))
    if cap > 0:
        ds = ds * (1.0 - t * t)
    dq = torch.matmul(ds, k) * scale
    dk = torch.matmul(ds.transpose(2, 3), q) * scale
    # gradients of a key head: the sum over the query heads that read it
    dk, dv = (y.reshape(n, hkv, hq // hkv, sk, d).sum(2).transpose(1, 2) for y in (dk, dv))
    return out, lse, dq.transpose(1, 2), dk, dv


def _turn(x, cos, sin, inter):
    """Rotates the first 2 * cos.shape[-1] values of each head of x (..., heads, d) in 32 bits; cos, sin (..., rd / 2)."""
    half = cos.shape[-1]
    cos, sin = cos.unsqueeze(-2), sin.unsqueeze(-2)
    a, rest = x[..., :2 * half].float(), x[..., 2 * half:].float()
    if inter:
        u, w = a[..., 0::2], a[..., 1::2]
        turned = torch.stack((u * cos - w * sin, u * sin + w * cos), -1).flatten(-2)
    else:
        u, w = a[..., :half], a[..., half:]
        turned = torch.cat((u * cos - w * sin, u * sin + w * cos), -1)
    return torch.cat((turned, rest), -1).to(torch.bfloat16)


def _run_rotary(case, s):
    if own:
        from exact_tiled_attention_41_b200 import attention as A
        y = A.apply_rotary(s["x"], s["cos"], s["sin"], s["offset"], case["inter"], cu_seqlens=s["cu"])
        dx = A.apply_rotary(s["dy"], s["cos"], s["sin"], s["offset"], case["inter"], inverse=True, cu_seqlens=s["cu"])
        return y, dx
    if case["packed"]:
        cu = s["cu"].long()
        tok = torch.arange(s["x"].shape[0], device="cuda")
        seq = torch.searchsorted(cu[1:], tok, right=True)
        pos = tok - cu[seq] + (s["offset"][seq] if torch.is_tensor(s["offset"]) else 0)
    else:
        pos = torch.arange(case["hi"], device="cuda")[None, :].expand(case["n"], -1)
        pos = pos + (s["offset"][:, None] if torch.is_tensor(s["offset"]) else 0)
    cos, sin = s["cos"][pos], s["sin"][pos]
    return _turn(s["x"], cos, sin, case["inter"]), _turn(s["dy"], cos, -sin, case["inter"])


def _run_table(case, s):
    scaling, rows, rd = case["scaling"], case["rows"], case["rd"]
    if own:
        from exact_tiled_attention_41_b200 import attention as A
        return A.rotary_tables(rows, rd, s["base"], scaling=scaling, factor=s["factor"], original_seqlen=4096,
                               low_rotations=1.0, high_rotations=32.0, amplitude=s["amplitude"])
    base, factor = s["base"], s["factor"]
    if scaling == "base":
        base = base * factor ** (rd / (rd - 2.0))
    f = base ** (-torch.arange(0, rd, 2, dtype=torch.float64, device="cuda") / rd)
    if scaling == "linear":
        f = f / factor
    elif scaling == "by_parts":   # turns within the original context decide between f / factor and f
        g = ((4096 * f / (2.0 * math.pi) - 1.0) / (32.0 - 1.0)).clamp(0.0, 1.0)
        f = (1.0 - g) * f / factor + g * f
    a = torch.arange(rows, dtype=torch.float64, device="cuda")[:, None] * f[None, :]
    return (torch.cos(a) * s["amplitude"]).float(), (torch.sin(a) * s["amplitude"]).float()


def _run_decode(case, s):
    window = (case["wl"], -1)
    if own:
        from exact_tiled_attention_41_b200 import attention as A
        out, lse = A.flash_attn_with_kvcache(s["q"], s["k_cache"], s["v_cache"], s["lens"], s["scale"], case["causal"],
                                             k=s["k"], v=s["v"], block_table=s["table"], window_size=window,
                                             softcap=case["cap"], alibi_slopes=s["slopes"], rotary_cos=s["cos"],
                                             rotary_sin=s["sin"], rotary_interleaved=case["inter"])
        return (out, lse, s["k_cache"], s["v_cache"]) if case["new"] else (out, lse)
    q, n, new, page = s["q"], case["n"], case["new"], case["page"]
    lens = s["lens"].long()
    row = torch.arange(n, device="cuda")[:, None]
    if case["rd"]:
        # one query, or queries that do not see different keys, all stand at the sequence's end
        step = torch.arange(case["sq"], device="cuda") * (1 if case["causal"] or case["wl"] >= 0 else 0)
        pos = lens[:, None] + step[None, :]
        q = _turn(q, s["cos"][pos], s["sin"][pos], case["inter"])
    if new:
        pos = lens[:, None] + torch.arange(new, device="cuda")[None, :]
        k = _turn(s["k"], s["cos"][pos], s["sin"][pos], case["inter"]) if case["rd"] else s["k"]
        if page:
            at = (s["table"].long().gather(1, pos // page), pos % page)
        else:
            at = (row.expand(-1, new), pos)
        s["k_cache"][at], s["v_cache"][at] = k, s["v"]
    if page:
        k, v = s["k_cache"][s["table"].long()].flatten(1, 2), s["v_cache"][s["table"].long()].flatten(1, 2)
    else:
        k, v = s["k_cache"], s["v_cache"]
    out, lse = _plain_attention(q, k, v, None, torch.full_like(lens, case["sq"]), lens + new, s["scale"], case["causal"],
                                window, case["cap"], s["slopes"])
    out = out.to(torch.bfloat16)
    return (out, lse, s["k_cache"], s["v_cache"]) if new else (out, lse)


# --------------------------------------------------------------------------------------------- in 64 bits
def exact(case, seed):
    """The definition, one sequence and query head at a time, in 64 bits; gradients by differentiation."""
    s = prepare(case, seed)
    op = case["op"]
    if op == "table":
        rd = case["rd"]
        i = np.arange(rd // 2, dtype=np.longdouble)
        base = np.longdouble(s["base"])
        if case["scaling"] == "base":
            base = base * np.longdouble(s["factor"]) ** (np.longdouble(rd) / (rd - 2))
        f = np.exp(-2 * i / rd * np.log(base))
        if case["scaling"] == "linear":
            f = f / s["factor"]
        if case["scaling"] == "by_parts":
            share = np.minimum(1, np.maximum(0, (f * 4096 / (2 * np.arccos(np.longdouble(-1))) - 1) / 31))
            f = f / s["factor"] * (1 - share) + f * share
        a = np.outer(np.arange(case["rows"], dtype=np.longdouble), f)
        return (np.cos(a) * s["amplitude"]).astype(np.float64), (np.sin(a) * s["amplitude"]).astype(np.float64)
    if op == "rotary":
        return _exact_rotary(case, s)
    if op == "decode":
        return _exact_decode(case, s)
    hq, group, train = case["hq"], case["hq"] // case["hkv"], op == "train"
    lens = _lengths(case)
    out, lse = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda"), []
    dq, dk, dv = out.clone(), *(torch.zeros(s["k"].shape, dtype=torch.float64, device="cuda") for _ in range(2))
    start = 0
    for b in range(case["n"]):
        if case["packed"]:
            at = slice(start, start + lens[b])
            start += lens[b]
            q1, k1, v1 = s["q"][at], s["k"][at], s["v"][at]
        else:
            at = b
            q1, k1, v1 = s["q"][b], s["k"][b], s["v"][b]
        rows = []
        for h in range(hq):
            q, k, v = (x.double().requires_grad_(train) for x in (q1[:, h], k1[:, h // group], v1[:, h // group]))
            o, l = _exact_head(q, k, v, s["scale"], case, s["slopes"], h)
            rows.append(l.detach())
            out[at][:, h] = o.detach()
            if train and q.numel() and k.numel():
                grads = torch.autograd.grad(o, (q, k, v), s["do"][at][:, h].double())
                dq[at][:, h] = grads[0]
                dk[at][:, h // group] += grads[1]
                dv[at][:, h // group] += grads[2]
        lse.append(torch.stack(rows))
    lse = torch.cat(lse, 1) if case["packed"] else torch.stack(lse)
    return (out, lse, dq, dk, dv) if train else (out, lse)


def _exact_head(q, k, v, scale, case, slopes, h):
    """softmax of one head's scores over the keys its mask leaves; rows without keys give 0 and -inf."""
    lq, lk = q.shape[0], k.shape[0]
    x = scale * (q @ k.T)
    if case["cap"] > 0:
        e = torch.exp(-2.0 / case["cap"] * x)
        x = case["cap"] * (2.0 / (1.0 + e) - 1.0)
    place = torch.arange(lq, device="cuda")[:, None] + (lk - lq)
    key = torch.arange(lk, device="cuda")[None, :]
    if slopes is not None:
        x = x - float(slopes[h]) * (place - key).abs().double()
    right = 0 if case["causal"] else case.get("wr", -1)
    hide = torch.zeros(lq, lk, dtype=torch.bool, device="cuda")
    if right >= 0:
        hide |= key > place + right
    if case["wl"] >= 0:
        hide |= key < place - case["wl"]
    if lk == 0:
        return torch.zeros(lq, v.shape[1], dtype=torch.float64, device="cuda") + 0 * q, torch.full((lq,), -math.inf, dtype=torch.float64, device="cuda")
    empty = hide.all(1)
    x = x.masked_fill(hide & ~empty[:, None], -math.inf)
    lse = torch.logsumexp(x, 1)
    o = torch.exp(x - lse[:, None]) @ v
    return torch.where(empty[:, None], torch.zeros_like(o), o), lse.masked_fill(empty, -math.inf)


def _exact_turn(x, cos, sin, inter):
    """Rotation as a product of complex numbers; cos, sin (rows, rd / 2) for x (rows, heads, d)."""
    half = cos.shape[1]
    z = torch.complex(cos.double(), sin.double())[:, None]
    y = x.double()
    first, second = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if inter else (slice(0, half), slice(half, 2 * half))
    w = torch.complex(y[..., first], y[..., second]) * z
    y[..., first], y[..., second] = w.real, w.imag
    return y


def _exact_rotary(case, s):
    lens = _lengths(case)
    first = s["offset"].tolist() if torch.is_tensor(s["offset"]) else [0] * case["n"]
    at = torch.cat([torch.arange(f, f + x, device="cuda") for f, x in zip(first, lens)])
    got = [_exact_turn(x.reshape(-1, case["h"], case["d"]), s["cos"][at], sign * s["sin"][at], case["inter"]).reshape(x.shape)
           for x, sign in ((s["x"], 1), (s["dy"], -1))]
    return tuple(got)


def _exact_decode(case, s):
    n, sq, new, page, group = case["n"], case["sq"], case["new"], case["page"], case["hq"] // case["hkv"]
    lens = _lengths(case)
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros((n, case["hq"], sq), dtype=torch.float64, device="cuda")
    for b in range(n):
        q, have = s["q"][b].double(), lens[b]
        if case["rd"]:
            # the queries keep their type after the turn, and so do the keys in the cache
            at = torch.arange(sq, device="cuda") * int(case["causal"] or case["wl"] >= 0) + have
            q = _exact_turn(s["q"][b], s["cos"][at], s["sin"][at], case["inter"]).to(torch.bfloat16).double()
        for i in range(new):
            k1 = s["k"][b, i:i + 1]
            if case["rd"]:
                at = torch.tensor([have + i], device="cuda")
                k1 = _exact_turn(k1, s["cos"][at], s["sin"][at], case["inter"]).to(torch.bfloat16)
            where = (int(s["table"][b, (have + i) // page]), (have + i) % page) if page else (b, have + i)
            s["k_cache"][where], s["v_cache"][where] = k1[0], s["v"][b, i]
        if page:
            k, v = (c[s["table"][b].long()].reshape(-1, case["hkv"], case["d"]) for c in (s["k_cache"], s["v_cache"]))
        else:
            k, v = s["k_cache"][b], s["v_cache"][b]
        for h in range(case["hq"]):
            k1, v1 = (x[:have + new, h // group].double() for x in (k, v))
            out[b, :, h], lse[b, h] = _exact_head(q[:, h], k1, v1, s["scale"], case, s["slopes"], h)
    return (out, lse, s["k_cache"], s["v_cache"]) if new else (out, lse)
