"""fp64 reference of capped and biased attention, rotary positions and their tables.

TEST INFRASTRUCTURE ONLY -- see the package docstring.  Materialises scores and
probabilities for one (sequence, query head) at a time, like attention.py.

Sources and readings:

* flash-attention README, ``flash_attn_func`` docstring: alibi_slopes -- a bias of
  -alibi_slope * |i + seqlen_k - seqlen_q - j| is added to the score of query i and
  key j; slopes are (nheads,) or (batch, nheads), float32.
* README, changelog 2.6: softcapping is named without a formula.  Reading:
  score = softcap * tanh(scale * q.k / softcap), before the bias and the mask.
* README, ``flash_attn_with_kvcache`` docstring: rotary_cos / rotary_sin
  (seqlen_ro, rotary_dim / 2); rotary_interleaved pairs dimensions 0 and 1, 2 and
  3, ..., otherwise dimension i and i + rotary_dim / 2; new keys are rotated at
  cache_seqlens, cache_seqlens + 1, ...; the queries at the same indices under a
  causal mask or a window, else all at cache_seqlens.

``head`` also returns elementwise bounds on the errors that rounding may cause in a
kernel with bf16 operands and fp32 sums; they count roundings and nothing else
(a rounding to bf16 is off by at most 2^-8 of the value, half a step).
"""

from __future__ import annotations

import numpy as np

from .attention import allowed_mask

BF16 = 2.0 ** -8


def scores(q, k, scale, softcap=0.0, slope=None):
    """(x, t): modified scores of one head and, with a cap, the tanh (else None)."""
    x = scale * (q @ k.T)
    t = None
    if softcap > 0:
        t = np.tanh(x / softcap)
        x = softcap * t
    if slope is not None:
        i = np.arange(q.shape[0])[:, None]
        j = np.arange(k.shape[0])[None, :]
        x = x - slope * np.abs(i + k.shape[0] - q.shape[0] - j)
    return x, t


def head(q, k, v, scale, mask, softcap=0.0, slope=None, do=None, q_err=0.0):
    """One query head against one KV head.  Returns a dict with o, lse and, given do, dq, dk, dv, and for each name
    a bound ``<name>_tol``.  q_err: relative error that q may already have (rotated and rounded elsewhere)."""
    q, k, v = (np.asarray(a, np.float64) for a in (q, k, v))
    x, t = scores(q, k, scale, softcap, slope)
    x = np.where(mask, x, -np.inf)
    m = x.max(axis=1, initial=-np.inf, keepdims=True)
    empty = np.isneginf(m)
    e = np.exp(x - np.where(empty, 0.0, m))
    l = e.sum(axis=1, keepdims=True)
    p = e / np.where(empty, 1.0, l)
    with np.errstate(divide="ignore"):
        lse = np.where(empty, 0.0, m)[:, 0] + np.log(l[:, 0])
    o = p @ v
    # scores: D products summed in fp32 (each step off by 2^-23 of the running sum at most), the bias and its sum by
    # 3 fp32 roundings; then one exponential, 2^-21 relative.  The tanh: its polynomials (arguments up to 1) are within
    # 5e-7 of the value, and the multi-function unit's form, within 2e-7 of 1, is at most 2e-7 / tanh(1) = 2.7e-7 of it
    # beyond: 6e-7 of the capped score with the rounding of the product.  Up to a cap of 55 the unit may serve smaller
    # arguments too, off by 2e-7 of the cap (the bound takes twice that, as everywhere below it)
    size = scale * (np.abs(q) @ np.abs(k).T)
    x_err = size * (q.shape[1] * 2.0 ** -23 + 2.0 ** -22 + q_err)
    if softcap > 0:
        x_err = x_err + 4e-7 * np.minimum(softcap, np.maximum(1.5 * softcap * np.abs(t), 55.0))
    if slope is not None:
        i, j = np.arange(q.shape[0])[:, None], np.arange(k.shape[0])[None, :]
        x_err = x_err + 2.0 ** -22 * abs(slope) * np.abs(i + k.shape[0] - q.shape[0] - j)
    x_err = np.where(mask, x_err, 0.0)
    worst = x_err.max(axis=1, initial=0.0)
    lse_tol = worst + 2.0 ** -20 * (1.0 + np.abs(np.where(empty[:, 0], 0.0, lse)))
    p_rel = BF16 + 2 * worst[:, None] + 2.0 ** -18   # bf16 P, and its exponent's error against the maximum and sum
    o_tol = p_rel * (p @ np.abs(v)) + BF16 * np.abs(o) + 1e-30
    out = dict(o=o, lse=lse, o_tol=o_tol, lse_tol=lse_tol)
    if do is None:
        return out
    do = np.asarray(do, np.float64)
    dp = do @ v.T
    delta = (p * dp).sum(axis=1, keepdims=True)
    g = np.ones_like(p) if t is None else 1.0 - t * t
    ds = p * (dp - delta) * g
    # dS: P before rounding (p_rel without bf16), dP an fp32 sum of D products, Delta from the stored (rounded) O,
    # 1 - tanh^2 off by 8e-7, then one rounding to bf16
    p_pre = p_rel - BF16
    dp_err = (v.shape[1] * 2.0 ** -23) * (np.abs(do) @ np.abs(v).T)
    delta_err = (np.abs(do) * o_tol).sum(axis=1, keepdims=True) + 2.0 ** -20 * (np.abs(do) * np.abs(o)).sum(axis=1, keepdims=True)
    ds_err = (BF16 + p_pre) * np.abs(ds) + p * g * (dp_err + delta_err) + 8e-7 * p * np.abs(dp - delta)
    tiny = 1e-30
    out["dv"] = p.T @ do
    out["dv_tol"] = (p_rel * p).T @ np.abs(do) + BF16 * np.abs(out["dv"]) + tiny
    out["dq"] = scale * (ds @ k)
    out["dq_tol"] = scale * (ds_err @ np.abs(k)) * 1.01 + BF16 * np.abs(out["dq"]) + tiny
    out["dk"] = scale * (ds.T @ q)
    out["dk_tol"] = scale * (ds_err.T @ np.abs(q)) * 1.01 + BF16 * np.abs(out["dk"]) + tiny
    return out


def attention(q, k, v, scale, causal=False, window=(-1, -1), softcap=0.0, slopes=None, do=None):
    """A batch (B, S, H, D), or lists of B sequences (S_b, H, D); slopes (Hq,) or (B, Hq) or None.  Returns a list of
    dicts per sequence with o (Lq, Hq, D), lse (Hq, Lq), dq, dk, dv and their tolerances; dk and dv are summed over
    the query heads of a KV head."""
    res = []
    for b in range(len(q)):
        Lq, Hq, D = q[b].shape
        Lk, Hkv = k[b].shape[:2]
        group = Hq // Hkv
        mask = allowed_mask(Lq, Lk, causal, window)
        r = dict(o=np.zeros((Lq, Hq, D)), o_tol=np.zeros((Lq, Hq, D)), lse=np.zeros((Hq, Lq)), lse_tol=np.zeros((Hq, Lq)))
        if do is not None:
            for n, like in (("dq", q[b]), ("dk", k[b]), ("dv", v[b])):
                r[n], r[n + "_tol"] = np.zeros(like.shape), np.zeros(like.shape)
        for h in range(Hq):
            s = None if slopes is None else float(slopes[h] if np.ndim(slopes) == 1 else slopes[b][h])
            one = head(q[b][:, h], k[b][:, h // group], v[b][:, h // group], scale, mask, softcap, s,
                       None if do is None else do[b][:, h])
            for n in ("o", "dq"):
                for suffix in ("", "_tol"):
                    if n + suffix in one:
                        r[n + suffix][:, h] = one[n + suffix]
            r["lse"][h], r["lse_tol"][h] = one["lse"], one["lse_tol"]
            if do is not None:
                for n in ("dk", "dv"):
                    for suffix in ("", "_tol"):
                        r[n + suffix][:, h // group] += one[n + suffix]
        res.append(r)
    return res


def rotary_tables(rows, rotary_dim, base=10000.0, scaling="none", factor=1.0, original=0, low=1.0, high=32.0,
                  amplitude=1.0):
    """Cosines and sines (rows, rotary_dim / 2) from the definition, in long double."""
    i = np.arange(rotary_dim // 2, dtype=np.longdouble)
    base = np.longdouble(base)
    if scaling == "base":
        base = base * np.longdouble(factor) ** (np.longdouble(rotary_dim) / np.longdouble(rotary_dim - 2))
    f = base ** (-2 * i / rotary_dim)
    if scaling == "linear":
        f = f / np.longdouble(factor)
    elif scaling == "by_parts":
        r = original * f / (2 * np.longdouble("3.14159265358979323846264338327950288"))
        g = np.clip((r - low) / (high - low), 0, 1)
        f = (1 - g) * f / np.longdouble(factor) + g * f
    a = np.arange(rows, dtype=np.longdouble)[:, None] * f[None, :]
    return (amplitude * np.cos(a)).astype(np.float64), (amplitude * np.sin(a)).astype(np.float64)


def rotate(x, cos, sin, positions, interleaved, inverse=False):
    """x (tokens, H, D) rotated by row positions[t] of cos, sin (rows, rotary_dim / 2)."""
    x = np.asarray(x, np.float64)
    half = cos.shape[1]
    c, s = cos[positions][:, None], sin[positions][:, None] * (-1 if inverse else 1)
    y = x.copy()
    a, b = (x[..., :2 * half:2], x[..., 1:2 * half:2]) if interleaved else (x[..., :half], x[..., half:2 * half])
    ya, yb = a * c - b * s, b * c + a * s
    if interleaved:
        y[..., :2 * half:2], y[..., 1:2 * half:2] = ya, yb
    else:
        y[..., :half], y[..., half:2 * half] = ya, yb
    return y


def rotate_tol(x, y, cos, sin, positions, interleaved):
    """Bound on the rounding error of ``rotate``: two fp32 roundings of the products, one to bf16."""
    size = rotate(np.abs(x), np.abs(cos), -np.abs(sin), positions, interleaved)
    size = np.maximum(np.abs(size), rotate(np.abs(x), np.abs(cos), np.abs(sin), positions, interleaved, False))
    return BF16 * np.abs(y) * 1.001 + 2.0 ** -22 * np.abs(size) + 1e-38
