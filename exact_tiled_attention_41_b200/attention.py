"""Torch-tensor entry points over the C ABI: allocation of outputs and workspace
(PyTorch's caching allocator) and argument marshalling; every step of the
computation runs in libfa.so's CUDA kernels.  Inputs must be contiguous bf16
CUDA tensors; anything else raises -- there is no CPU path.

Shapes follow the flash-attention README (flash_attn_func, flash_attn_varlen_func,
flash_attn_with_kvcache docstrings): q (B, Sq, Hq, D), k/v (B, Sk, Hkv, D); varlen
q (total_q, Hq, D) with int32 cu_seqlens; caches (B, capacity, Hkv, D).
softmax_scale defaults to 1/sqrt(D) (README, "How to use FlashAttention").
window_size = (left, right) is the sliding window of the flash_attn_func docstring
(-1 = unbounded side); deterministic selects the backward whose dq does not depend
on the order of float additions.

Scores may be capped by a tanh (softcap) and biased by the distance of query and key
(alibi_slopes, float32 (Hq,) or (B, Hq); data, without a gradient):
    x_ij = softcap tanh(scale q_i.k_j / softcap) - slope_h |i + Sk - Sq - j|.
Rotary positions: rotary_tables builds the cosines and sines, apply_rotary (RotaryFunction for
autograd) rotates queries and keys, and flash_attn_with_kvcache rotates the new ones itself.
Calls run on the device of their first tensor, on its current stream.
"""

from __future__ import annotations

import functools
import math

import torch
from torch.autograd.function import once_differentiable

from . import abi


def _check(t: torch.Tensor, name: str, dtype=torch.bfloat16):
    if t.__class__ is torch.Tensor and t.is_cuda and t.dtype is dtype and t.is_contiguous():
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (no CPU path)")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _raise(status: int, where: str):
    if status != abi.FA_OK:
        raise abi.FAError(status, where)


def _workspace(nbytes: int, device) -> torch.Tensor | None:
    if nbytes == 0:
        return None
    # torch's allocator returns >= 512-byte aligned blocks
    return torch.empty(nbytes, dtype=torch.uint8, device=device)


def _on_device(fn):
    """Runs fn with the device of its first tensor current (its stream and context are the ones used)."""
    @functools.wraps(fn)
    def run(*args, **kwargs):
        t = args[0] if args else None
        if not isinstance(t, torch.Tensor):   # keywords in any order, a scale first perhaps
            t = next((a for a in (*args, *kwargs.values()) if isinstance(a, torch.Tensor)), None)
        if t is not None and t.is_cuda and t.get_device() != torch._C._cuda_getDevice():
            with torch.cuda.device(t.device):
                return fn(*args, **kwargs)
        return fn(*args, **kwargs)
    return run


def _score(softcap, alibi_slopes, q, B, Hq):
    """(softcap, slopes, batch stride) as the C calls take them."""
    if alibi_slopes is None:
        return softcap, None, 0
    _check(alibi_slopes, "alibi_slopes", torch.float32)
    if alibi_slopes.device != q.device:
        raise ValueError("alibi_slopes must be on the device of q")
    if alibi_slopes.shape == (Hq,):
        return softcap, alibi_slopes, 0
    if alibi_slopes.shape == (B, Hq):
        return softcap, alibi_slopes, Hq
    raise ValueError(f"alibi_slopes must be ({Hq},) or ({B}, {Hq}), got {tuple(alibi_slopes.shape)}")


def _window(window_size):
    left, right = window_size
    return int(left), int(right)


@_on_device
def flash_attn_func(q, k, v, softmax_scale=None, causal=False, window_size=(-1, -1), softcap=0.0, alibi_slopes=None):
    """Forward: returns (out (B, Sq, Hq, D) bf16, lse (B, Hq, Sq) fp32)."""
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _check(t, n)
    B, Sq, Hq, D = q.shape
    Sk, Hkv = k.shape[1], k.shape[2]
    scale = 1.0 / math.sqrt(D) if softmax_scale is None else softmax_scale
    out = torch.empty_like(q)
    lse = torch.empty((B, Hq, Sq), dtype=torch.float32, device=q.device)
    nb = abi.fa_fwd_workspace_size(B, Hq, Hkv, Sq, Sk, D)
    ws = _workspace(nb, q.device)
    _raise(abi.fa_fwd_mod(q, k, v, out, lse, B, Hq, Hkv, Sq, Sk, D, scale, causal, *_window(window_size),
                          *_score(softcap, alibi_slopes, q, B, Hq), ws, nb), "fa_fwd")
    return out, lse


@_on_device
def flash_attn_backward(dout, q, k, v, out, lse, softmax_scale=None, causal=False, window_size=(-1, -1),
                        deterministic=False, softcap=0.0, alibi_slopes=None):
    """Backward: returns (dq, dk, dv) shaped like q, k, v; out and lse from the forward with the same arguments."""
    for t, n in ((dout, "dout"), (q, "q"), (k, "k"), (v, "v"), (out, "out")):
        _check(t, n)
    _check(lse, "lse", torch.float32)
    B, Sq, Hq, D = q.shape
    Sk, Hkv = k.shape[1], k.shape[2]
    scale = 1.0 / math.sqrt(D) if softmax_scale is None else softmax_scale
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    nb = abi.fa_bwd_workspace_size(B, Hq, Hkv, Sq, Sk, D)
    ws = _workspace(nb, q.device)
    _raise(abi.fa_bwd_mod(q, k, v, out, dout, lse, dq, dk, dv, B, Hq, Hkv, Sq, Sk, D, scale, causal,
                          *_window(window_size), deterministic, *_score(softcap, alibi_slopes, q, B, Hq), ws, nb),
           "fa_bwd")
    return dq, dk, dv


@_on_device
def flash_attn_varlen_func(q, k, v, cu_seqlens_q, cu_seqlens_k, max_seqlen_q, max_seqlen_k, softmax_scale=None,
                           causal=False, window_size=(-1, -1), softcap=0.0, alibi_slopes=None):
    """Packed forward: returns (out (total_q, Hq, D), lse (Hq, total_q))."""
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _check(t, n)
    _check(cu_seqlens_q, "cu_seqlens_q", torch.int32)
    _check(cu_seqlens_k, "cu_seqlens_k", torch.int32)
    total_q, Hq, D = q.shape
    total_k, Hkv = k.shape[0], k.shape[1]
    nseq = cu_seqlens_q.numel() - 1
    scale = 1.0 / math.sqrt(D) if softmax_scale is None else softmax_scale
    out = torch.empty_like(q)
    lse = torch.empty((Hq, total_q), dtype=torch.float32, device=q.device)
    nb = abi.fa_varlen_fwd_workspace_size(nseq, total_q, total_k, Hq, Hkv, D)
    ws = _workspace(nb, q.device)
    _raise(abi.fa_varlen_fwd_mod(q, k, v, out, lse, cu_seqlens_q, cu_seqlens_k, nseq, max_seqlen_q, max_seqlen_k,
                                 total_q, total_k, Hq, Hkv, D, scale, causal, *_window(window_size),
                                 *_score(softcap, alibi_slopes, q, nseq, Hq), ws, nb), "fa_varlen_fwd")
    return out, lse


@_on_device
def flash_attn_varlen_backward(dout, q, k, v, out, lse, cu_seqlens_q, cu_seqlens_k, max_seqlen_q, max_seqlen_k,
                               softmax_scale=None, causal=False, window_size=(-1, -1), deterministic=False,
                               softcap=0.0, alibi_slopes=None):
    for t, n in ((dout, "dout"), (q, "q"), (k, "k"), (v, "v"), (out, "out")):
        _check(t, n)
    _check(lse, "lse", torch.float32)
    total_q, Hq, D = q.shape
    total_k, Hkv = k.shape[0], k.shape[1]
    nseq = cu_seqlens_q.numel() - 1
    scale = 1.0 / math.sqrt(D) if softmax_scale is None else softmax_scale
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    nb = abi.fa_varlen_bwd_workspace_size(nseq, total_q, total_k, Hq, Hkv, D)
    ws = _workspace(nb, q.device)
    _raise(abi.fa_varlen_bwd_mod(q, k, v, out, dout, lse, dq, dk, dv, cu_seqlens_q, cu_seqlens_k, nseq, max_seqlen_q,
                                 max_seqlen_k, total_q, total_k, Hq, Hkv, D, scale, causal, *_window(window_size),
                                 deterministic, *_score(softcap, alibi_slopes, q, nseq, Hq), ws, nb), "fa_varlen_bwd")
    return dq, dk, dv


@_on_device
def flash_attn_with_kvcache(q, k_cache, v_cache, cache_seqlens, softmax_scale=None, causal=False, num_splits=0,
                            return_lse=True, k=None, v=None, cache_batch_idx=None, block_table=None,
                            window_size=(-1, -1), softcap=0.0, alibi_slopes=None, rotary_cos=None, rotary_sin=None,
                            rotary_interleaved=True):
    """Attention of new queries against a KV cache (README, flash_attn_with_kvcache docstring).

    q (B, Sq, Hq, D); caches (B_cache, capacity, Hkv, D), or pages (num_blocks, page_block_size, Hkv, D)
    with block_table (B, max_blocks_per_seq) int32; cache_seqlens int32 (B,) or an int.  If k / v
    (B, seqlen_new, Hkv, D) are given they are written into the caches in place at cache_seqlens first.
    With rotary_cos / rotary_sin (seqlen_ro, rotary_dim / 2) float32 (and k, v) the new keys are rotated at
    cache_seqlens, cache_seqlens + 1, ... on their way into the cache, and the queries at the same positions
    under a causal mask or window, else all at cache_seqlens; the pairs are adjacent values
    (rotary_interleaved) or values rotary_dim / 2 apart.  Positions past the tables are refused for an int
    cache_seqlens, and otherwise become zeros with an error in the device status (abi.fa_get_device_status).
    Returns (out (B, Sq, Hq, D), lse (B, Hq, Sq) or None).
    """
    for t, n in ((q, "q"), (k_cache, "k_cache"), (v_cache, "v_cache")):
        _check(t, n)
    B, Sq, Hq, D = q.shape
    cached = cache_seqlens if isinstance(cache_seqlens, int) else None
    if cached is not None:
        cache_seqlens = torch.full((B,), cache_seqlens, dtype=torch.int32, device=q.device)
    _check(cache_seqlens, "cache_seqlens", torch.int32)
    if (k is None) != (v is None):
        raise ValueError("k and v must be given together")
    sn = 0
    if k is not None:
        _check(k, "k")
        _check(v, "v")
        sn = k.shape[1]
        if k.shape != v.shape or k.shape != (B, sn, k_cache.shape[2], D):
            raise ValueError(f"k and v must be (B, seqlen_new, Hkv, D), got {tuple(k.shape)} and {tuple(v.shape)}")
    if cache_batch_idx is not None:
        _check(cache_batch_idx, "cache_batch_idx", torch.int32)
    max_blocks = 0
    if block_table is not None:
        _check(block_table, "block_table", torch.int32)
        max_blocks = block_table.shape[1]
    cache_batch, cap, Hkv = k_cache.shape[0], k_cache.shape[1], k_cache.shape[2]
    scale = 1.0 / math.sqrt(D) if softmax_scale is None else softmax_scale
    out = torch.empty_like(q)
    lse = torch.empty((B, Hq, Sq), dtype=torch.float32, device=q.device) if return_lse else None
    rows, rd = _rotary_tables_shape(rotary_cos, rotary_sin, q, D)
    nb = abi.fa_fwd_kvcache_mod_workspace_size(B, Hq, Hkv, Sq, D, cap, max_blocks, num_splits, rd)
    ws = _workspace(nb, q.device)
    left, right = _window(window_size)
    if rd and cached is not None:
        # the queries' last position, and that of the new keys which the cache has room for
        room = cap * max(max_blocks, 1)
        cached = min(max(cached, 0), room)
        in_order = causal or 0 <= left < 1 << 30 or 0 <= right < 1 << 30
        _check_positions(cached, max(cached + (Sq - 1 if in_order else 0), min(cached + sn, room) - 1), rows)
    _raise(abi.fa_fwd_kvcache_mod(q, k_cache, v_cache, cache_seqlens, k, v, sn, cache_batch_idx, block_table,
                                  max_blocks, cache_batch, cap, out, lse, B, Hq, Hkv, Sq, D, scale, causal, left,
                                  right, num_splits, *_score(softcap, alibi_slopes, q, B, Hq), rotary_cos, rotary_sin,
                                  rows, rd, rotary_interleaved, ws, nb), "fa_fwd_kvcache")
    return out, lse


def _rotary_tables_shape(cos, sin, x, D):
    """(rows, rotary_dim) of a pair of tables, (0, 0) without tables."""
    if cos is None and sin is None:
        return 0, 0
    if cos is None or sin is None:
        raise ValueError("rotary_cos and rotary_sin must be given together")
    _check(cos, "rotary_cos", torch.float32)
    _check(sin, "rotary_sin", torch.float32)
    if cos.dim() != 2 or cos.shape != sin.shape or cos.device != x.device or sin.device != x.device:
        raise ValueError("rotary_cos and rotary_sin must be (seqlen_ro, rotary_dim / 2) on the device of the input")
    rows, half = cos.shape
    if half == 0 or 2 * half > D or half % 8 != 0:
        raise ValueError(f"rotary_dim must be a multiple of 16, at most {D}; got {2 * half}")
    return rows, 2 * half


def _check_positions(first, last, rows):
    """Refuses positions that the host knows: first (of 32 bits) and, where it is known, last (inside the tables)."""
    if not -1 << 31 <= first < 1 << 31 or (last is not None and last >= rows):
        raise ValueError(f"position {first if last is None else last} lies past the tables of {rows} rows")


_SCALINGS = {"none": abi.FA_ROTARY_PLAIN, "linear": abi.FA_ROTARY_LINEAR, "base": abi.FA_ROTARY_BASE,
             "by_parts": abi.FA_ROTARY_BY_PARTS}


def rotary_tables(seqlen, rotary_dim, base=10000.0, scaling="none", factor=1.0, original_seqlen=0, low_rotations=1.0,
                  high_rotations=32.0, amplitude=1.0, device=None):
    """Cosines and sines (seqlen, rotary_dim / 2) float32 of positions 0 .. seqlen - 1:
    amplitude * cos / sin(p * f_i), f_i = base^(-2i / rotary_dim), with f_i scaled for long contexts:

    "linear": f_i / factor; "base": f_i of base * factor^(rotary_dim / (rotary_dim - 2));
    "by_parts": pairs that turn less than low_rotations times within original_seqlen tokens are slowed by factor,
    those that turn more than high_rotations times are left, the others lie between (linearly in the rotations).
    """
    if scaling not in _SCALINGS:
        raise ValueError(f"scaling must be one of {sorted(_SCALINGS)}, got {scaling!r}")
    device = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    if device.type != "cuda":
        raise ValueError("device must be a CUDA device (no CPU path)")
    with torch.cuda.device(device):
        # both tables in one allocation; each starts on a 16-byte boundary (rotary_dim / 2 is a multiple of 8)
        cos, sin = torch.empty((2, max(seqlen, 0), max(rotary_dim, 0) // 2), dtype=torch.float32, device=device).unbind(0)
        _raise(abi.fa_rotary_tables(cos, sin, seqlen, rotary_dim, base, _SCALINGS[scaling], factor, original_seqlen,
                                    low_rotations, high_rotations, amplitude), "fa_rotary_tables")
    return cos, sin


def _rotary_strides(t, name):
    """(sequence, token, head) strides in elements; 0 where a dimension has one entry."""
    *strides, last = t.stride()
    if last != 1:
        raise ValueError(f"{name} must have its head dimension contiguous")
    s = [st if n > 1 else 0 for st, n in zip(strides, t.shape)]
    return s if len(s) == 3 else [0] + s


@_on_device
def apply_rotary(x, cos, sin, seqlen_offsets=0, interleaved=True, inverse=False, cu_seqlens=None, out=None):
    """Rotates the first 2 * cos.shape[1] values of each head of x by the angles of its token's position.

    x (B, S, H, D), or (total, H, D) with cu_seqlens int32 (B + 1,): bf16 with the head dimension contiguous and
    the other strides multiples of 8 (a slice of a packed projection will do).  cos, sin (seqlen_ro, rotary_dim / 2)
    float32.  A token's position is its index in its sequence plus seqlen_offsets (an int, or int32 (B,)).  Positions past
    the tables are refused where they are known here (equal lengths and an int); else the call rotates to zeros there and
    leaves an error in the device status (abi.fa_get_device_status).
    Pairs are adjacent values (interleaved) or values rotary_dim / 2 apart.  inverse rotates by the opposite angle,
    which is the gradient (RotaryFunction records it for autograd; this call does not).  out may be x (in place);
    other overlaps are not supported.  A given out is refused while gradients are recorded and it or x requires one,
    and its version counter moves on, so that autograd notices where it had saved it.  Returns out, contiguous unless
    given.  Rows behind the last sequence of a packed batch are zeros in a new out and are not written in a given one.
    """
    if not isinstance(x, torch.Tensor):
        raise TypeError("x must be a torch.Tensor")
    if not x.is_cuda:
        raise ValueError("x must be a CUDA tensor (no CPU path)")
    if x.dtype != torch.bfloat16:
        raise TypeError(f"x must be {torch.bfloat16}, got {x.dtype}")
    if x.dim() != (4 if cu_seqlens is None else 3):
        raise ValueError("x must be (B, S, H, D), or (total, H, D) with cu_seqlens")
    H, D = x.shape[-2:]
    rows, rd = _rotary_tables_shape(cos, sin, x, D)
    if rd == 0:
        raise ValueError("cos and sin must be given")
    if cu_seqlens is None:
        B, S, total = x.shape[0], x.shape[1], 0
    else:
        _check(cu_seqlens, "cu_seqlens", torch.int32)
        B, S, total = cu_seqlens.numel() - 1, 0, x.shape[0]
    offsets = None
    if isinstance(seqlen_offsets, torch.Tensor):
        offsets, seqlen_offsets = seqlen_offsets, 0
        _check(offsets, "seqlen_offsets", torch.int32)
        if offsets.shape != (B,):
            raise ValueError(f"seqlen_offsets must be an int or ({B},)")
    for t, n in ((offsets, "seqlen_offsets"), (cu_seqlens, "cu_seqlens"), (out, "out")):
        if t is not None and t.device != x.device:
            raise ValueError(f"{n} must be on the device of x")
    new = out is None
    if new:
        out = torch.empty_like(x, memory_format=torch.contiguous_format)
    elif out.shape != x.shape or out.dtype != x.dtype:
        raise ValueError("out must have the shape and type of x")
    elif torch.is_grad_enabled() and (x.requires_grad or out.requires_grad):
        raise ValueError("x and a given out must not require grad: the rotation is not recorded (RotaryFunction records it)")
    if x.numel() == 0:
        return out
    if offsets is None:
        _check_positions(seqlen_offsets, seqlen_offsets + S - 1 if cu_seqlens is None else None, rows)
    _raise(abi.fa_rotary(x, out, cos, sin, cu_seqlens, offsets, seqlen_offsets, B, S, total, H, D, rd, rows,
                         *_rotary_strides(x, "x"), *_rotary_strides(out, "out"), interleaved, inverse, new), "fa_rotary")
    if not new and not out.is_inference():
        torch.autograd.graph.increment_version(out)
    return out


@_on_device
def merge_attention_parts(o_parts, lse_parts, out_dtype=torch.bfloat16, out=None):
    """Merge results over disjoint key sets: o_parts (C, B, S, H, D) bf16 or fp32 and lse_parts (C, B, H, S)
    fp32, as fa_fwd writes them per key set.  Returns (out (B, S, H, D), lse (B, H, S))."""
    if o_parts.dtype not in (torch.bfloat16, torch.float32):
        raise TypeError("o_parts must be bfloat16 or float32")
    _check(o_parts, "o_parts", o_parts.dtype)
    _check(lse_parts, "lse_parts", torch.float32)
    C, B, S, H, D = o_parts.shape
    if tuple(lse_parts.shape) != (C, B, H, S):
        raise ValueError("lse_parts must be (C, B, H, S)")
    if out is None:
        out = torch.empty((B, S, H, D), dtype=out_dtype, device=o_parts.device)
    _check(out, "out", out.dtype)
    lse = torch.empty((B, H, S), dtype=torch.float32, device=o_parts.device)
    _raise(abi.fa_merge_lse(o_parts, lse_parts, C, B, S, H, D, o_parts.dtype == torch.float32, out, lse,
                            out.dtype == torch.float32), "fa_merge_lse")
    return out, lse


class FlashAttnFunction(torch.autograd.Function):
    """Autograd wrapper: forward = fa_fwd_mod, backward = fa_bwd_mod."""

    @staticmethod
    def forward(ctx, q, k, v, softmax_scale=None, causal=False, window_size=(-1, -1), deterministic=False, softcap=0.0,
                alibi_slopes=None):
        if alibi_slopes is not None and alibi_slopes.requires_grad:
            raise ValueError("alibi_slopes have no gradient")
        out, lse = flash_attn_func(q, k, v, softmax_scale, causal, window_size, softcap, alibi_slopes)
        ctx.save_for_backward(q, k, v, out, lse, alibi_slopes)
        ctx.softmax_scale, ctx.causal = softmax_scale, causal
        ctx.window_size, ctx.deterministic, ctx.softcap = window_size, deterministic, softcap
        return out

    @staticmethod
    def backward(ctx, dout):
        q, k, v, out, lse, alibi_slopes = ctx.saved_tensors
        dq, dk, dv = flash_attn_backward(dout.contiguous(), q, k, v, out, lse, ctx.softmax_scale, ctx.causal,
                                         ctx.window_size, ctx.deterministic, ctx.softcap, alibi_slopes)
        return dq, dk, dv, None, None, None, None, None, None


class RotaryFunction(torch.autograd.Function):
    """Autograd wrapper of apply_rotary; the gradient is the rotation by the opposite angle (first order only)."""

    @staticmethod
    def forward(ctx, x, cos, sin, seqlen_offsets=0, interleaved=True, cu_seqlens=None):
        if cos.requires_grad or sin.requires_grad:
            raise ValueError("rotary tables have no gradient")
        tensor = isinstance(seqlen_offsets, torch.Tensor)
        ctx.save_for_backward(cos, sin, seqlen_offsets if tensor else None, cu_seqlens)
        ctx.offset, ctx.interleaved = 0 if tensor else seqlen_offsets, interleaved
        return apply_rotary(x, cos, sin, seqlen_offsets, interleaved, False, cu_seqlens)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        cos, sin, offsets, cu_seqlens = ctx.saved_tensors
        dx = apply_rotary(dy.contiguous(), cos, sin, ctx.offset if offsets is None else offsets, ctx.interleaved, True,
                          cu_seqlens)
        return dx, None, None, None, None, None
