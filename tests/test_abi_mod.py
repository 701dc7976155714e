"""CPU checks of the C entry points with score modifiers and rotary positions: bad arguments are refused before
anything is launched, and the workspace sizes follow their rules."""

import math
import os

import pytest

from exact_tiled_attention_41_b200 import abi

FAKE = 0x10000
S0 = 0


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(abi.LIB_PATH):
        from exact_tiled_attention_41_b200 import build
        build.build()
    return abi.load()


BAD_SCORES = [
    (dict(softcap=-1.0), abi.FA_ERR_INVALID_ARG),
    (dict(softcap=math.nan), abi.FA_ERR_INVALID_ARG),
    (dict(softcap=math.inf), abi.FA_ERR_INVALID_ARG),
    (dict(softcap=1e-30), abi.FA_ERR_UNSUPPORTED),
    (dict(softcap=1e30), abi.FA_ERR_UNSUPPORTED),
    (dict(alibi_slopes=FAKE, alibi_batch_stride=3), abi.FA_ERR_INVALID_ARG),     # fewer than Hq
    (dict(alibi_slopes=FAKE, alibi_batch_stride=-4), abi.FA_ERR_INVALID_ARG),
    (dict(alibi_slopes=FAKE + 2), abi.FA_ERR_ALIGNMENT),
]


@pytest.mark.parametrize("kw,want", BAD_SCORES)
def test_every_call_refuses_bad_modifiers(lib, kw, want):
    m = dict(softcap=0.0, alibi_slopes=None, alibi_batch_stride=0)
    m.update(kw)
    score = tuple(m.values())
    dense = (1, 4, 2, 128, 128, 128, 0.1, 1, -1, -1)
    assert abi.fa_fwd_mod(FAKE, FAKE, FAKE, FAKE, FAKE, *dense, *score, stream=S0) == want
    need = abi.fa_bwd_workspace_size(1, 4, 2, 128, 128, 128)
    assert abi.fa_bwd_mod(*([FAKE] * 9), *dense, 0, *score, FAKE, need, S0) == want
    packed = (2, 10, 10, 20, 20, 4, 2, 64, 0.1, 1, -1, -1)
    assert abi.fa_varlen_fwd_mod(*([FAKE] * 7), *packed, *score, stream=S0) == want
    need = abi.fa_varlen_bwd_workspace_size(2, 20, 20, 4, 2, 64)
    assert abi.fa_varlen_bwd_mod(*([FAKE] * 11), *packed, 0, *score, FAKE, need, S0) == want
    assert _kv(**m) == want


def test_a_scale_too_small_for_the_bias_is_refused(lib):
    assert abi.fa_fwd_mod(FAKE, FAKE, FAKE, FAKE, FAKE, 1, 4, 2, 128, 128, 128, 1e-25, 1, -1, -1, 0.0, FAKE, 0,
                          stream=S0) == abi.FA_ERR_UNSUPPORTED


def _kv(**kw):
    a = dict(q=FAKE, k_cache=FAKE, v_cache=FAKE, cache_seqlens=FAKE, k_new=FAKE, v_new=FAKE, seqlen_new=1,
             cache_batch_idx=None, block_table=None, max_blocks_per_seq=0, cache_batch=8, cache_capacity=1024,
             out=FAKE, lse=None, B=8, Hq=4, Hkv=2, Sq=3, D=128, softmax_scale=0.1, causal=1, window_left=-1,
             window_right=-1, num_splits=0, softcap=0.0, alibi_slopes=None, alibi_batch_stride=0, rotary_cos=None,
             rotary_sin=None, rotary_len=0, rotary_dim=0, rotary_interleaved=1, workspace=FAKE, workspace_bytes=1 << 40,
             stream=S0)
    a.update(kw)
    return abi.fa_fwd_kvcache_mod(**a)


ROT = dict(rotary_cos=FAKE, rotary_sin=FAKE, rotary_len=100, rotary_dim=64)


@pytest.mark.parametrize("kw,want", [
    (dict(ROT, rotary_dim=24), abi.FA_ERR_INVALID_ARG),              # README: a multiple of 16
    (dict(ROT, rotary_dim=144), abi.FA_ERR_INVALID_ARG),             # more than D
    (dict(ROT, rotary_dim=-16), abi.FA_ERR_INVALID_ARG),
    (dict(ROT, rotary_dim=0), abi.FA_ERR_INVALID_ARG),               # tables without a dimension
    (dict(ROT, rotary_sin=None), abi.FA_ERR_INVALID_ARG),
    (dict(ROT, rotary_len=0), abi.FA_ERR_INVALID_ARG),
    (dict(ROT, k_new=None, v_new=None, seqlen_new=0), abi.FA_ERR_INVALID_ARG),   # nothing new to rotate
    (dict(ROT, rotary_cos=FAKE + 4), abi.FA_ERR_ALIGNMENT),
])
def test_cache_call_refuses_bad_rotary_arguments(lib, kw, want):
    assert _kv(**kw) == want


def test_cache_workspace_holds_the_rotated_queries(lib):
    args = (8, 16, 4, 3, 128, 4096, 0, 0)
    plain = abi.fa_fwd_kvcache_mod_workspace_size(*args, 0)
    assert plain >= abi.fa_fwd_kvcache_ex_workspace_size(*args)      # the split with modifiers may be finer
    assert abi.fa_fwd_kvcache_mod_workspace_size(*args[:-1], 3, 0) == abi.fa_fwd_kvcache_ex_workspace_size(*args[:-1], 3)
    with_q = abi.fa_fwd_kvcache_mod_workspace_size(*args, 64)
    assert plain + 8 * 3 * 16 * 128 * 2 <= with_q <= plain + 8 * 3 * 16 * 128 * 2 + 255
    assert abi.fa_fwd_kvcache_mod_workspace_size(*args, 20) == 0
    assert _kv(**ROT, workspace_bytes=abi.fa_fwd_kvcache_mod_workspace_size(8, 4, 2, 3, 128, 1024, 0, 0, 64) - 1) == abi.FA_ERR_WORKSPACE


def _rotary(**kw):
    a = dict(x=FAKE, y=2 * FAKE, rotary_cos=FAKE, rotary_sin=FAKE, cu_seqlens=None, seqlen_offsets=None, seqlen_offset=0,
             num_seqs=2, S=4, total=0, H=3, D=64, rotary_dim=32, rotary_len=16, x_stride_seq=768, x_stride_tok=192,
             x_stride_head=64, y_stride_seq=768, y_stride_tok=192, y_stride_head=64, interleaved=1, inverse=0, stream=S0)
    a.update(kw)
    return abi.fa_rotary(**a)


@pytest.mark.parametrize("kw,want", [
    (dict(x=None), abi.FA_ERR_INVALID_ARG),
    (dict(rotary_sin=None), abi.FA_ERR_INVALID_ARG),
    (dict(num_seqs=0), abi.FA_ERR_INVALID_ARG),
    (dict(S=0), abi.FA_ERR_INVALID_ARG),
    (dict(cu_seqlens=FAKE), abi.FA_ERR_INVALID_ARG),                 # total missing
    (dict(seqlen_offset=-1), abi.FA_ERR_INVALID_ARG),
    (dict(rotary_len=0), abi.FA_ERR_INVALID_ARG),
    (dict(rotary_dim=24), abi.FA_ERR_INVALID_ARG),
    (dict(rotary_dim=80), abi.FA_ERR_INVALID_ARG),
    (dict(D=96), abi.FA_ERR_UNSUPPORTED),
    (dict(S=(1 << 30) + 1), abi.FA_ERR_UNSUPPORTED),
    (dict(x_stride_tok=188), abi.FA_ERR_ALIGNMENT),
    (dict(x_stride_head=-64), abi.FA_ERR_INVALID_ARG),
    (dict(y_stride_head=0), abi.FA_ERR_INVALID_ARG),                 # outputs on each other
    (dict(y_stride_tok=0), abi.FA_ERR_INVALID_ARG),
    (dict(y=FAKE, y_stride_tok=256), abi.FA_ERR_INVALID_ARG),        # in place with other strides
    (dict(x=FAKE + 8), abi.FA_ERR_ALIGNMENT),
    (dict(rotary_cos=FAKE + 4), abi.FA_ERR_ALIGNMENT),
    (dict(seqlen_offsets=FAKE + 1), abi.FA_ERR_ALIGNMENT),
])
def test_rotary_refuses_bad_arguments(lib, kw, want):
    assert _rotary(**kw) == want


def test_rotary_in_place_refuses_a_zeroed_tail(lib):
    assert _rotary(cu_seqlens=FAKE, total=8, y=FAKE, zero_tail=1) == abi.FA_ERR_INVALID_ARG


@pytest.mark.parametrize("kw,want", [
    (dict(rotary_cos=None), abi.FA_ERR_INVALID_ARG),
    (dict(rotary_len=0), abi.FA_ERR_INVALID_ARG),
    (dict(rotary_dim=8), abi.FA_ERR_INVALID_ARG),
    (dict(rotary_dim=272), abi.FA_ERR_UNSUPPORTED),
    (dict(base=1.0), abi.FA_ERR_INVALID_ARG),
    (dict(base=math.inf), abi.FA_ERR_INVALID_ARG),
    (dict(amplitude=math.nan), abi.FA_ERR_INVALID_ARG),
    (dict(scaling=4), abi.FA_ERR_INVALID_ARG),
    (dict(scaling=abi.FA_ROTARY_LINEAR, factor=0.5), abi.FA_ERR_INVALID_ARG),
    (dict(scaling=abi.FA_ROTARY_BY_PARTS, original_len=0), abi.FA_ERR_INVALID_ARG),
    (dict(scaling=abi.FA_ROTARY_BY_PARTS, low_rotations=4.0, high_rotations=4.0), abi.FA_ERR_INVALID_ARG),
    (dict(rotary_sin=FAKE + 8), abi.FA_ERR_ALIGNMENT),
])
def test_tables_refuse_bad_arguments(lib, kw, want):
    a = dict(rotary_cos=FAKE, rotary_sin=FAKE, rotary_len=16, rotary_dim=32, base=1e4, scaling=0, factor=2.0,
             original_len=2048, low_rotations=1.0, high_rotations=32.0, amplitude=1.0, stream=S0)
    a.update(kw)
    assert abi.fa_rotary_tables(**a) == want
