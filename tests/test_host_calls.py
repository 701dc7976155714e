"""CPU checks of the host side of the calls: what the entry points do with their arguments before anything is launched."""

import enum
import os

import pytest

from exact_tiled_attention_41_b200 import abi

FAKE = 0x10000


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(abi.LIB_PATH):
        from exact_tiled_attention_41_b200 import build
        build.build()
    return abi.load()


@pytest.mark.parametrize("offset,S", [(13, 4), (16, 1), (1 << 30, 4), (1, 1 << 30), (1 << 30, 1 << 30)])
def test_rotary_refuses_positions_past_the_tables(lib, offset, S):
    def call(**kw):
        a = dict(x=FAKE, y=2 * FAKE, rotary_cos=FAKE, rotary_sin=FAKE, cu_seqlens=None, seqlen_offsets=None,
                 seqlen_offset=offset, num_seqs=1, S=S, total=0, H=1, D=64, rotary_dim=32, rotary_len=16, x_stride_seq=64,
                 x_stride_tok=64, x_stride_head=64, y_stride_seq=64, y_stride_tok=64, y_stride_head=64, interleaved=1,
                 inverse=0, stream=0)
        a.update(kw)
        return abi.fa_rotary(**a)
    # a misaligned table, looked at later, stands for a call that would be launched
    assert call(rotary_cos=FAKE + 4) == abi.FA_ERR_INVALID_ARG
    assert call(rotary_cos=FAKE + 4, seqlen_offset=12, S=4) == abi.FA_ERR_ALIGNMENT


def test_the_device_is_that_of_the_first_tensor_however_it_is_passed(monkeypatch):
    import torch
    from exact_tiled_attention_41_b200 import attention as A

    class OnGpu1(torch.Tensor):
        is_cuda = property(lambda self: True)
        device = property(lambda self: "cuda:1")

        def get_device(self):
            return 1

    entered = []

    class Device:
        def __init__(self, d):
            entered.append(d)

        def __enter__(self):
            return self

        def __exit__(self, *exc):
            return False

    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch.cuda, "device", Device)
    t = torch.zeros(2).as_subclass(OnGpu1)
    run = A._on_device(lambda *args, **kwargs: len(entered))
    assert run(t, 1.0) == 1
    assert run(q=t) == 2
    assert run(softmax_scale=0.5, causal=True, q=t) == 3
    assert run(None, q=t) == 4
    assert run(1, scale=2.0) == 4
    assert entered == ["cuda:1"] * 4


def test_addresses_may_be_any_integers():
    class Address(enum.IntEnum):
        BUFFER = FAKE

    assert abi._ptr(Address.BUFFER) == FAKE and abi._ptr(FAKE) == FAKE and abi._ptr(None) is None
