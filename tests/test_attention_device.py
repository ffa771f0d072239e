"""Tensors of another device than the current one are refused: the library would launch on the current
one.  Without a GPU, with tensors that only say where they are."""
import pytest
import torch

import hybrid_linear_attention_kda_gb300 as kda
from hybrid_linear_attention_kda_gb300 import attention


class OnDevice1(torch.Tensor):
    is_cuda = property(lambda self: True)
    device = property(lambda self: torch.device("cuda", 1))

    def get_device(self):
        return 1


def _t(*shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype).as_subclass(OnDevice1)


def _i(*shape):
    return _t(*shape, dtype=torch.int32)


@pytest.fixture
def current(monkeypatch):
    def refuse():
        raise AssertionError("the binding reached the library")
    monkeypatch.setattr(kda, "load", refuse)

    def set_to(index):
        monkeypatch.setattr(attention, "_current_device", lambda: index)
    return set_to


CALLS = {
    "prefill": lambda: kda.attn_prefill(_t(6, 4, 64), _t(6, 2, 64), _t(6, 2, 64), _i(2)),
    "paged": lambda: kda.attn_prefill_paged(_t(6, 4, 64), _t(3, 2, 16, 64), _t(3, 2, 16, 64), _i(1, 2), _i(1), _i(2)),
    "decode": lambda: kda.attn_decode(_t(6, 4, 64), _t(3, 2, 16, 64), _t(3, 2, 16, 64), _i(6, 2), _i(6)),
    "append": lambda: kda.kda_cache_append(_t(6, 2, 64), _t(6, 2, 64), _i(6), _t(3, 2, 16, 64), _t(3, 2, 16, 64)),
    "plan": lambda: kda.cache_plan(_i(2), _i(2), _i(2, 3), _i(4), _i(1), _i(1), block_size=16, n_blocks=9, max_tokens=4,
                                   cu_seqlens=_i(3), kv_lens=_i(2), slot_map=_i(4), positions=_i(4)),
}


@pytest.mark.parametrize("call", CALLS)
def test_another_device_is_refused(current, call):
    current(0)
    with pytest.raises(ValueError, match="cuda:1, which is not the current device"):
        CALLS[call]()


def test_the_current_device_is_taken(current):
    current(1)
    assert attention._first(_t(6, 4, 64), "q")[4] == 1
