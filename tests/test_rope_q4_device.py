"""Tensors of another device than the current one are refused by the rotation and the 4-bit cache's calls too.  Without a
GPU, with tensors that only say where they are."""
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


def _cache():
    codes, scales = _t(3, 2, 16, 32, dtype=torch.uint8), _t(3, 2, 16, 1, 2, dtype=torch.bfloat16)
    return kda.Q4Cache(codes, scales, codes, scales)


CALLS = {
    "norm_rope": lambda: kda.qk_norm_rope(_t(6, 4, 64), _t(6, 2, 64), _i(6)),
    "append_rope": lambda: kda.cache_append_rope(_t(6, 2, 64), _t(6, 2, 64), _i(6), None, _i(6), _t(3, 2, 16, 64), _t(3, 2, 16, 64)),
    "append_q4": lambda: kda.cache_append_q4(_t(6, 2, 64), _t(6, 2, 64), _i(6), _cache()),
    "unpack_q4": lambda: kda.cache_unpack_q4(_cache(), _i(1, 2), _i(1), _t(3, 2, 16, 64), _t(3, 2, 16, 64), _i(1, 2)),
    "decode_q4": lambda: kda.attn_decode_q4(_t(6, 4, 64), _cache(), _i(6, 2), _i(6)),
}


@pytest.mark.parametrize("call", CALLS)
def test_another_device_is_refused(monkeypatch, call):
    def refuse():
        raise AssertionError("the binding reached the library")
    monkeypatch.setattr(kda, "load", refuse)
    monkeypatch.setattr(attention, "_current_device", lambda: 0)
    with pytest.raises(ValueError, match="cuda:1, which is not the current device"):
        CALLS[call]()
