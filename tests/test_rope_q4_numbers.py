"""Numbers beyond fp32 reach the library as infinities, which it refuses by name, in the rotation's and the 4-bit cache's
calls as in the others.  Without a GPU: the library refuses them before it looks at a tensor."""
import pytest
import torch

import hybrid_linear_attention_kda_gb300 as kda
from hybrid_linear_attention_kda_gb300 import attention, build as kbuild, cache_q4, rope


class OnDevice0(torch.Tensor):
    is_cuda = property(lambda self: True)
    device = property(lambda self: torch.device("cuda", 0))

    def get_device(self):
        return 0


def _t(*shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype).as_subclass(OnDevice0)


def _i(*shape):
    return _t(*shape, dtype=torch.int32)


def _cache():
    codes, scales = (lambda: _t(3, 2, 16, 32, dtype=torch.uint8)), (lambda: _t(3, 2, 16, 1, 2, dtype=torch.bfloat16))
    return kda.Q4Cache(codes(), scales(), codes(), scales())


CALLS = {
    "norm_rope": ("eps", lambda x: kda.qk_norm_rope(_t(6, 4, 64), _t(6, 2, 64), _i(6), eps=x, q_out=_t(6, 4, 64), k_out=_t(6, 2, 64))),
    "append_rope": ("eps", lambda x: kda.cache_append_rope(_t(6, 2, 64), _t(6, 2, 64), _i(6), None, _i(6), _t(3, 2, 16, 64),
                                                           _t(3, 2, 16, 64), eps=x)),
    "decode_q4": ("scale", lambda x: kda.attn_decode_q4(_t(6, 4, 64), _cache(), _i(6, 2), _i(6), scale=x, o=_t(6, 4, 64),
                                                        workspace=_t(1 << 26, dtype=torch.uint8))),
}


@pytest.mark.parametrize("x", [1e39, -1e39, float("inf"), float("nan")])
@pytest.mark.parametrize("call", CALLS)
def test_refused_by_name(monkeypatch, call, x):
    kbuild.build()
    monkeypatch.setattr(attention, "_current_device", lambda: 0)
    for module in (rope, cache_q4):
        monkeypatch.setattr(module, "_current_stream", lambda index: None)
    name, run = CALLS[call]
    with pytest.raises(kda.KdaError, match=f"{name} must be finite"):
        run(x)
