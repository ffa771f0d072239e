"""The 4-bit cache's calls with every tensor at 16 bytes' alignment and no more: caches and projections carved out of a
larger allocation."""
import numpy as np
import pytest
import torch

import _attention as A
import _q4
from oracle import cache_q4 as oq

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def _carved(x):
    """A copy of x that starts 16 bytes behind a multiple of 32."""
    room = torch.empty(x.numel() * x.element_size() + 64, dtype=torch.uint8, device=x.device)
    first = (16 - room.data_ptr()) % 32
    y = room[first:first + x.numel() * x.element_size()].view(x.dtype).view(x.shape)
    y.copy_(x)
    assert y.data_ptr() % 32 == 16
    return y


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("carved", [(True, True), (True, False), (False, True)])
def test_unpack(kda, cuda_device, dtype, d, carved):
    """Either full-width cache, or both, at an odd multiple of 16 bytes."""
    dev, H, bs, kv = cuda_device, 3, 16, [5, 0, 37]
    c = _q4.Paged(1, kv, H, d, bs, dtype, dev)
    to = np.array([[4, -1, -1], [-1, -1, -1], [1, 5, 0]], np.int32)
    first = [2, 0, 3]
    caches = [A.randn(2 + i, (6, H, bs, d), dtype, dev) for i in range(2)]
    caches = [_carved(t) if odd else t for t, odd in zip(caches, carved)]
    want = [t.cpu().clone() for t in caches]
    for x in range(2):
        v = torch.from_numpy(oq.values(c.codes[x], c.s[x], c.m[x])).to(dtype)
        for i, n in enumerate(kv):
            for j in range(first[i], n):
                want[x][to[i, j // bs], :, j % bs] = v[c.table_np[i, j // bs], :, j % bs]
    kda.cache_unpack_q4(c.cache, c.table, c.kv_lens, *caches, torch.from_numpy(to).to(dev),
                        first=torch.tensor(first, dtype=torch.int32, device=dev))
    assert kda.kda_check_status() == 0
    assert torch.equal(caches[0].cpu(), want[0]) and torch.equal(caches[1].cpu(), want[1])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d", [64, 128])
def test_append_and_decode(kda, cuda_device, dtype, d):
    dev, H, bs, kv = cuda_device, 2, 16, [5, 37]
    c = _q4.Paged(3, kv, H, d, bs, dtype, dev)
    c.cache = kda.Q4Cache(*(_carved(t) for t in c.cache))
    q = _carved(A.randn(4, (2, 4, d), dtype, dev))
    o, lse = c.decode(kda, q, o=_carved(torch.zeros_like(q)))
    assert kda.kda_check_status() == 0
    _q4.check(o, lse, q, c, d ** -0.5, dtype)
    k, v = (_carved(A.randn(5 + i, (3, H, d), dtype, dev)) for i in range(2))
    slots = [c.n_blocks * bs - 1, 0, 17]
    outs = [_carved(torch.zeros_like(k)) for _ in range(2)]
    kda.cache_append_q4(k, v, torch.tensor(slots, dtype=torch.int32, device=dev), c.cache, k_out=outs[0], v_out=outs[1])
    assert kda.kda_check_status() == 0
    for i, x in enumerate((k, v)):
        codes, s, m = oq.quantize(x.float().cpu().numpy())
        assert torch.equal(outs[i].cpu(), torch.from_numpy(oq.values(codes, s, m)).to(dtype))
        for t, slot in enumerate(slots):
            assert np.array_equal(c.cache[2 * i][slot // bs, :, slot % bs].cpu().numpy(), oq.packed(codes[t]))
            assert torch.equal(c.cache[2 * i + 1][slot // bs, :, slot % bs].cpu(), _q4.bf16(np.stack([s[t], m[t]], -1)))
