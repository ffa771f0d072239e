"""One token, as a slice of a row whose width is no multiple of 16 bytes: the distance to a token that is
not there is of no account."""
import pytest
import torch

import _attention as A

pytestmark = pytest.mark.gpu


def _odd(x):
    """The same token with a stride of one element more."""
    _, heads, d = x.shape
    y = torch.empty((2, heads * d + 1), dtype=x.dtype, device=x.device)[:1].as_strided(x.shape, (heads * d + 1, d, 1))
    return y.copy_(x)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_one_token_of_any_stride(kda, cuda_device, dtype):
    H, H_kv, d, bs = 4, 2, 64, 16
    c = A.Paged(1, [40], H_kv, d, bs, dtype, cuda_device)
    q, k, v = A.packed(2, [1], H, H_kv, d, dtype, cuda_device)
    cu = A.cu_of([1], cuda_device)
    calls = [lambda q, k, v, o: kda.attn_prefill(q, k, v, cu, o=o),
             lambda q, k, v, o: kda.attn_prefill_paged(q, c.k, c.v, c.table, c.kv_lens, cu, o=o),
             lambda q, k, v, o: kda.attn_decode(q, c.k, c.v, c.table, c.kv_lens, o=o)]
    for call in calls:
        want, got = torch.empty_like(q), _odd(torch.zeros_like(q))
        call(q, k, v, want)
        call(_odd(q), _odd(k), _odd(v), got)
        assert torch.equal(got, want)
    slot = torch.full((1,), 3, dtype=torch.int32, device=cuda_device)
    k1, v1, k2, v2 = c.k.clone(), c.v.clone(), c.k.clone(), c.v.clone()
    kda.kda_cache_append(k, v, slot, k1, v1)
    kda.kda_cache_append(_odd(k), _odd(v), slot, k2, v2)
    assert torch.equal(k1[0, :, 3], k[0]) and torch.equal(k2[0, :, 3], k[0]) and torch.equal(v2[0, :, 3], v[0])
    assert kda.kda_check_status() == 0
