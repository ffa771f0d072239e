"""Where rows are written, in which order sequences are taken, and how a prefix is cut change no
result.  The bounds are derived in ``_attention``."""
import pytest
import torch

import _attention as A

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("d,H,H_kv,bs", [(128, 40, 8, 32), (64, 6, 2, 16), (128, 3, 3, 64)])
def test_prefix_of_many_blocks_and_empty_suffixes(kda, cuda_device, dtype, d, H, H_kv, bs):
    """A prefix cut into several blocks of keys, with suffixes of zero, one and more behind it."""
    prefix, start = [1536, 768], [0, 9, 12]
    suffix = [0, 1, 0, 15, 16, 0, 33, 90, 0, 0, 2, 40]
    kv = [prefix[0 if s < 9 else 1] + x for s, x in enumerate(suffix)]
    c = A.Paged(31, kv, H_kv, d, bs, dtype, cuda_device, groups=[(0, 9, prefix[0] // bs), (9, 12, prefix[1] // bs)])
    q = A.randn(32, (12, H, d), dtype, cuda_device)
    start, prefix = (torch.tensor(x, dtype=torch.int32, device=cuda_device) for x in (start, prefix))
    o, lse = kda.attn_decode(q, c.k, c.v, c.table, c.kv_lens, group_start=start, prefix_lens=prefix, want_lse=True)
    assert kda.kda_check_status() == 0
    keys, values = c.keys_values()
    A.check(o, lse, A.split(q, [1] * 12), keys, values, [k - 1 for k in kv], d ** -0.5, dtype)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("first,gap", [(16, 0), (0, 16), (16, 48)])
def test_output_rows_at_any_16_bytes(kda, cuda_device, dtype, d, first, gap):
    """Rows that begin on 32 bytes, and rows that do not: the same bits, and nothing beside them."""
    lens, H, H_kv = [130, 1, 66], 6, 2
    T, size = sum(lens), torch.finfo(dtype).bits // 8
    q, k, v = A.packed(33, lens, H, H_kv, d, dtype, cuda_device)
    cu = A.cu_of(lens, cuda_device)
    want, _ = kda.attn_prefill(q, k, v, cu)
    stride = H * d + gap // size
    buf = torch.full((first // size + T * stride,), 7.0, dtype=dtype, device=cuda_device)
    rows = buf[first // size:].view(T, stride)
    o = rows[:, :H * d].view(T, H, d)
    kda.attn_prefill(q, k, v, cu, o=o)
    assert kda.kda_check_status() == 0
    assert torch.equal(o, want)
    assert (buf[:first // size] == 7).all() and (rows[:, H * d:] == 7).all()


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("n", [2, 20, 32, 33, 70])
def test_order_of_sequences(kda, cuda_device, dtype, n):
    """A sequence's result does not depend on its place in the batch, packed or paged."""
    lens = [1 + 37 * s * s % 300 for s in range(n)]
    kv = [x + 16 * (s % 5) for s, x in enumerate(lens)]
    d, H, H_kv, bs = 64, 4, 2, 16
    q, k, v = A.packed(34, lens, H, H_kv, d, dtype, cuda_device)
    c = A.Paged(35, kv, H_kv, d, bs, dtype, cuda_device)
    order = list(reversed(range(n)))
    parts = [torch.split(x, lens) for x in (q, k, v)]
    q2, k2, v2 = (torch.cat([p[s] for s in order]) for p in parts)
    cu, cu2 = A.cu_of(lens, cuda_device), A.cu_of([lens[s] for s in order], cuda_device)
    index = torch.tensor(order, device=cuda_device)
    a, la = kda.attn_prefill(q, k, v, cu, want_lse=True)
    b, lb = kda.attn_prefill(q2, k2, v2, cu2, want_lse=True)
    pa, _ = kda.attn_prefill_paged(q, c.k, c.v, c.table, c.kv_lens, cu)
    pb, _ = kda.attn_prefill_paged(q2, c.k, c.v, c.table[index].contiguous(), c.kv_lens[index].contiguous(), cu2)
    assert kda.kda_check_status() == 0
    for x, y in ((a, b), (la, lb), (pa, pb)):
        x, y = torch.split(x, lens), torch.split(y, [lens[s] for s in order])
        assert all(torch.equal(x[s], y[at]) for at, s in enumerate(order))
