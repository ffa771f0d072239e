"""Prompt attention with few rows and many keys: the keys are cut into blocks that run side by side
and are joined.  Against the float64 reference, and against the same call without a workspace (one
thread block walks all of a row's keys)."""
import ctypes

import numpy as np
import pytest
import torch

import _attention as A

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def _splits(kda, T, H, H_kv, d, dtype, n, table_stride=0, bs=16):
    """Bytes of workspace that the sizes ask for: more than none when the keys are cut."""
    a = kda.AttnPrefillArgs()
    a.n_seqs, a.n_heads, a.n_kv_heads, a.d, a.dtype, a.scale = n, H, H_kv, d, int(dtype == F32), 1.0
    a.total_tokens, a.q_stride, a.k_stride, a.v_stride, a.o_stride = T, H * d, H_kv * d, H_kv * d, H * d
    a.n_blocks, a.block_size, a.table_stride = 1, bs, table_stride
    a.block_table = 0x100 if table_stride else None
    return kda.kda_attn_prefill_workspace_size(a)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("d,H,H_kv,bs", [(128, 4, 2, 16), (64, 6, 1, 64), (128, 3, 3, 256)])
def test_few_queries_behind_a_long_cache(kda, cuda_device, dtype, d, H, H_kv, bs):
    """Sequences of very different lengths, so that some blocks of keys hold nothing for a row; an empty
    sequence, and one with more queries than positions."""
    new, kv = [1, 20, 3, 0, 9, 40], [2500, 1733, 3, 700, 5, 1200]
    c = A.Paged(20, kv, H_kv, d, bs, dtype, cuda_device)
    assert _splits(kda, sum(new), H, H_kv, d, dtype, len(new), c.table.shape[1], bs) > 0
    q = A.randn(21, (sum(new), H, d), dtype, cuda_device, 2.0)
    o, lse = kda.attn_prefill_paged(q, c.k, c.v, c.table, c.kv_lens, A.cu_of(new, cuda_device), want_lse=True)
    torch.cuda.synchronize()
    assert kda.kda_check_status() == 0
    keys, values = c.keys_values()
    firsts = [b - a for a, b in zip(new, kv)]
    A.check(o, lse, A.split(q, new), keys, values, firsts, d ** -0.5, dtype)
    assert (o[24:28] == 0).all() and (lse[24:28] == float("-inf")).all()
    # without a workspace: the same within the same bounds
    a = kda.AttnPrefillArgs(len(new), H, H_kv, d, int(dtype == F32), d ** -0.5, sum(new), H * d, 0, 0, H * d, q.data_ptr(), None,
                            None, o.zero_().data_ptr(), lse.zero_().data_ptr(), A.cu_of(new, cuda_device).data_ptr(),
                            c.k.data_ptr(), c.v.data_ptr(), c.table.data_ptr(), c.kv_lens.data_ptr(), c.n_blocks, bs, c.table.shape[1])
    cu = A.cu_of(new, cuda_device)
    a.cu_seqlens = cu.data_ptr()
    kda.kda_attn_prefill(a)
    A.check(o, lse, A.split(q, new), keys, values, firsts, d ** -0.5, dtype)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("d", [64, 128])
def test_one_long_prompt_of_few_heads(kda, cuda_device, dtype, d):
    lens, H = [2050], 2
    assert _splits(kda, lens[0], H, 1, d, dtype, 1) > 0
    q, k, v = A.packed(22, lens, H, 1, d, dtype, cuda_device, fused=True)
    ws = torch.zeros(_splits(kda, lens[0], H, 1, d, dtype, 1), dtype=torch.uint8, device=cuda_device)
    o, lse = kda.attn_prefill(q, k, v, A.cu_of(lens, cuda_device), want_lse=True, workspace=ws)
    assert kda.kda_check_status() == 0 and ws.any()
    rows = [0, 1, 63, 64, 127, 128, 500, 511, 512, 513, 1023, 1024, 1700, 2047, 2048, 2049]
    qs, ks, vs = A.np64(q), A.np64(k), A.np64(v)
    for i in rows:
        A.check(o[i:i + 1], lse[i:i + 1], [qs[i:i + 1]], [ks], [vs], [i], d ** -0.5, dtype)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("poison", [float("nan"), float("inf")])
def test_hidden_values_and_skipped_sequences(kda, cuda_device, dtype, poison):
    """Later tokens' NaN or infinities change nothing before them; a bad sequence's rows stay unwritten."""
    d, T = 128, 1300
    q, k, v = A.packed(23, [T], 2, 1, d, dtype, cuda_device)
    cu = torch.tensor([0, 1200, 1100], dtype=torch.int32, device=cuda_device)     # the second is bad
    assert _splits(kda, T, 2, 1, d, dtype, 2) > 0
    o, lse = torch.full_like(q, 7.0), torch.full((T, 2), 7.0, device=cuda_device)
    kda.attn_prefill(q, k, v, cu, o=o, lse=lse)
    assert kda.kda_check_status() == kda.KDA_DEV_BAD_SEQLENS
    assert (o[1200:] == 7).all() and (lse[1200:] == 7).all() and not (o[:1200] == 7).all()
    v2 = v.clone()
    v2[1150:, :, ::2] = poison
    o2, lse2 = torch.full_like(q, 7.0), torch.full((T, 2), 7.0, device=cuda_device)
    kda.attn_prefill(q, k, v2, cu, o=o2, lse=lse2)
    kda.kda_check_status()
    assert torch.equal(o2[:1150], o[:1150]) and torch.equal(lse2, lse) and torch.equal(o2[:1200, :, 1::2], o[:1200, :, 1::2])
    got = o2[1150:1200, :, ::2].float()
    assert (torch.isnan(got) if np.isnan(poison) else got == poison).all()


def test_workspace_refusals(kda, cuda_device):
    lens, H, d = [2050], 2, 128
    q, k, v = A.packed(24, lens, H, 1, d, BF, cuda_device)
    need = _splits(kda, 2050, H, 1, d, BF, 1)
    cu, o = A.cu_of(lens, cuda_device), torch.empty_like(q)
    ws = torch.empty(need + 256, dtype=torch.uint8, device=cuda_device)
    a = kda.AttnPrefillArgs(1, H, 1, d, 0, 0.1, 2050, H * d, d, d, H * d, q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(),
                            None, cu.data_ptr())
    a.workspace, a.workspace_bytes = ws.data_ptr() + 16, need
    assert kda.load().kda_attn_prefill(ctypes.byref(a), None) == kda.KDA_ERR_INVALID_ARG
    with pytest.raises(ValueError, match="contiguous"):
        kda.attn_prefill(q, k, v, cu, workspace=torch.empty((need, 2), dtype=torch.uint8, device=cuda_device)[:, 0])
