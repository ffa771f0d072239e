"""Prompt attention on the GPU against the float64 reference, at the sizes and masks where tiles,
pages and heads end unevenly.  The bounds are derived in ``_attention``."""
import numpy as np
import pytest
import torch

import _attention as A

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def _prefill(kda, q, k, v, lens, dev, **kw):
    o, lse = kda.attn_prefill(q, k, v, A.cu_of(lens, dev), want_lse=True, **kw)
    torch.cuda.synchronize()
    assert kda.kda_check_status() == 0
    return o, lse


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens", [[1], [2, 63, 1], [64, 65], [127, 128, 129], [0, 5, 0, 200, 0], [257, 300]])
@pytest.mark.parametrize("H,H_kv", [(2, 2), (8, 2)])
def test_prompt_lengths(kda, cuda_device, dtype, d, lens, H, H_kv):
    q, k, v = A.packed(1, lens, H, H_kv, d, dtype, cuda_device)
    o, lse = _prefill(kda, q, k, v, lens, cuda_device)
    A.check(o, lse, A.split(q, lens), A.split(k, lens), A.split(v, lens), [0] * len(lens), d ** -0.5, dtype)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("H,H_kv", [(1, 1), (3, 1), (5, 1), (14, 2), (48, 1), (100, 1), (128, 1)])
def test_head_groups(kda, cuda_device, dtype, H, H_kv):
    """Groups that divide a row tile, that do not, and that are larger than it."""
    lens, d = [70, 3, 41], 64
    q, k, v = A.packed(2, lens, H, H_kv, d, dtype, cuda_device)
    o, lse = _prefill(kda, q, k, v, lens, cuda_device)
    A.check(o, lse, A.split(q, lens), A.split(k, lens), A.split(v, lens), [0] * 3, d ** -0.5, dtype)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("scale", [-0.2, 0.0, 1.5])
def test_scale_and_fused_projection_views(kda, cuda_device, dtype, scale):
    """q, k and v as slices of one projection's output; peaked, flat and inverted scores."""
    lens, H, H_kv, d = [130, 77], 6, 3, 128
    q, k, v = A.packed(3, lens, H, H_kv, d, dtype, cuda_device, fused=True)
    assert not q.is_contiguous()
    o, lse = _prefill(kda, q, k, v, lens, cuda_device, scale=scale)
    A.check(o, lse, A.split(q, lens), A.split(k, lens), A.split(v, lens), [0, 0], scale, dtype)


@pytest.mark.parametrize("dtype", [F32, BF])
def test_output_into_a_view_leaves_its_neighbours(kda, cuda_device, dtype):
    lens, H, d = [50, 9], 4, 64
    q, k, v = A.packed(4, lens, H, H, d, dtype, cuda_device)
    buf = torch.full((70, H + 2, d), 7.0, dtype=dtype, device=cuda_device)
    o = buf[:59, 1:H + 1]
    kda.attn_prefill(q, k, v, A.cu_of(lens, cuda_device), o=o)
    torch.cuda.synchronize()
    A.check(o, None, A.split(q, lens), A.split(k, lens), A.split(v, lens), [0, 0], d ** -0.5, dtype)
    assert (buf[59:] == 7).all() and (buf[:, 0] == 7).all() and (buf[:, H + 1] == 7).all()


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("poison", [float("nan"), float("inf"), float("-inf")])
def test_hidden_positions_never_reach_a_result(kda, cuda_device, dtype, d, poison):
    """The last tokens of each sequence hold NaN or infinities in k and v: the queries before them, and
    the other sequences, are unchanged bit for bit; the queries that see them are not finite."""
    lens, H, H_kv = [100, 200, 330], 4, 2
    q, k, v = A.packed(5, lens, H, H_kv, d, dtype, cuda_device)
    clean, lse0 = _prefill(kda, q, k, v, lens, cuda_device)
    k2, v2 = k.clone(), v.clone()
    bad = [90, 100 + 137, 300 + 257]
    for t, end in zip(bad, np.cumsum(lens)):
        v2[t:end, :, ::3] = poison
        if np.isnan(poison):
            k2[t:end] = poison
    o, lse = _prefill(kda, q, k2, v2, lens, cuda_device)
    for t, end, begin in zip(bad, np.cumsum(lens), np.cumsum([0] + lens)):
        assert torch.equal(o[begin:t], clean[begin:t]) and torch.equal(lse[begin:t], lse0[begin:t])
        got = o[t:end, :, ::3].float()
        assert (torch.isnan(got) if np.isnan(poison) else got == poison).all()
        if not np.isnan(poison):
            keep = [c for c in range(d) if c % 3]
            assert torch.equal(o[t:end][:, :, keep], clean[t:end][:, :, keep])


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("bs,d,H,H_kv", [(16, 128, 8, 2), (32, 64, 6, 2), (64, 64, 4, 4), (128, 128, 4, 1), (256, 64, 3, 3)])
def test_paged_prompts(kda, cuda_device, dtype, bs, d, H, H_kv):
    """Queries behind a cached prefix; pages that end inside a tile; NaN in every unowned slot."""
    new, kv = [1, 40, 129, 17, 256, 5], [1, 40 + 256, 129 + 77, 300, 256, 5 + 511]
    c = A.Paged(6, kv, H_kv, d, bs, dtype, cuda_device)
    q = A.randn(7, (sum(new), H, d), dtype, cuda_device)
    o, lse = kda.attn_prefill_paged(q, c.k, c.v, c.table, c.kv_lens, A.cu_of(new, cuda_device), want_lse=True)
    torch.cuda.synchronize()
    assert kda.kda_check_status() == 0
    keys, values = c.keys_values()
    A.check(o, lse, A.split(q, new), keys, values, [b - a for a, b in zip(new, kv)], d ** -0.5, dtype)


@pytest.mark.parametrize("dtype", [F32, BF])
def test_more_queries_than_positions_leave_empty_rows(kda, cuda_device, dtype):
    new, kv, d = [20, 140, 3], [5, 130, 0], 64
    c = A.Paged(8, kv, 1, d, 16, dtype, cuda_device)
    q = A.randn(9, (sum(new), 2, d), dtype, cuda_device)
    o, lse = kda.attn_prefill_paged(q, c.k, c.v, c.table, c.kv_lens, A.cu_of(new, cuda_device), want_lse=True)
    torch.cuda.synchronize()
    assert kda.kda_check_status() == 0
    keys, values = c.keys_values()
    A.check(o, lse, A.split(q, new), keys, values, [b - a for a, b in zip(new, kv)], d ** -0.5, dtype)
    assert (o[:15] == 0).all() and (lse[:15] == float("-inf")).all() and (o[160:] == 0).all()


@pytest.mark.parametrize("dtype", [F32, BF])
def test_paged_equals_packed(kda, cuda_device, dtype):
    """The same keys from the cache and from packed tensors give the same bits."""
    lens, H, H_kv, d, bs = [200, 64, 333], 4, 2, 128, 16
    q, k, v = A.packed(10, lens, H, H_kv, d, dtype, cuda_device)
    want, _ = _prefill(kda, q, k, v, lens, cuda_device)
    c = A.Paged(11, lens, H_kv, d, bs, dtype, cuda_device)
    slots = [int(c.table_np[s, j // bs]) * bs + j % bs for s, n in enumerate(lens) for j in range(n)]
    kda.kda_cache_append(k, v, torch.tensor(slots, dtype=torch.int32, device=cuda_device), c.k, c.v)
    got, _ = kda.attn_prefill_paged(q, c.k, c.v, c.table, c.kv_lens, A.cu_of(lens, cuda_device))
    assert torch.equal(got, want)


def test_bad_sequences_are_skipped_and_flagged(kda, cuda_device):
    d = 64
    q, k, v = A.packed(12, [90], 2, 2, d, BF, cuda_device)
    o = torch.full_like(q, 7.0)
    cu = torch.tensor([0, 30, 20, 60, 300], dtype=torch.int32, device=cuda_device)     # the second and fourth are bad
    kda.attn_prefill(q, k, v, cu, o=o)
    assert kda.kda_check_status() == kda.KDA_DEV_BAD_SEQLENS
    # rows 20 .. 29 belong to the first and the third sequence alike
    A.check(o[:20], None, [A.np64(q[:20])], [A.np64(k[:20])], [A.np64(v[:20])], [0], d ** -0.5, BF)
    assert (o[60:] == 7).all()


@pytest.mark.parametrize("dtype", [F32, BF])
def test_bad_table_entries_and_lengths_are_flagged(kda, cuda_device, dtype):
    new, kv, d = [20, 30, 10], [200, 30, 10], 64
    c = A.Paged(13, kv, 1, d, 16, dtype, cuda_device)
    q = A.randn(14, (60, 2, d), dtype, cuda_device)
    c.table[0, 2], c.table[0, 5] = c.n_blocks, -5
    c.kv_lens[2] = c.table.shape[1] * 16 + 1
    o = torch.full_like(q, 7.0)
    kda.attn_prefill_paged(q, c.k, c.v, c.table, c.kv_lens, A.cu_of(new, cuda_device), o=o)
    assert kda.kda_check_status() == kda.KDA_DEV_BAD_SLOT | kda.KDA_DEV_BAD_SEQLENS
    keys, values = c.keys_values()
    A.check(o[20:50], None, [A.np64(q[20:50])], keys[1:2], values[1:2], [0], d ** -0.5, dtype)
    assert (o[50:] == 7).all()


@pytest.mark.parametrize("dtype", [F32, BF])
def test_same_call_twice_same_bits_on_another_stream(kda, cuda_device, dtype):
    lens, H, H_kv, d = [700, 33, 410], 8, 2, 128
    q, k, v = A.packed(15, lens, H, H_kv, d, dtype, cuda_device)
    a, la = _prefill(kda, q, k, v, lens, cuda_device)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    b, lb = kda.attn_prefill(q, k, v, A.cu_of(lens, cuda_device), want_lse=True, stream=side)
    side.synchronize()
    assert torch.equal(a, b) and torch.equal(la, lb)


@pytest.mark.parametrize("dtype", [F32, BF])
def test_long_ragged_prompts(kda, cuda_device, dtype):
    """Rows against thousands of keys, against the formula in float64 on the GPU."""
    lens, H, H_kv, d = [1, 1500, 2777], 4, 1, 128
    q, k, v = A.packed(16, lens, H, H_kv, d, dtype, cuda_device)
    q *= 3                                                    # peaked weights
    o, lse = _prefill(kda, q, k, v, lens, cuda_device)
    at = 0
    for n in lens:
        qs, ks, vs = (x[at:at + n].double() for x in (q, k, v))
        x = torch.einsum("ihd,jd->hij", qs, ks[:, 0]) * d ** -0.5
        x.masked_fill_(torch.ones((n, n), dtype=torch.bool, device=cuda_device).triu(1), float("-inf"))
        w = torch.softmax(x, -1)
        ref, spread = torch.einsum("hij,jd->ihd", w, vs[:, 0]), torch.einsum("hij,jd->ihd", w, vs[:, 0].abs())
        e = A.score_error(A.np64(qs), A.np64(ks), d ** -0.5, d)
        r = A.half_step(dtype)
        f = 2 * e + 2.0 ** -20 + n * A.U + (r if dtype == BF else 0.0)
        assert ((o[at:at + n].double() - ref).abs() <= f * spread + r * ref.abs() * (1 + f)).all()
        ref_lse = torch.logsumexp(x, -1).T
        assert ((lse[at:at + n].double() - ref_lse).abs() <= e + 2.0 ** -20 + n * A.U + 4 * A.U * ref_lse.abs()).all()
        at += n
