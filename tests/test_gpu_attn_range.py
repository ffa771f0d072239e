"""Products q . k near the ends of fp32's range: rows whose products are all far below zero, and scales
that make up for it or would take such numbers past the range.

Equal keys have equal scores, bit for bit, so that a row's result is the mean of the values it sees: off by
K u for the sums (u = 2^-24), 2^-20 for the exponentials and the division, half a step for the output and,
in bf16, 2 |score| u: its exponents are the scores' products with the scale less a rounded one, so that all
weights miss 1 by the same factor, which their rounding to bf16 takes off and their sum keeps.  The lse is
off by the score's own error, 2 (d + 4) u of its size, and by the sum's."""
import math

import pytest
import torch

import _attention as A

pytestmark = pytest.mark.gpu
F32, BF = torch.float32, torch.bfloat16


def _weights(n, score, dtype):
    return n * A.U + 2.0 ** -20 + (2 * abs(score) * A.U if dtype == BF else 0.0)


def _check(o, lse, score, values, firsts, dtype):
    """o [T, H, d], lse [T, H] of queries that see the first n of values [K, H_kv, d], n listed by query."""
    r = A.half_step(dtype)
    for i, n in enumerate(firsts):
        v = values[:n].double()
        G = o.shape[1] // v.shape[1]
        mean, spread = v.mean(0).repeat_interleave(G, 0), v.abs().mean(0).repeat_interleave(G, 0)
        bound = _weights(n, score, dtype) * spread * (1 + r) + r * mean.abs()
        assert ((o[i].double() - mean).abs() <= bound).all(), i
        ref = score + math.log(n)
        off = (lse[i].double() - ref).abs()
        assert (off <= 2 * (o.shape[2] + 4) * A.U * abs(score) + 2.0 ** -20 + n * A.U + 4 * A.U * abs(ref)).all(), i


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype,size,scale", [(F32, 2.0 ** 50, 1.0), (F32, 2.0 ** 60, 1.0), (F32, 2.0 ** 60, 2.0 ** -120),
                                              (BF, 2.0 ** 50, 2.0 ** -100), (BF, 2.0 ** 60, 2.0 ** -120)])
def test_products_far_below_zero(kda, cuda_device, dtype, d, size, scale):
    """Products of -d size^2, for prompts, resumed prompts (split and unsplit) and decode."""
    dev, H, H_kv, bs = cuda_device, 4, 2, 16
    score = -d * size * size * scale
    lens = [300, 1, 129]
    q, k, v = A.packed(1, lens, H, H_kv, d, dtype, dev)
    q, k = torch.full_like(q, size), torch.full_like(k, -size)
    o, lse = kda.attn_prefill(q, k, v, A.cu_of(lens, dev), scale=scale, want_lse=True)
    at = 0
    for n in lens:
        rows = [0, n // 2, n - 1]
        _check(o[at:at + n][rows], lse[at:at + n][rows], score, v[at:at + n], [i + 1 for i in rows], dtype)
        at += n
    kv = [700, 33, 16]
    c = A.Paged(2, kv, H_kv, d, bs, dtype, dev)
    c.k.fill_(-size)
    values = [torch.from_numpy(x) for x in c.keys_values()[1]]
    for new in ([3, 5, 1], [400, 33, 9]):
        q = torch.full((sum(new), H, d), size, dtype=dtype, device=dev)
        o, lse = kda.attn_prefill_paged(q, c.k, c.v, c.table, c.kv_lens, A.cu_of(new, dev), scale=scale, want_lse=True)
        at = 0
        for n, K, vs in zip(new, kv, values):
            _check(o[at:at + n].cpu(), lse[at:at + n].cpu(), score, vs, [K - n + 1 + i for i in range(n)], dtype)
            at += n
    q = torch.full((3, H, d), size, dtype=dtype, device=dev)
    o, lse = kda.attn_decode(q, c.k, c.v, c.table, c.kv_lens, scale=scale, want_lse=True)
    for s, (K, vs) in enumerate(zip(kv, values)):
        _check(o[s:s + 1].cpu(), lse[s:s + 1].cpu(), score, vs, [K], dtype)
    assert kda.kda_check_status() == 0


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("scale", [1e9, -1e20, 1e-30])
def test_empty_rows_at_any_scale(kda, cuda_device, dtype, scale):
    """More queries than positions: the rows that see nothing are zeros among rows that see equal keys."""
    dev, d, new, kv = cuda_device, 64, [140, 20], [130, 5]
    c = A.Paged(3, kv, 1, d, 16, dtype, dev)
    size = 2.0 ** -round(torch.tensor(abs(scale)).log2().item() / 2)
    c.k.fill_(size)
    q = torch.full((160, 2, d), size, dtype=dtype, device=dev)
    o, lse = kda.attn_prefill_paged(q, c.k, c.v, c.table, c.kv_lens, A.cu_of(new, dev), scale=scale, want_lse=True)
    assert kda.kda_check_status() == 0
    for at, n, K, vs in zip([0, 140], new, kv, c.keys_values()[1]):
        empty = n - K
        assert (o[at:at + empty] == 0).all() and (lse[at:at + empty] == float("-inf")).all()
        vs, r = torch.from_numpy(vs), A.half_step(dtype)
        for i in range(empty, n):
            m, spread = vs[:i - empty + 1].mean(0), vs[:i - empty + 1].abs().mean(0)
            bound = _weights(K, d * size * size * scale, dtype) * spread * (1 + r) + r * m.abs()
            assert ((o[at + i].double().cpu() - m).abs() <= bound).all()
