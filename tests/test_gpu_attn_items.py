"""Prompt attention in bf16 with several items of work to a thread block: what a block keeps of one
item's non-finite values never reaches another, and no item waits for a later one.

Sequences are short and many, so that every block takes a dozen items.  Each sequence holds NaN, +inf
or -inf in one column of v, at a key that the first half of an item's rows sees, or that only the second
half sees; rows that see it get it, everything else is the clean call's, bit for bit."""
import numpy as np
import pytest
import torch

import _attention as A

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
KINDS = [float("nan"), float("inf"), float("-inf")]


def _check(kda, call, v_at, marks, lens, firsts, d):
    """call() before and after the marked values are written.  marks: per sequence, (key, column, value)
    or None; v_at(s, key) is the view [H_kv, d] of that key's values."""
    clean, lse0 = call()
    assert kda.kda_check_status() == 0
    for s, mark in enumerate(marks):
        if mark:
            v_at(s, mark[0])[:, mark[1]] = mark[2]
    o, lse = call()
    assert kda.kda_check_status() == 0
    assert torch.equal(lse, lse0)
    want = clean.float()
    at = 0
    for n, first, mark in zip(lens, firsts, marks):
        if mark and n and mark[0] < first + n:
            want[at + max(0, mark[0] - first):at + n, :, mark[1]] = mark[2]
        at += n
    same = (o.float() == want) | (torch.isnan(o) & torch.isnan(want))
    assert same.all(), torch.nonzero(~same)[:4].tolist()


@pytest.mark.parametrize("d", [64, 128])
def test_values_that_only_the_second_row_tile_sees(kda, cuda_device, d):
    """One query head a key/value head: an item is 256 tokens, its first row tile has a key tile less."""
    n, L, H = 100, 256, 8
    lens = [L] * n
    q, k, v = A.packed(30, lens, H, H, d, BF, cuda_device)
    cu = A.cu_of(lens, cuda_device)
    rng = np.random.RandomState(31)
    marks = [(128 + rng.randint(128), rng.randint(d), KINDS[s % 3]) for s in range(n)]
    _check(kda, lambda: kda.attn_prefill(q, k, v, cu, want_lse=True), lambda s, key: v[s * L + key], marks, lens, [0] * n, d)


@pytest.mark.parametrize("d", [64, 128])
def test_notes_of_earlier_items_are_forgotten(kda, cuda_device, d):
    """In the same column throughout: items that hold a value at their first key, in turn with items that
    hold another one only where the second row tile sees it, and with items that hold none."""
    n, L, H = 120, 256, 8
    lens = [L] * n
    q, k, v = A.packed(37, lens, H, H, d, BF, cuda_device)
    cu = A.cu_of(lens, cuda_device)
    rng = np.random.RandomState(38)
    key = lambda s: 0 if s % 2 else 128 + rng.randint(128)
    marks = [(key(s), d - 1, KINDS[s // 2 % 3]) if s % 5 else None for s in range(n)]
    _check(kda, lambda: kda.attn_prefill(q, k, v, cu, want_lse=True), lambda s, key: v[s * L + key], marks, lens, [0] * n, d)


@pytest.mark.parametrize("d", [64, 128])
def test_ragged_items(kda, cuda_device, d):
    """Items of one to several key tiles, with and without such values, at keys of both row tiles."""
    rng = np.random.RandomState(32)
    lens = [int(x) for x in rng.choice([1, 7, 100, 128, 129, 250, 256, 300, 400, 513, 700], 150)]
    H, H_kv = 8, 4
    q, k, v = A.packed(33, lens, H, H_kv, d, BF, cuda_device)
    cu = A.cu_of(lens, cuda_device)
    begin = np.concatenate([[0], np.cumsum(lens)])
    marks = [(rng.randint(L), rng.randint(d), KINDS[rng.randint(3)]) if s % 4 else None for s, L in enumerate(lens)]
    _check(kda, lambda: kda.attn_prefill(q, k, v, cu, want_lse=True), lambda s, key: v[begin[s] + key], marks, lens,
           [0] * len(lens), d)


@pytest.mark.parametrize("d,bs", [(64, 32), (128, 16)])
def test_resumed_items(kda, cuda_device, d, bs):
    """Behind cached keys, four query heads a key/value head: row tiles of 32 tokens on both sides of a key
    tile's end; single tokens that see whole key tiles; more queries than keys; sequences without keys."""
    rng = np.random.RandomState(34)
    forms = [(64, 128 * 2 + 20), (64, 128 + 32), (1, 256), (1, 128), (40, 10), (3, 0), (70, 70), (200, 390), (33, 128 + 1)]
    picks = [forms[i] for i in rng.randint(len(forms), size=220)]
    new, kv = [a for a, _ in picks], [b for _, b in picks]
    H, H_kv = 16, 4
    c = A.Paged(35, kv, H_kv, d, bs, BF, cuda_device)
    q = A.randn(36, (sum(new), H, d), BF, cuda_device)
    cu = A.cu_of(new, cuda_device)
    marks = []
    for a, b in picks:
        back = rng.randint(min(b, 32)) if b else 0                # mostly among the last keys
        marks.append((b - 1 - back, rng.randint(d), KINDS[rng.randint(3)]) if b and rng.randint(4) else None)
    _check(kda, lambda: kda.attn_prefill_paged(q, c.k, c.v, c.table, c.kv_lens, cu, want_lse=True),
           lambda s, key: c.v[int(c.table_np[s, key // bs]), :, key % bs], marks, new, [b - a for a, b in picks], d)


@pytest.mark.parametrize("d", [64, 128])
def test_rows_of_a_warp_that_go_separate_ways(kda, cuda_device, d):
    """Rows move their maximum at different key tiles or never, end inside a warp, and lie on 16 bytes
    only, so that each lane stores its own."""
    lens = [300, 41, 129, 517, 77, 256, 3] * 8
    H, H_kv = 4, 2
    q, k, v = A.packed(39, lens, H, H_kv, d, BF, cuda_device)
    T = sum(lens)
    rng = np.random.RandomState(40)
    q *= torch.from_numpy(rng.choice([0.0, 0.1, 1.0, 4.0], (T, H, 1))).to(BF).to(cuda_device)
    k *= torch.from_numpy(rng.choice([0.1, 1.0, 6.0], (T, H_kv, 1), p=[0.5, 0.45, 0.05])).to(BF).to(cuda_device)
    buf = torch.full((T * (H * d + 8) + 8,), 7.0, dtype=BF, device=cuda_device)
    o = buf[8:].as_strided((T, H, d), (H * d + 8, d, 1))
    _, lse = kda.attn_prefill(q, k, v, A.cu_of(lens, cuda_device), o=o, want_lse=True)
    assert kda.kda_check_status() == 0
    A.check(o, lse, A.split(q, lens), A.split(k, lens), A.split(v, lens), [0] * len(lens), d ** -0.5, BF)
    assert (buf[:8] == 7).all() and (buf[8:].view(T, H * d + 8)[:, H * d:] == 7).all()
