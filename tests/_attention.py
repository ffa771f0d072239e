"""Shared by the attention tests: inputs, references and the error bounds they are held to.

Bounds, from the arithmetic alone (u = 2^-24, the fp32 half step; r = half a step of the storage
type, relative to the value):
  scores   a dot product of d terms in fp32 is off by at most (d + 2) u sum |q_c k_c|; with the
           scale and the log2(e) factor, two more roundings of the score itself.  e is the largest
           such error of a batch, in units of the exponent.
  weights  each is off by a factor 1 +- (2 e + 2^-20) (exp's own error included) and, for bf16, by
           its rounding r; sums over K keys add K u.
  output   |o - ref| <= (weights' factor) * sum_j w_j |v_j| + r |ref|
  lse      |lse - ref| <= e + 2^-20 + K u + 4 u |ref|
"""
import numpy as np
import torch

from oracle import attention as oa

U = 2.0 ** -24


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def np64(x):
    return x.detach().double().cpu().numpy()


def score_error(q, k, scale, d):
    """A bound on the fp32 error of scale * q . k over all pairs (times 2 for the base-2 detour)."""
    big = np.abs(q).max(axis=(0, 1)) @ np.abs(k).max(axis=(0, 1)) if q.size and k.size else 0.0
    return 2 * (d + 4) * U * abs(scale) * big


def check(o, lse, q, keys, values, firsts, scale, dtype):
    """o [T, H, d] and lse [T, H] of the sequences whose queries, keys and values are listed."""
    at = 0
    o = np64(o)
    lse = None if lse is None else np64(lse)
    for qs, ks, vs, first in zip(q, keys, values, firsts):
        L = qs.shape[0]
        ref, ref_lse, spread = oa.attention(qs, ks, vs, first, scale)
        K = max(1, ks.shape[0])
        e = score_error(qs, ks, scale, qs.shape[2])
        r = half_step(dtype)
        w = 2 * e + 2.0 ** -20 + K * U + (r if dtype == torch.bfloat16 else 0.0)
        bound = w * spread + r * np.abs(ref) * (1 + w) + 1e-30
        got = o[at:at + L]
        assert np.isfinite(got).all()
        bad = np.abs(got - ref) > bound
        assert not bad.any(), (L, K, float(np.abs(got - ref).max()), float((np.abs(got - ref) / bound).max()),
                               np.argwhere(bad)[:4].tolist())
        if lse is not None:
            gl = lse[at:at + L]
            none = ref_lse == -np.inf
            assert (gl[none] == -np.inf).all()
            off = np.abs(gl[~none] - ref_lse[~none])
            assert (off <= e + 2.0 ** -20 + K * U + 4 * U * np.abs(ref_lse[~none])).all(), float(off.max(initial=0))
        at += L


def randn(seed, shape, dtype, dev, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(dtype).to(dev)


def cu_of(lens, dev):
    return torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device=dev)


def packed(seed, lens, H, H_kv, d, dtype, dev, fused=False):
    T = int(sum(lens))
    if fused:
        x = randn(seed, (T, H + 2 * H_kv, d), dtype, dev)
        return x[:, :H], x[:, H:H + H_kv], x[:, H + H_kv:]
    return randn(seed, (T, H, d), dtype, dev), randn(seed + 1, (T, H_kv, d), dtype, dev), randn(seed + 2, (T, H_kv, d), dtype, dev)


def split(x, lens):
    x = np64(x)
    ends = np.cumsum(lens)
    return [x[e - n:e] for n, e in zip(lens, ends)]


class Paged:
    """A cache in which sequence s holds kv[s] positions; groups [(first, last, blocks)] share blocks.
    Everything that no sequence owns is NaN."""

    def __init__(self, seed, kv, H_kv, d, bs, dtype, dev, groups=(), extra=3, stride=None):
        rng = np.random.RandomState(seed)
        need = [-(-n // bs) for n in kv]
        shared = {}
        for a, b, blocks in groups:
            for s in range(a, b):
                shared[s] = (a, blocks)
        own = [n - (shared[s][1] if s in shared and shared[s][0] != s else 0) for s, n in enumerate(need)]
        n_blocks = sum(own) + extra
        perm = rng.permutation(n_blocks)
        self.table_np = np.full((len(kv), stride or max(1, max(need, default=1))), -1, np.int32)
        at = 0
        for s, n in enumerate(need):
            if s in shared and shared[s][0] != s:
                a, blocks = shared[s]
                self.table_np[s, :blocks] = self.table_np[a, :blocks]
                self.table_np[s, blocks:n] = perm[at:at + n - blocks]
                at += n - blocks
            else:
                self.table_np[s, :n] = perm[at:at + n]
                at += n
        k = np.full((n_blocks, H_kv, bs, d), np.nan, np.float32)
        v = k.copy()
        for s, n in enumerate(kv):
            for j in range(n):
                b = self.table_np[s, j // bs]
                if np.isnan(k[b, 0, j % bs, 0]):
                    k[b, :, j % bs] = rng.randn(H_kv, d)
                    v[b, :, j % bs] = rng.randn(H_kv, d)
        self.k = torch.from_numpy(k).to(dtype).to(dev)
        self.v = torch.from_numpy(v).to(dtype).to(dev)
        self.table = torch.from_numpy(self.table_np).to(dev)
        self.kv_lens = torch.tensor(kv, dtype=torch.int32, device=dev)
        self.kv, self.n_blocks = kv, n_blocks

    def keys_values(self):
        k, v = np64(self.k), np64(self.v)
        return ([oa.gather(k, self.table_np[s], n) for s, n in enumerate(self.kv)],
                [oa.gather(v, self.table_np[s], n) for s, n in enumerate(self.kv)])
