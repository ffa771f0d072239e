"""Shared by the tests of the 4-bit cache: a paged cache in 4 bits with its float64 values, and the bound of decode attention
over it.

Bound, from the arithmetic (u = 2^-24; r = half a step of the output's type).  A position's key channel is m + n s, at most
A = 15 s + |m| in magnitude.
  scores   sums of d products in fp32, each accumulation cut or rounded (2 u), and the parts' factors: off by at most
           (d + 16) 2 u sum |q_c| A_c; fp32 q is cut into two parts of 11 bits, 4 u more of the same sum.  e bounds this over
           a batch, times scale, and twice for the base-2 detour.
  weights  are off by a factor 1 +- (2 e + 2^-20); times s they are rounded to fp16: w = 2^-11 (bf16), or 2^-21
           (two parts of 11 bits).  What falls under fp16's range is below K u of the sum, counted there.  A bf16 prefix has
           weights in bf16, w = 2^-8; an fp32 one fp32 weights, within 2^-21.
  output   the sums over K positions, accumulated in fp32 (2 u each), are of p s (n - 8) and p (m + 8 s); spread is the sum
           of their magnitudes:  |o - ref| <= (2 e + 2^-20 + 2 K u) spread + sum of w spread + r |ref|.
  lse      |lse - ref| <= e + 2^-20 + K u + 4 u |ref|
Positions of a shared prefix are full-width keys and values; their magnitudes take the places of A and of the spread.
"""
import numpy as np
import torch

import _attention as A
from oracle import attention as oa
from oracle import cache_q4 as oq

BF, F32 = torch.bfloat16, torch.float32


def bf16(x):
    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(BF)


class Paged:
    """A 4-bit cache in which sequence s holds own[s] positions behind the prefix[g] of its group; groups [(first, last)].
    The prefixes lie in full-width caches.  Whatever nobody owns has codes of 15 and NaN for scales (full width: NaN)."""

    def __init__(self, seed, own, H_kv, d, bs, dtype, dev, groups=(), prefix=(), extra=3, stride=None, std=1.0):
        rng = np.random.RandomState(seed)
        self.kv = list(own)
        before = [0] * len(own)
        for (a, b), length in zip(groups, prefix):
            for s in range(a, b):
                before[s] = length
                self.kv[s] += length
        need = [-(-n // bs) for n in self.kv]
        self.n_blocks = sum(n - b // bs for n, b in zip(need, before)) + extra
        wide_blocks = sum(length // bs for length in prefix) + extra
        perm, wide_perm = rng.permutation(self.n_blocks), rng.permutation(wide_blocks)
        self.table_np = np.full((len(own), stride or max(1, max(need, default=1))), -1, np.int32)
        codes = np.full((2, self.n_blocks, H_kv, bs, d), 15, np.uint8)
        s_, m_ = (np.full((2, self.n_blocks, H_kv, bs, d // 64), np.nan, np.float32) for _ in range(2))
        wide = np.full((2, wide_blocks, H_kv, bs, d), np.nan, np.float32)
        at = 0
        for (a, b), length in zip(groups, prefix):
            for j in range(length // bs):
                block = wide_perm[at]
                at += 1
                self.table_np[a:b, j] = block
                wide[:, block] = rng.randn(2, H_kv, bs, d) * std
        at = 0
        for i, n in enumerate(self.kv):
            for j in range(before[i] // bs, need[i]):
                block = perm[at]
                at += 1
                self.table_np[i, j] = block
                live = min(bs, n - j * bs)
                c, s, m = oq.quantize((rng.randn(2, H_kv, live, d) * std).astype(np.float32))
                codes[:, block, :, :live], s_[:, block, :, :live], m_[:, block, :, :live] = c, s, m
        self.codes, self.s, self.m = codes, s_, m_
        self.groups, self.before, self.dev = groups, before, dev
        self.upload()
        self.wide = [torch.from_numpy(x).to(dtype).to(dev) for x in wide]
        self.table = torch.from_numpy(self.table_np).to(dev)
        self.kv_lens = torch.tensor(self.kv, dtype=torch.int32, device=dev)
        self.group_start = torch.tensor([g[0] for g in groups] + [groups[-1][1]], dtype=torch.int32, device=dev) if groups else None
        self.prefix_lens = torch.tensor(list(prefix), dtype=torch.int32, device=dev) if groups else None

    def upload(self):
        import hybrid_linear_attention_kda_gb300 as kda
        t = []
        for x in range(2):
            t += [torch.from_numpy(oq.packed(self.codes[x])).to(self.dev),
                  bf16(np.stack([self.s[x], self.m[x]], -1)).to(self.dev)]
        self.cache = kda.Q4Cache(*t)

    def decode(self, kda, q, **kw):
        kw.setdefault("want_lse", True)
        if self.groups:
            kw |= dict(k_prefix=self.wide[0], v_prefix=self.wide[1], group_start=self.group_start, prefix_lens=self.prefix_lens)
        o, lse = kda.attn_decode_q4(q, self.cache, self.table, self.kv_lens, **kw)
        torch.cuda.synchronize()
        return o, lse

    def sequence(self, i):
        """(keys, values, key magnitudes, value magnitudes) [K, H_kv, d] of sequence i, in float64."""
        bs, n, b = self.codes.shape[3], self.kv[i], self.before[i]
        own = [self.table_np[i, j // bs] for j in range(b, n)]
        off = [j % bs for j in range(b, n)]
        out = []
        for x in range(2):
            wide = oa.gather(A.np64(self.wide[x]), self.table_np[i], b)
            v, size = _meaning(*(t[x][own, :, off] if own else t[x][:0, :, 0] for t in (self.codes, self.s, self.m)), x == 0)
            out.append((np.concatenate([wide, v]), np.concatenate([np.abs(wide), size])))
        return out[0][0], out[1][0], out[0][1], out[1][1]


class Packed:
    """What the 4-bit cache stands for after packed sequences of lengths kv, k and v [T, H_kv, d], were appended."""

    def __init__(self, k, v, kv):
        self.kv, self.quantized = kv, [oq.quantize(t.float().cpu().numpy()) for t in (k, v)]

    def sequence(self, i):
        at = slice(sum(self.kv[:i]), sum(self.kv[:i + 1]))
        (k, k_size), (v, v_size) = (_meaning(*(t[at] for t in q), x == 0) for x, q in enumerate(self.quantized))
        return k, v, k_size, v_size


def _meaning(codes, s, m, keys):
    """(values, magnitudes) of keys or values, in float64."""
    v = oq.values(codes, s, m)
    s, m = (np.repeat(t.astype(np.float64), 64, -1) for t in (s, m))
    return v, 15 * s + np.abs(m) if keys else s * np.abs(codes - 8.0) + np.abs(m + 8 * s)


def check(o, lse, q, c, scale, dtype, only=None):
    """Decode attention of every sequence (or those in `only`) against float64."""
    o, lse, qn = A.np64(o), A.np64(lse), A.np64(q)
    d = qn.shape[2]
    for i in range(len(c.kv)) if only is None else only:
        keys, values, key_size, value_size = c.sequence(i)
        ref, ref_lse, spread = attention(qn[i], keys, values, value_size, scale)
        before = c.before[i] if hasattr(c, "before") else 0
        wide = attention(qn[i], keys, values, np.where(np.arange(len(keys))[:, None, None] < before, value_size, 0), scale)[2]
        K, r = keys.shape[0], A.half_step(dtype)
        if K == 0:
            assert (o[i] == 0).all() and (lse[i] == -np.inf).all()
            continue
        e = 2 * (d + 18) * 2 * A.U * abs(scale) * float(np.abs(qn[i]).max(0) @ key_size.max((0, 1)))
        f = 2 * e + 2.0 ** -20 + 2 * K * A.U
        rounded = 2.0 ** -11 * (spread - wide) + 2.0 ** -8 * wide if dtype == BF else 2.0 ** -21 * spread
        bound = (f * spread + rounded) * (1 + r) + r * np.abs(ref) + 1e-30
        off = np.abs(o[i] - ref)
        assert np.isfinite(o[i]).all() and (off <= bound).all(), (i, K, float((off / bound).max()), np.argwhere(off > bound)[:4].tolist())
        assert (np.abs(lse[i] - ref_lse) <= e + 2.0 ** -20 + K * A.U + 4 * A.U * np.abs(ref_lse)).all(), (i, K, float(np.abs(lse[i] - ref_lse).max()))


def attention(q, k, v, v_size, scale):
    """One query [H, d] over [K, H_kv, d]: (o, lse, weighted magnitudes of the values)."""
    K, H_kv, d = k.shape
    G = q.shape[0] // H_kv
    o, spread, lse = np.zeros_like(q), np.zeros_like(q), np.full(q.shape[0], -np.inf)
    for h in range(q.shape[0] if K else 0):
        x = scale * (k[:, h // G] @ q[h])
        w = np.exp(x - x.max())
        lse[h] = x.max() + np.log(w.sum())
        o[h], spread[h] = (w @ y[:, h // G] / w.sum() for y in (v, v_size))
    return o, lse, spread
