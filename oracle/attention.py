"""Float64 reference of the softmax-attention side: masked attention of one sequence, reads of a
paged cache, and the step plan, each written from its definition.

    x_ij = scale q_i . k_j over the keys j that query i sees,
    o_i = sum_j exp(x_ij) v_j / sum_j exp(x_ij),   lse_i = log sum_j exp(x_ij);
    a query that sees nothing has o = 0 and lse = -inf.
"""
import numpy as np


def attention(q, k, v, first, scale):
    """q [L, H, d], k, v [K, H_kv, d]; query i sees the keys 0 .. first + i.  Returns (o, lse,
    spread): spread [L, H, d] is sum_j w_ij |v_j|, the scale of rounding errors in the weights."""
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    L, H, d = q.shape
    G = H // k.shape[1]
    o, spread = np.zeros((L, H, d)), np.zeros((L, H, d))
    lse = np.full((L, H), -np.inf)
    for i in range(L):
        n = min(k.shape[0], first + i + 1)
        if n <= 0:
            continue
        for h in range(H):
            x = scale * (k[:n, h // G] @ q[i, h])
            m = x.max()
            w = np.exp(x - m)
            total = w.sum()
            lse[i, h] = m + np.log(total)
            o[i, h] = w @ v[:n, h // G] / total
            spread[i, h] = w @ np.abs(v[:n, h // G]) / total
    return o, lse, spread


def gather(cache, row, n):
    """The first n positions [n, H_kv, d] of a table row; cache [n_blocks, H_kv, block_size, d]."""
    bs = cache.shape[2]
    return np.stack([cache[row[j // bs], :, j % bs] for j in range(n)]) if n else np.zeros((0, cache.shape[1], cache.shape[3]))


def plan(cached, new, table, free, begin, block_size, max_tokens):
    """The step plan of valid inputs, token by token."""
    table = np.array(table)
    take, cu, slots, positions, kv = begin, [0], [], [], []
    for s, (c, t) in enumerate(zip(cached, new)):
        for pos in range(c, c + t):
            if pos % block_size == 0:
                table[s, pos // block_size] = free[take]
                take += 1
            slots.append(int(table[s, pos // block_size]) * block_size + pos % block_size)
            positions.append(pos)
        cu.append(len(slots))
        kv.append(c + t)
    pad = [-1] * (max_tokens - len(slots))
    return dict(table=table, cu_seqlens=cu, kv_lens=kv, slot_map=slots + pad, positions=positions + pad, free_end=take)
