"""Python binding of the norms and position rotation of queries and keys (``include/kda_rope.h``), alone and on the
way into the paged cache.

Argument marshalling only, as in the package itself; the header states formulas, layouts and errors.  q, k and v may be
views of a fused projection's output.  All tensors are on the current device: the library launches there.
"""
import ctypes
import struct
from decimal import Decimal, localcontext

import torch

import hybrid_linear_attention_kda_gb300 as _kda
from .attention import _cache, _current_stream, _dev, _elsewhere, _empty, _F32, _first, _I32, _on, _shape, _tokens
from .attention_abi import PACK, CacheAppendRopeArgs, QkRopeArgs

_I64, _byref = torch.int64, ctypes.byref
_pack_rope, _pack_append = (struct.Struct(PACK[block]).pack for block in (QkRopeArgs, CacheAppendRopeArgs))
_TWO_PI = Decimal("6.28318530717958647692528676655900576839433879875021164194989")


def rope_turns(inv_freq, device=None):
    """The frequencies of a rotation in turns a position, as the calls take them: int64 [n], bit patterns of the header's
    64-bit fractions of a turn.  inv_freq: radians a position, a sequence of numbers or a tensor [n] (for the usual base:
    ``base ** (-2 * i / rot_dim)``, in float64).  Made once, where the weights are."""
    values = inv_freq.tolist() if isinstance(inv_freq, torch.Tensor) else [float(f) for f in inv_freq]
    if device is None:
        device = inv_freq.device if isinstance(inv_freq, torch.Tensor) else torch.device("cuda", torch.cuda.current_device())
    turns = []
    with localcontext() as ctx:
        ctx.prec = 80
        for f in values:
            x = Decimal(f)
            if not x.is_finite():
                raise ValueError(f"inv_freq must be finite (got {f})")
            x = int((x / _TWO_PI % 1 * 2 ** 64).to_integral_value()) % 2 ** 64
            turns.append(x - 2 ** 64 if x >= 2 ** 63 else x)
    return torch.tensor(turns, dtype=torch.int64, device=device)


def _rotation(turns, d, dev, index):
    """(address, rotated channels) of the frequencies."""
    if turns is None:
        return 0, 0
    n, = _shape(turns, "turns", 1)
    if 2 * n > d:
        raise ValueError(f"turns holds {n} frequencies for {d // 2} pairs of channels")
    return (_dev(turns, "turns", _I64, (n,), dev, index) if n else 0), 2 * n


def kda_qk_norm_rope(args: QkRopeArgs, stream=None):
    _kda._check(_kda.load().kda_qk_norm_rope(_byref(args), _kda._stream_handle(stream)))


def qk_norm_rope(q, k, positions, turns=None, *, interleaved=False, q_weight=None, k_weight=None, eps=1e-6, q_out=None,
                 k_out=None, stream=None):
    """Norms and rotation of queries and keys (``kda_qk_norm_rope``): q [T, H, d], k [T, H_kv, d]; positions int32 [T], -1
    for tokens to be skipped; turns from ``rope_turns``, rotating the first 2 n channels (None: none); q_weight, k_weight
    fp32 [d] (None: no norm).  The outputs are allocated unless given; q_out=q and k_out=k work in place.  Returns (q_out,
    k_out)."""
    if _elsewhere(stream, q):
        with _on(stream, q):
            return qk_norm_rope(q, k, positions, turns, interleaved=interleaved, q_weight=q_weight, k_weight=k_weight,
                                eps=eps, q_out=q_out, k_out=k_out)
    shape, dtype, code, dev, ix, qp, qs = _first(q, "q")
    T, H, d = shape
    kv = (T, _shape(k, "k", 3)[1], d)
    kp, ks = _tokens(k, "k", dtype, kv, dev, ix)
    pos = _dev(positions, "positions", _I32, (T,), dev, ix)
    tp, rot = _rotation(turns, d, dev, ix)
    wq = 0 if q_weight is None else _dev(q_weight, "q_weight", _F32, (d,), dev, ix)
    wk = 0 if k_weight is None else _dev(k_weight, "k_weight", _F32, (d,), dev, ix)
    q_out = _empty(shape, dtype=dtype, device=dev) if q_out is None else q_out
    k_out = _empty(kv, dtype=dtype, device=dev) if k_out is None else k_out
    qo, qos = _tokens(q_out, "q_out", dtype, shape, dev, ix)
    ko, kos = _tokens(k_out, "k_out", dtype, kv, dev, ix)
    a = _pack_rope(T, H, kv[1], d, code, rot, 1 if interleaved else 0, eps, 0, qs, ks, qos, kos, qp, kp, qo, ko, wq, wk, tp, pos)
    status = _kda.load().kda_qk_norm_rope(a, _current_stream(ix))
    if status:
        _kda._check(status)
    return q_out, k_out


def kda_cache_append_rope(args: CacheAppendRopeArgs, stream=None):
    _kda._check(_kda.load().kda_cache_append_rope(_byref(args), _kda._stream_handle(stream)))


def cache_append_rope(k, v, positions, turns, slot_map, k_cache, v_cache, *, q=None, q_out=None, interleaved=False,
                      q_weight=None, k_weight=None, eps=1e-6, stream=None):
    """k, normed and rotated, and v into the paged cache, and q, if given, normed and rotated to q_out
    (``kda_cache_append_rope``).  k, v [T, H_kv, d]; positions and slot_map int32 [T], as ``cache_plan`` gives them; caches
    [n_blocks, H_kv, block_size, d]; q [T, H, d]; the rest as for ``qk_norm_rope``.  Returns q_out, allocated unless given
    (None without q)."""
    if q is None and (q_out is not None or q_weight is not None):
        raise ValueError("q_out and q_weight come with q")
    if _elsewhere(stream, k):
        with _on(stream, k):
            return cache_append_rope(k, v, positions, turns, slot_map, k_cache, v_cache, q=q, q_out=q_out,
                                     interleaved=interleaved, q_weight=q_weight, k_weight=k_weight, eps=eps)
    shape, dtype, code, dev, ix, kp, ks = _first(k, "k")
    T, H_kv, d = shape
    vp, vs = _tokens(v, "v", dtype, shape, dev, ix)
    pos = _dev(positions, "positions", _I32, (T,), dev, ix)
    slots = _dev(slot_map, "slot_map", _I32, (T,), dev, ix)
    kc, vc, n_blocks, bs = _cache(k_cache, v_cache, dtype, H_kv, d, dev, ix)
    tp, rot = _rotation(turns, d, dev, ix)
    wq = 0 if q_weight is None else _dev(q_weight, "q_weight", _F32, (d,), dev, ix)
    wk = 0 if k_weight is None else _dev(k_weight, "k_weight", _F32, (d,), dev, ix)
    H = qp = qs = qo = qos = 0
    if q is not None:
        H = _shape(q, "q", 3)[1]
        qp, qs = _tokens(q, "q", dtype, (T, H, d), dev, ix)
        q_out = _empty((T, H, d), dtype=dtype, device=dev) if q_out is None else q_out
        qo, qos = _tokens(q_out, "q_out", dtype, (T, H, d), dev, ix)
    a = _pack_append(T, H, H_kv, d, code, rot, 1 if interleaved else 0, eps, 0, qs, ks, qos, 0, qp, kp, qo, 0, wq, wk, tp, pos,
                     vp, vs, slots, kc, vc, n_blocks, bs, 0)
    status = _kda.load().kda_cache_append_rope(a, _current_stream(ix))
    if status:
        _kda._check(status)
    return q_out
