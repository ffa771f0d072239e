"""The plan's outputs and inputs: overlaps are refused, neighbours in one buffer are fine."""
import ctypes

import numpy as np
import pytest
import torch

import hybrid_linear_attention_kda_gb300 as kda
from hybrid_linear_attention_kda_gb300 import build as kbuild
from oracle import attention as oa

P, N, STRIDE, FREE, T = 0x100000, 5, 4, 7, 10
INPUTS = {"cached_lens": N, "new_lens": N, "free_blocks": FREE, "free_begin": 1}
OUTPUTS = {"free_end": 1, "block_table": N * STRIDE, "kv_lens": N, "cu_seqlens": N + 1, "slot_map": T, "positions": T}


@pytest.fixture(scope="module")
def lib():
    kbuild.build()
    return kda.load()


@pytest.mark.parametrize("given", INPUTS)
@pytest.mark.parametrize("out", OUTPUTS)
@pytest.mark.parametrize("end", ["same", "first", "last"])
def test_overlaps_are_refused(lib, given, out, end):
    a = kda.CachePlanArgs(N, 16, STRIDE, FREE, 8, T)
    for i, name in enumerate([*INPUTS, *OUTPUTS]):
        setattr(a, name, P + 0x1000 * i)
    at = getattr(a, given)
    # on the input's first element, or sharing one element with its start or its end
    shift = {"same": 0, "first": -4 * (OUTPUTS[out] - 1), "last": 4 * (INPUTS[given] - 1)}[end]
    setattr(a, out, at + shift)
    assert lib.kda_cache_plan(ctypes.byref(a), None) == kda.KDA_ERR_INVALID_ARG
    error = lib.kda_last_error().decode()
    assert error == f"{out} overlaps {given}" or {given, out} == {"free_begin", "free_end"}


@pytest.mark.gpu
def test_neighbours_in_one_buffer(kda, cuda_device):
    """More tokens than one thread block plans, all arrays side by side; the lengths stay as they were."""
    rng = np.random.RandomState(1)
    n, bs = 300, 16
    cached, new = rng.randint(0, 100, n), rng.randint(0, 20, n)
    have, need = -(-cached // bs), -(-(cached + new) // bs)
    perm = rng.permutation(int(need.sum()))
    table = np.full((n, int(need.max()) + 1), -1, np.int32)
    at = 0
    for s, h in enumerate(have):
        table[s, :h] = perm[at:at + h]
        at += h
    free, tokens = perm[at:], int(new.sum()) + 9
    parts = {"cached": cached, "kv": np.zeros(n), "new": new, "cu": np.zeros(n + 1), "begin": [0], "end": [-1], "free": free,
             "slots": np.zeros(tokens), "positions": np.zeros(tokens), "table": table.reshape(-1)}
    flat = torch.from_numpy(np.concatenate([np.asarray(x).astype(np.int32) for x in parts.values()])).to(cuda_device)
    x = dict(zip(parts, torch.split(flat, [len(p) for p in parts.values()])))
    kda.cache_plan(x["cached"], x["new"], x["table"].view(n, -1), x["free"], x["begin"], x["end"], block_size=bs,
                   n_blocks=len(perm), max_tokens=tokens, kv_lens=x["kv"], cu_seqlens=x["cu"], slot_map=x["slots"],
                   positions=x["positions"])
    assert kda.kda_check_status() == 0
    want = oa.plan(cached.tolist(), new.tolist(), table, free, 0, bs, tokens)
    for mine, theirs in [("table", "table"), ("kv", "kv_lens"), ("cu", "cu_seqlens"), ("slots", "slot_map"),
                         ("positions", "positions")]:
        assert np.array_equal(x[mine].cpu().numpy(), np.asarray(want[theirs]).reshape(-1)), mine
    assert int(x["end"]) == want["free_end"]
    assert np.array_equal(x["cached"].cpu().numpy(), cached) and np.array_equal(x["new"].cpu().numpy(), new)
    with pytest.raises(kda.KdaError, match="kv_lens overlaps cached_lens"):
        kda.cache_plan(x["cached"], x["new"], x["table"].view(n, -1), x["free"], x["begin"], x["end"], block_size=bs,
                       n_blocks=len(perm), max_tokens=tokens, kv_lens=x["cached"])
