"""Pins of the float64 attention reference: closed forms and invariants, no GPU."""
import numpy as np

from oracle import attention as oa


def _draw(seed, L, K, H, H_kv, d):
    r = np.random.RandomState(seed)
    return r.randn(L, H, d), r.randn(K, H_kv, d), r.randn(K, H_kv, d)


def test_one_key_returns_its_value():
    q, k, v = _draw(0, 1, 1, 4, 2, 8)
    o, lse, _ = oa.attention(q, k, v, 0, 0.3)
    assert np.allclose(o[0], np.repeat(v[0], 2, axis=0))
    assert np.allclose(lse[0, 3], 0.3 * k[0, 1] @ q[0, 3])


def test_equal_scores_average_the_values():
    q, k, v = _draw(1, 3, 5, 2, 1, 8)
    o, lse, _ = oa.attention(q * 0, k, v, 2, 1.0)
    for i in range(3):
        assert np.allclose(o[i], v[:3 + i].mean(0))
        assert np.allclose(lse[i], np.log(3 + i))


def test_values_move_the_output_and_keys_the_weights():
    q, k, v = _draw(2, 4, 9, 2, 2, 8)
    o, lse, _ = oa.attention(q, k, v, 5, 0.5)
    o2, lse2, _ = oa.attention(q, k, v + 3.0, 5, 0.5)
    assert np.allclose(o2, o + 3.0) and np.allclose(lse2, lse)
    shift = np.random.RandomState(3).randn(8)
    o3, lse3, _ = oa.attention(q, k + shift, v, 5, 0.5)      # every score of a row moves by the same amount
    assert np.allclose(o3, o) and np.allclose(lse3, lse + 0.5 * (q @ shift))


def test_rows_that_see_nothing():
    q, k, v = _draw(4, 5, 3, 1, 1, 8)
    o, lse, _ = oa.attention(q, k, v, -2, 1.0)
    assert (o[:2] == 0).all() and (lse[:2] == -np.inf).all() and np.isfinite(lse[2:]).all()


def test_two_blocks_of_keys_join_to_the_whole():
    """The join rule of split keys: weights exp(lse_p - lse)."""
    q, k, v = _draw(5, 1, 20, 2, 1, 8)
    whole, lse, _ = oa.attention(q, k, v, 19, 0.4)
    a, la, _ = oa.attention(q, k[:7], v[:7], 6, 0.4)
    b, lb, _ = oa.attention(q, k[7:], v[7:], 12, 0.4)
    assert np.allclose(np.exp(la - lse)[..., None] * a + np.exp(lb - lse)[..., None] * b, whole)


def test_plan_takes_blocks_in_order():
    p = oa.plan([0, 3, 4, 7], [5, 1, 0, 2], np.full((4, 3), -1) + np.array([[0], [10], [11], [13]]) * 0, [9, 8, 7, 6, 5], 1, 4, 10)
    assert p["cu_seqlens"] == [0, 5, 6, 6, 8] and p["kv_lens"] == [5, 4, 4, 9]
    assert p["table"][0].tolist() == [8, 7, -1] and p["table"][3][2] == 6 and p["free_end"] == 4
    assert p["slot_map"][:5] == [32, 33, 34, 35, 28] and p["slot_map"][8:] == [-1, -1]
