"""The plain forms of speculative decoding pinned to closed forms, without a GPU."""
import math

import numpy as np
import pytest

import kv4_spec_ref as ref


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_is_a_complex_product(interleaved):
    """Pairs as complex numbers turn by exp(i angle): relative 2^-22 (two products and a sum, fp32), and the table's 2^-24."""
    rng = np.random.default_rng(0)
    x, rot = rng.standard_normal((5, 2, 64)).astype(np.float32), 48
    pos = np.array([0, 1, 77, 4000, 131071])
    y = ref.rotate(x, ref.table(131072, rot), pos, interleaved)
    a, b = (np.s_[..., 0:rot:2], np.s_[..., 1:rot:2]) if interleaved else (np.s_[..., :rot // 2], np.s_[..., rot // 2:rot])
    z = (x[a] + 1j * x[b].astype(np.float64)) * np.exp(1j * pos[:, None, None] * 10000.0 ** (-2.0 * np.arange(rot // 2) / rot))
    assert np.abs(y[a] + 1j * y[b].astype(np.float64) - z).max() <= 2.0 ** -21 * np.abs(z).max()
    assert np.array_equal(y[..., rot:], x[..., rot:]) and np.array_equal(y[0], x[0])


def test_logits_go_by_the_distance_of_positions():
    rng = np.random.default_rng(1)
    q, k = rng.standard_normal((2, 1, 1, 32)).astype(np.float32)
    tab = ref.table(5000, 32)
    dots = [float((ref.rotate(q, tab, [p + 37], False) * ref.rotate(k, tab, [p], False)).sum()) for p in (0, 500, 4900)]
    assert max(dots) - min(dots) <= 1e-4


def test_a_chain_is_causal_and_a_flat_tree_is_alone():
    for window in (0, 1, 3, 9):
        ok = ref.sees(ref.random_tree(5, None, "chain"), 12, window)
        for i in range(5):
            pos = 7 + i
            assert ok[i].tolist() == [j <= pos and (not window or j > pos - window) for j in range(12)]
        flat = ref.sees([-1] * 5, 12, window)
        for i in range(5):
            assert flat[i].nonzero()[0].tolist() == [j for j in range(7) if not window or j > 7 - window] + [7 + i]


def test_siblings_do_not_see_each_other_and_keys_below_zero_do_not_exist():
    parents = [-1, -1, 0, 0, 3]
    ok = ref.sees(parents, 8, 0)
    assert ok[:, :3].all() and ok[4, 3:].tolist() == [True, False, False, True, True] and ok[2, 3:].tolist() == [True, False, True, False, False]
    few = ref.sees(parents, 3, 0)  # tokens 0 and 1 have no key
    assert few.tolist() == [[False] * 3, [False] * 3, [True, False, False], [False, True, False], [False, True, True]]
    assert ref.sees(parents, 0, 0).shape == (5, 0)


def test_attention_of_equal_logits_is_a_mean():
    v = np.arange(12.0).reshape(4, 3)
    ok = np.array([[True, False, True, True], [False] * 4])
    out, lse = ref.attention(np.zeros((2, 1, 3)), np.ones((4, 3)), v, ok, 0.0, 1.0)
    assert np.allclose(out[0, 0], v[[0, 2, 3]].mean(0)) and math.isclose(lse[0, 0], math.log(3))
    assert (out[1] == 0).all() and np.isneginf(lse[1]).all()
