"""Pins of the decode-loop oracle (CPU): several-axis rotation, attention
weights, the eviction rule and renumbered keys."""

import itertools

import numpy as np
import pytest

import oracle


@pytest.mark.parametrize("pairing", [oracle.NEOX_HALF, oracle.INTERLEAVED])
def test_equal_axes_are_one_position(pairing):
    rng = np.random.default_rng(0)
    rows, theta = rng.normal(size=(3, 16)), oracle.rope_inv_freq(16, 1e4)
    got = oracle.rotate_axes(rows, [5, 5, 5], [0, 0, 1, 1, 2, 2, 2, 0], theta, pairing, 0, 16)
    np.testing.assert_allclose(got, oracle.rotate(rows, 5, theta, pairing), rtol=0, atol=1e-14)


@pytest.mark.parametrize("pairing", [oracle.NEOX_HALF, oracle.INTERLEAVED])
def test_each_axis_turns_its_own_frequencies(pairing):
    rng = np.random.default_rng(1)
    rows, theta, axis = rng.normal(size=(2, 16)), oracle.rope_inv_freq(16, 1e4), [0, 1, 0, 1, 2, 2, 1, 0]
    got = oracle.rotate_axes(rows, [0, 9, 0], axis, theta, pairing, 0, 16)
    want = oracle.rotate(rows, 9, theta, pairing)
    a, b = oracle.rope_pairs(16, pairing)
    for f in range(8):
        for d in (a[f], b[f]):
            np.testing.assert_allclose(got[:, d], want[:, d] if axis[f] == 1 else rows[:, d], rtol=0, atol=1e-14)


def test_attention_weights_add_up_and_match_the_gathered_rows():
    rng = np.random.default_rng(2)
    bs, heads, d = 4, 2, 8
    kc, vc = rng.normal(size=(9, bs, heads, d)), rng.normal(size=(9, bs, heads, d))
    tables, lens = np.array([[3, 0, 7], [1, 8, 2], [5, 6, 4]]), [10, 0, 3]
    q = rng.normal(size=(3, 6, d))
    out, lse, w = oracle.attend_paged(q, kc, vc, tables, lens, bs, 0.3, np.zeros((9, heads, bs)))
    keys = kc[[3, 0, 7]].reshape(12, heads, d)[:10]
    vals = vc[[3, 0, 7]].reshape(12, heads, d)[:10]
    want, want_lse = oracle.attention_decode(q[0], keys, vals, 0.3)
    np.testing.assert_array_equal(out[0], want)
    np.testing.assert_array_equal(lse[0], want_lse)
    assert np.all(out[1] == 0) and np.all(np.isneginf(lse[1]))
    np.testing.assert_allclose(w[[3, 0, 7]].sum(axis=(0, 2)), [3, 3], atol=1e-12)   # three query heads each
    assert w[7, :, 2:].sum() == 0 and w[[1, 8, 2]].sum() == 0
    _, _, shared = oracle.attend_paged(q, kc, vc, tables, lens, bs, 0.3, np.zeros((9, 1, bs)))
    np.testing.assert_allclose(shared[:, 0], w.sum(axis=1), atol=1e-12)


def test_kept_slots_by_brute_force():
    rng = np.random.default_rng(3)
    for _ in range(40):
        n = int(rng.integers(1, 9))
        budget = int(rng.integers(1, n + 2))
        a = int(rng.integers(0, budget + 1))
        b = int(rng.integers(0, budget - a + 1))
        w = rng.integers(0, 3, size=n).astype(float)
        got = oracle.kept_slots(w, n, budget, a, b)
        if n <= budget:
            assert got == list(range(n))
            continue
        must = set(range(a)) | set(range(n - b, n))
        # the heaviest set; of equal sums the lexicographically smallest
        best = min((s for s in itertools.combinations(range(n), budget) if must <= set(s)),
                   key=lambda s: (-sum(w[i] for i in s if i not in must), s))
        assert got == list(best)
    assert oracle.kept_slots([np.nan, -np.inf, 0.0, -0.0], 4, 3, 0, 0) == [1, 2, 3]
    assert oracle.kept_slots([0.0, -0.0, 0.0], 3, 2, 0, 0) == [0, 1]


def test_renumbered_keys_are_forward_rope_at_their_new_places():
    rng = np.random.default_rng(4)
    bs, heads, d, n = 4, 2, 8, 11
    theta = oracle.rope_inv_freq(d, 1e4)
    raw = rng.normal(size=(n, heads, d))
    tables = np.array([[2, 0, 1]])
    kc, vc = np.zeros((3, bs, heads, d)), rng.normal(size=(3, bs, heads, d))
    for s in range(n):
        kc[tables[0][s // bs], s % bs] = oracle.rotate(raw[s], s, theta, oracle.NEOX_HALF)
    w = rng.random((3, heads, bs))
    k2, v2, w2, kept, lens = oracle.evict_tokens(kc, vc, w, tables, [n], bs, 6, 1, 2, True, theta, oracle.NEOX_HALF, 0, d)
    assert lens.tolist() == [6]
    for h in range(heads):
        for j, s in enumerate(kept[0, h]):
            to, frm = (tables[0][j // bs], j % bs), (tables[0][s // bs], s % bs)
            np.testing.assert_allclose(k2[to][h], oracle.rotate(raw[s][h], j, theta, oracle.NEOX_HALF), atol=1e-13)
            np.testing.assert_array_equal(v2[to][h], vc[frm][h])
            assert w2[to[0], h, to[1]] == w[frm[0], h, frm[1]]
