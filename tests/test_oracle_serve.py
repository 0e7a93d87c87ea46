"""Pins of the fp64 oracle of a serving step's operators."""

import numpy as np
import pytest

import oracle
from oracle import serve


def test_map_places_every_token_in_a_block_of_its_own():
    rng = np.random.default_rng(1)
    for bs in (1, 3, 16):
        lens = [5, 0, 40, 17, 16]
        grow = [1, 7, -25, bs, -16]
        cols = 60
        have = [-(-n // bs) for n in lens]
        order = list(rng.permutation(sum(have) + 30))
        tables = np.full((5, cols), -7)
        at = 0
        for r, n in enumerate(have):
            tables[r, :n] = order[at:at + n]
            at += n
        pile = order[at:]
        new, t, free, top, ptr, req, slot, pos, status = serve.map_tokens(lens, grow, tables, pile + [0] * at, len(pile), bs, 8 + bs + 3,
                                                                          [10, 0, 0, 5, 0])
        assert status == 0 and new == [n + g for n, g in zip(lens, grow)] and ptr == [0, 1, 8, 8, 8 + bs, 8 + bs]
        assert req[:8] == [0] + [1] * 7 and slot == [5] + list(range(7)) + [17 + j for j in range(bs)] + [-1] * 3
        assert pos[0] == 15 and pos[8] == 22 and pos[-1] == 0
        used = [int(x) for r, n in enumerate(new) for x in t[r][:-(-n // bs)]]
        # every block is in exactly one place: a table, or the pile
        assert sorted(used + [int(x) for x in free[:top]]) == sorted(order)


def test_map_refuses_in_order():
    tables = np.full((4, 4), -1)
    new, t, free, top, ptr, req, slot, pos, status = serve.map_tokens([0, 0, 0, 1], [4, 9, 4, 1], tables, [5, 6, 7, 0, 0, 0, 0, 0], 3, 4, 18)
    # the second needs three blocks where two are left; the third is behind it; the fourth needs none
    assert status == serve.CAPACITY and new == [4, 0, 0, 2] and top == 2 and t[0][0] == 7
    assert ptr == [0, 4, 13, 17, 18] and slot == [0, 1, 2, 3] + [-1] * 13 + [1]
    # token rows run out inside the second request
    new, *_, slot, _, status = serve.map_tokens([0, 0], [2, 2], np.full((2, 1), -1), [0, 1], 2, 4, 3)
    assert status == serve.CAPACITY and new == [2, 0] and slot == [0, 1, -1]
    # lengths and counts outside their limits
    new, *_, status = serve.map_tokens([-1, 9, 3], [1, 0, -4], np.zeros((3, 2), int), [0], 5, 4, 1)
    assert status == serve.BAD_LENGTH and new == [-1, 9, 3]
    # more blocks given back than the pile has places
    new, _, free, top, *_, status = serve.map_tokens([8, 8], [-4, -8], np.array([[0, 1], [0, 1]]), [9, 9], 1, 4, 0)
    assert status == serve.CAPACITY and new == [4, 8] and top == 2 and free == [9, 1]


def test_head_norm_is_scale_free_and_weighted():
    rng = np.random.default_rng(2)
    x, w = rng.standard_normal((3, 4, 64)), rng.standard_normal(64)
    y = serve.head_norm(x, w, 0.0)
    np.testing.assert_allclose(serve.head_norm(17.0 * x, w, 0.0), y, rtol=1e-13)
    np.testing.assert_allclose(np.square(y / w).mean(-1), 1.0, rtol=1e-12)
    np.testing.assert_allclose(serve.head_norm(x, w - 1.0, 0.0, 1.0), y, rtol=1e-12)
    np.testing.assert_allclose(serve.head_norm(np.zeros(8), np.ones(8), 1e-6), 0.0)


@pytest.mark.parametrize("window,n_first", [(0, 0), (1, 0), (5, 0), (5, 2), (3, 30), (1000, 4)])
def test_attend_tokens_is_decode_attention_slot_by_slot(window, n_first):
    rng = np.random.default_rng(3)
    k, v = rng.standard_normal((9, 4, 2, 16)), rng.standard_normal((9, 4, 2, 16))
    q = rng.standard_normal((4, 6, 16))
    tables, slot = np.array([[3, 1, 8, 0], [2, 4, 7, 6]]), [13, 2, -1, 9]
    out, lse = serve.attend_tokens(q, k, v, tables, [0, 2, 4], slot, 4, 0.3, window, n_first)
    for i, (r, s) in enumerate(zip([0, 0, 1, 1], slot)):
        slots = [t for t in range(s + 1) if not window or s - t < window or t < n_first]
        if not slots:
            assert np.all(out[i] == 0) and np.all(np.isneginf(lse[i]))
            continue
        # the same slots alone, in a cache of their own
        page = np.array([tables[r][t // 4] for t in slots]), np.array([t % 4 for t in slots])
        own_k, own_v = k[page][:, None], v[page][:, None]
        want, want_lse, _ = oracle.attend_paged(q[i:i + 1], own_k, own_v, np.arange(len(slots))[None], [len(slots)], 1, 0.3)
        np.testing.assert_allclose(out[i], want[0], rtol=1e-12, atol=1e-14)
        np.testing.assert_allclose(lse[i], want_lse[0], rtol=1e-12)


def test_attend_shared_is_paged_attention():
    rng = np.random.default_rng(4)
    k, v = rng.standard_normal((12, 4, 2, 16)), rng.standard_normal((12, 4, 2, 16))
    q = rng.standard_normal((4, 6, 16))
    prefix = 10
    tables = np.array([[5, 2, 9, 1], [5, 2, 0, 3], [5, 2, 8, 4], [5, 2, 6, 7]])
    # block 11 holds slots 8, 9 of the prefix: the same rows in each request's own block
    for r in range(4):
        for c in (k, v):
            c[tables[r][2], :2] = c[11, :2]
    lens = [16, 7, 0, 11]
    out, lse = serve.attend_shared(q, k, v, [5, 2, 11], prefix, tables, lens, 4, 0.3)
    want, want_lse, _ = oracle.attend_paged(q, k, v, tables, lens, 4, 0.3)
    np.testing.assert_allclose(out, want, rtol=1e-12, atol=1e-14)
    np.testing.assert_allclose(lse[[0, 1, 3]], want_lse[[0, 1, 3]], rtol=1e-12)
    assert np.all(np.isneginf(lse[2]))


def test_write_normed_is_norm_then_turn():
    rng = np.random.default_rng(5)
    q, k, w = rng.standard_normal((3, 4, 64)), rng.standard_normal((3, 2, 64)), rng.standard_normal((2, 64))
    theta = oracle.rope_inv_freq(64, 1e4)
    pos = np.array([[3, 1000, -5]])
    qq, kk = serve.write_normed(q, k, w[0], None, 1e-6, 0.0, pos, [0] * 32, theta, oracle.NEOX_HALF, 0, 64)
    for i in range(3):
        back = oracle.rotate_axes(qq[i], -pos[:, i], [0] * 32, theta, oracle.NEOX_HALF, 0, 64)
        np.testing.assert_allclose(back, serve.head_norm(q[i], w[0], 1e-6), atol=1e-11)
        back = oracle.rotate_axes(kk[i], -pos[:, i], [0] * 32, theta, oracle.NEOX_HALF, 0, 64)
        np.testing.assert_allclose(back, k[i], atol=1e-11)
