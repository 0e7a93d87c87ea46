"""Attention weights that enter the value product in two bf16 parts: single tokens
and shared prefixes, long ones in tiles and short ones row by row, keep 16 bits of
them, as pic_attend_paged does.

Tolerance.  A part rounds what is left to it by half a step, 2^-8 of it: both leave
2^-16 of a weight.  Sums over T slots add up to 2 T products, 2^-23 each.  Scores: as in
test_gpu_serve.py, (D + 8) 2^-23 sum |q k|; so that their term does not
hide the weights', keys have only four dims that are not zero.  The exponential:
2^-20.  All are relative to sum p |v|; the output adds half a step of bf16, 2^-8 of its
value."""

import math

import numpy as np
import pytest
import torch

import test_gpu_serve as serving
from position_independent_kv_stitch_gb300 import pic
from test_gpu_decode import Cache

PART, TWO_PARTS = 2.0 ** -8, 2.0 ** -16


def _expected(q, k, v, seen, scale):
    """Softmax attention in 64 bits, the weights, the log-sum-exp, and the bound on a score's error."""
    (hk, t, d), (n, hq, _) = k.shape, q.shape
    qd = q.double().reshape(n, hk, hq // hk, d)
    x = (torch.einsum("nhgd,htd->nhgt", qd, k) * scale).masked_fill(~seen[:, None, None], -math.inf)
    size = (torch.einsum("nhgd,htd->nhgt", qd.abs(), k.abs()) * abs(scale)).masked_fill(~seen[:, None, None], 0.0)
    lse = torch.logsumexp(x, -1)
    p = torch.exp(x - torch.where(lse.isinf(), 0.0, lse)[..., None])
    return torch.einsum("nhgt,htd->nhgd", p, v), p, lse, size.amax(-1) * (d + 8) * 2.0 ** -23


def _limit(want, p, v, s_err, seen, weight):
    rel = 2 * s_err + 2.0 ** -20 + 2 * seen.sum(-1)[:, None, None] * 2.0 ** -23 + weight
    off = rel[..., None] * torch.einsum("nhgt,htd->nhgd", p, v.abs())
    return off + 2.0 ** -8 * (want.abs() + off) + 1e-38


def _assert_rows(q, k, v, seen, scale, out, lse, what):
    if k.shape[1] == 0:
        assert bool((out == 0).all()) and bool((lse == -math.inf).all()), what
        return
    want, p, want_lse, s_err = _expected(q, k, v, seen, scale)
    lim = _limit(want, p, v, s_err, seen, TWO_PARTS)
    err = (out.double().reshape(want.shape) - want).abs()
    assert bool((err <= lim).all()), (what, float((err / lim).max()))


@pytest.fixture
def exact(monkeypatch):
    pic.load(build_if_missing=True)
    monkeypatch.setattr(serving, "_assert_rows", _assert_rows)


def _few_dims(c):
    c.k[..., 4:] = 0
    return c


@pytest.mark.gpu
@pytest.mark.parametrize("heads,hq,d,bs", [(2, 8, 128, 16), (8, 32, 128, 16), (3, 15, 64, 17), (2, 32, 256, 64), (1, 40, 128, 5)])
@pytest.mark.parametrize("window,n_first", [(0, 0), (33, 4)])
def test_single_tokens(exact, heads, hq, d, bs, window, n_first):
    lens = [1, 2, 5, 77, 16, 200, 15, 129]
    c = _few_dims(Cache(heads=heads, d=d, bs=bs, lens=lens, seed=hq))
    serving._attend(c, [[n - 1] for n in lens], hq, window, n_first, scale=0.5)
    c.close()


@pytest.mark.gpu
def test_single_tokens_beside_prompts(exact):
    """Of a call with prompts, the requests of one token."""
    lens = [300, 40, 7, 150, 90]
    c = _few_dims(Cache(heads=2, lens=lens, seed=3))
    serving._attend(c, [list(range(300)), [39], [6], list(range(100, 150)), [89]], 8, scale=0.5, check=(1, 2, 4))
    c.close()


@pytest.mark.gpu
@pytest.mark.parametrize("heads,hq,d,bs", [(2, 8, 128, 16), (5, 15, 64, 17), (2, 32, 256, 64)])
@pytest.mark.parametrize("prefix", [3, 150])
def test_short_prefixes(exact, heads, hq, d, bs, prefix):
    c = _few_dims(serving.Shared(prefix, [1, 0, 77, 16, None, 40], heads=heads, d=d, bs=bs, seed=hq))
    serving._shared(c, hq, scale=0.5)
    c.close()


@pytest.mark.gpu
@pytest.mark.parametrize("heads,hq,d,bs,n_req,slots", [(8, 32, 128, 16, 5, 33000), (8, 32, 128, 16, 36, 33000), (8, 32, 64, 16, 36, 40003),
                                                       (8, 32, 64, 16, 9, 40003), (2, 16, 256, 64, 12, 40000), (8, 32, 128, 5, 36, 33000),
                                                       (2, 8, 256, 4, 20, 33000), (1, 200, 128, 16, 30, 70000)])
@pytest.mark.parametrize("prefix", [5, 130, 300])
def test_prefixes_in_tiles(exact, heads, hq, d, bs, n_req, slots, prefix):
    """A prefix of few slots in a table of many, which goes in tiles: of one row block or two, from wide copies or rows."""
    c = _few_dims(serving.Shared(prefix, [3 * r % 50 for r in range(n_req)], heads=heads, d=d, bs=bs, seed=n_req))
    table = np.concatenate([c.prefix_table, np.full(slots // bs - len(c.prefix_table), -1, np.int32)])
    serving._shared(c, hq, scale=0.5, prefix_table=table)
    c.close()


@pytest.mark.parametrize("t", [5, 130, 300])
def test_the_tolerance_tells_one_part_from_two(t):
    g = torch.Generator().manual_seed(t)
    q, k, v = (torch.randn(s, generator=g).to(torch.bfloat16).double() for s in ((36, 8, 128), (2, t, 128), (2, t, 128)))
    k[..., 4:] = 0
    seen = torch.ones(36, t, dtype=torch.bool)
    want, p, _, s_err = _expected(q, k, v, seen, 0.5)
    lim = _limit(want, p, v, s_err, seen, TWO_PARTS)
    top = p / p.amax(-1, keepdim=True)
    one = top.to(torch.bfloat16).double()
    two = one + (top - one).to(torch.bfloat16).double()
    assert bool(((top - one).abs() <= PART * top).all()) and bool(((top - two).abs() <= TWO_PARTS * top).all())
    for weights, fits in ((one, False), (two, True)):
        out = (torch.einsum("nhgt,htd->nhgd", weights, v) / top.sum(-1, keepdim=True)).to(torch.bfloat16).double()
        assert bool(((out - want).abs() <= lim).all()) is fits
